// csrc/sample.cu's kernel, one row on one cluster, under a chosen schedule.
#include "emulator.h"

#include "sample_source.inc"

struct Launch {
    SampleArgs a;
    bool bf16, filter;
};

static void body(const void *p) {
    const Launch &l = *static_cast<const Launch *>(p);
    if (l.filter) {
        if (l.bf16) sample_kernel<true, true, 512, 1>(l.a);
        else sample_kernel<false, true, 512, 1>(l.a);
    } else {
        if (l.bf16) sample_kernel<true, false, 512, 2>(l.a);
        else sample_kernel<false, false, 512, 2>(l.a);
    }
}

// launch()'s status; *early counts accesses to CTAs that were not there,
// *syncs cluster barriers.
extern "C" int sample_row(const void *x, int bf16, int V, int C, const float *u, const float *temperature,
                          const int *top_k, const float *top_p, const float *min_p, int lag, int who, int from,
                          int64_t *token, float *logp, float *logp_all, int *kept, int *early,
                          int *syncs) {
    Launch l = {};
    l.bf16 = bf16;
    l.filter = temperature || top_k || top_p || min_p;
    const int E = bf16 ? 8 : 4;
    const int64_t chunks = (V + E - 1 + E - 1) / E;
    l.a.x = x;
    l.a.ld = V;
    l.a.B = 1;
    l.a.V = V;
    l.a.u = u;
    l.a.temperature = temperature;
    l.a.top_k = top_k;
    l.a.top_p = top_p;
    l.a.min_p = min_p;
    l.a.token = token;
    l.a.logp = logp;
    l.a.logp_all = logp_all;
    l.a.kept = kept;
    l.a.chunks_per_warp = warp_chunks(C, 512, chunks);
    const int status = emu::launch(body, &l, C, 512, l.filter ? filter_smem(C, chunks) : kHead,
                                   (emu::Lag)lag, who, from);
    *early = emu::cluster.early;
    *syncs = (int)emu::cluster.syncs;
    return status;
}
