// Backward of the gated activation h = silu(gate) up, with the 1x128
// quantization of both gradients fused: the inputs of the gate and up
// projections' DGrads, without BF16 gradients in between.  With s = 1 / (1 +
// e^-g):
//   dup = dh g s,   dgate = dh up s (1 + g (1 - s)).
// Both s and 1 - s come from t = e^-|g| in (0, 1]: r = 1 / (1 + t) is the larger
// of them and t r the smaller, so neither overflows nor cancels.  t is one
// exp2 of a binary32 product (relative error 2^-22 + |g| 2^-24), r a reciprocal
// approximation with one Newton step (its error below 2^-23); then the 1x128
// group rule of quant_rule.cuh on the binary32 values.
//
// Work is split as in the forward's quantizer: half a warp takes a group of 128
// (8 elements a lane, one 16-byte load of each tensor), a warp two neighbouring
// groups of a row, consecutive warps consecutive rows; the next item's loads go
// out before an item's arithmetic.
#include <cuda_bf16.h>

#include "jet_common.cuh"
#include "stream_ld.cuh"
#include "quant_rule.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kCtasPerSm = 4;

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// -dgate and -dup of one element, for the division routine
__device__ __forceinline__ void neg_gradients(float g, float u, float d, float &ng, float &nu) {
    const float t = exp2f(-1.4426950408889634f * fabsf(g));
    const float q = 1.0f + t;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(q));  // q in [1, 2]
    r = fmaf(fmaf(-q, r, 1.0f), r, r);
    const float tr = t * r;
    const float s = g >= 0.0f ? r : tr, c = g >= 0.0f ? tr : r;  // s and 1 - s
    const float nd = -d * s;
    nu = nd * g;
    ng = nd * u * fmaf(g, c, 1.0f);
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm)
swiglu_bwd_kernel(const uint16_t *__restrict__ gate, const uint16_t *__restrict__ up, int64_t ld,
                  const uint16_t *__restrict__ dh, int64_t M, int64_t F, uint8_t *__restrict__ qg,
                  float *__restrict__ sg, uint8_t *__restrict__ qu, float *__restrict__ su) {
    jet::griddep_launch_dependents();
    jet::griddep_wait();
    const int lane = threadIdx.x & 31, half = lane >> 4, j = lane & 15;
    const int64_t nfb = F / 128, npairs = (nfb + 1) / 2;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    // item t = (pair p, row m), t = p M + m, walked without a division
    const int64_t t0 = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t dp = warps / M, dm = warps % M;
    int64_t p = t0 / M, m = t0 % M;
    auto load = [&](int64_t p_, int64_t m_, uint4 (&v)[3]) {
        const int64_t fb = 2 * p_ + half;
        if (p_ < npairs && fb < nfb) {
            const int64_t col = fb * 128 + 8 * j;
            v[0] = ld_stream16(gate + m_ * ld + col);
            v[1] = ld_stream16(up + m_ * ld + col);
            v[2] = ld_stream16(dh + m_ * F + col);
        }
    };
    uint4 cur[3] = {};
    load(p, m, cur);
    while (p < npairs) {
        const int64_t fb = 2 * p + half;
        int64_t p2 = p + dp, m2 = m + dm;
        if (m2 >= M) {
            m2 -= M;
            ++p2;
        }
        uint4 nxt[3] = {};
        load(p2, m2, nxt);
        const uint32_t g[4] = {cur[0].x, cur[0].y, cur[0].z, cur[0].w},
                       u[4] = {cur[1].x, cur[1].y, cur[1].z, cur[1].w},
                       d[4] = {cur[2].x, cur[2].y, cur[2].z, cur[2].w};
        float ng[8], nu[8], ag = 0.0f, au = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            neg_gradients(lo(g[i]), lo(u[i]), lo(d[i]), ng[2 * i], nu[2 * i]);
            neg_gradients(hi(g[i]), hi(u[i]), hi(d[i]), ng[2 * i + 1], nu[2 * i + 1]);
            ag = max_abs2(ag, ng[2 * i], ng[2 * i + 1]);
            au = max_abs2(au, nu[2 * i], nu[2 * i + 1]);
        }
#pragma unroll
        for (int off = 8; off >= 1; off >>= 1) {
            ag = fmaxf(ag, __shfl_xor_sync(~0u, ag, off));
            au = fmaxf(au, __shfl_xor_sync(~0u, au, off));
        }
        if (fb < nfb) {
            const int64_t at = m * F + fb * 128 + 8 * j;
            const float s0 = group_scale(ag), s1 = group_scale(au);
            const Divisor d0 = make_divisor(s0), d1 = make_divisor(s1);
            *reinterpret_cast<uint2 *>(qg + at) = make_uint2(encode4(ng, d0), encode4(ng + 4, d0));
            *reinterpret_cast<uint2 *>(qu + at) = make_uint2(encode4(nu, d1), encode4(nu + 4, d1));
            if (j == 0) {
                sg[fb * M + m] = s0;
                su[fb * M + m] = s1;
            }
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) cur[i] = nxt[i];
        p = p2;
        m = m2;
    }
}

}  // namespace

jet_status jet_swiglu_bwd_quant_1x128(const uint16_t *gate, const uint16_t *up, int64_t ld,
                                      const uint16_t *dh, int64_t M, int64_t F, uint8_t *qg,
                                      float *sg, uint8_t *qu, float *su, jet_stream_t stream) {
    JET_REQUIRE(M >= 0 && F >= 0 && ld >= F, JET_ERR_SHAPE);
    const bool empty = M == 0 || F == 0;
    JET_REQUIRE(empty || (gate && up && dh && qg && sg && qu && su), JET_ERR_NULL);
    JET_REQUIRE(F % 128 == 0 && M < (int64_t)1 << 31 && ld < (int64_t)1 << 40, JET_ERR_SHAPE);
    JET_REQUIRE(ld % 8 == 0 && jet::aligned16(gate) && jet::aligned16(up) && jet::aligned16(dh) &&
                    jet::aligned16(qg) && jet::aligned16(sg) && jet::aligned16(qu) &&
                    jet::aligned16(su),
                JET_ERR_ALIGN);
    jet::DeviceInfo dev;
    const jet_status st = jet::current_device(&dev);
    if (st != JET_OK) return st;
    if (empty) return JET_OK;
    const int64_t items = M * ((F / 128 + 1) / 2);
    const int64_t want = (items + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t cap = (int64_t)dev.num_sms * kCtasPerSm;
    return jet::launch_pdl(swiglu_bwd_kernel, dim3((unsigned)(want < cap ? want : cap)),
                           dim3(kThreads), 0, jet::as_stream(stream), gate, up, ld, dh, M, F, qg,
                           sg, qu, su);
}
