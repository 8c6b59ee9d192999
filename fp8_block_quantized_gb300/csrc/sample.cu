// Sampling of one token per row of logits with temperature, top-k, top-p and
// min-p from given uniform numbers, with the drawn token's log-probabilities
// (jet_sample).
//
// Definition (per row; NaN logits are never drawn):
//   m = max x,  z_i = fl32(fl32(x_i - m) fl32(1/T)),  w_i = fl32(e^{z_i}),
//   kept: in the order of falling logit, ties by rising index, the tokens with
//     rank < k, then of those the ones with mass before them < p times the
//     mass of the first k, then those with w_i >= min_p (the largest w is 1):
//     every filter keeps a prefix of that order;
//   drawn: the first kept token, in index order, at which the running sum of
//     the kept weights exceeds u times their sum.
// The sums run over the 64-bit integers W_i = round(w_i 2^45): exact, so no
// order of summation, number of CTAs or batch changes a token.
//
// A cluster of 1 to 8 CTAs holds one row in its shared memory, read from HBM
// once; each warp owns a contiguous range of the row, so that a running sum in
// index order needs only one total per warp.  The filters' cut (the last kept
// token) is found without a sort of the row: a histogram of counts and masses
// over 2048 steps of z finds the step it lies in, and the few tokens of that
// step are ranked against each other; a step with too many of them is split
// again on the bits of the logits, and one of equal logits by counting.
#include <cooperative_groups.h>

#include "jet_common.cuh"

namespace {

namespace cg = cooperative_groups;

constexpr int kSaThreads = 512;
constexpr int kSaWarps = kSaThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;           // steps of 1/64 of z; z <= -32 is bin kBins
constexpr float kBinsPerZ = 64.0f;
constexpr int kListCap = 512;         // tokens ranked against each other
constexpr int64_t kSaMaxV = 262144;   // so that the sum of 2^45-scaled weights fits 64 bits
constexpr float kWeightScale = 0x1p45f;

typedef unsigned long long u64;

struct SampleArgs {
    const void *x;
    int64_t ld, B;
    int V;
    const float *u, *temperature, *top_p, *min_p;
    const int *top_k;
    int64_t *token;
    float *logp, *logp_all;
    int *kept;
    int chunks_per_warp;
};

struct Entry {
    unsigned key;
    int idx;
    u64 w;
};

// What a CTA of the cluster holds besides its slice of the row.  Arrays over
// ranks are written by the peers and read after a cluster barrier.
struct Shared {
    u64 warp_mass[kSaWarps], rank_mass[kMaxCluster], seg_mass[kMaxCluster];
    unsigned warp_cnt[kSaWarps], rank_cnt[kMaxCluster], seg_cnt[kMaxCluster];
    float warp_max[kSaWarps], rank_max[kMaxCluster];
    unsigned warp_lo[kSaWarps], warp_hi[kSaWarps], rank_lo[kMaxCluster], rank_hi[kMaxCluster];
    u64 scan_mass[kSaWarps];
    unsigned scan_cnt[kSaWarps];
    // the selected bin
    int sel_bin;
    unsigned sel_before, sel_cnt;
    u64 sel_mass;
    unsigned list_n;
    u64 best;
    // the cut: the last kept token
    unsigned cut_key;
    int cut_idx;
    u64 cut_mass;
};

struct FilterShared {
    u64 mass[kBins];
    unsigned cnt[kBins];
    Entry list[kListCap];
};

__device__ __forceinline__ unsigned key_of(float x) {  // orders as the logit does
    const unsigned b = __float_as_uint(x);
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

// A logit as the kernel holds it: NaN never drawn, one zero.
__device__ __forceinline__ float clean(float x) { return x == x ? x + 0.0f : -INFINITY; }

template <bool kBf16>
struct Elems;

template <>
struct Elems<false> {
    static constexpr int E = 4;
    typedef float T;
    static __device__ __forceinline__ void load(const uint4 &c, float (&f)[4]) {
        f[0] = __uint_as_float(c.x);
        f[1] = __uint_as_float(c.y);
        f[2] = __uint_as_float(c.z);
        f[3] = __uint_as_float(c.w);
    }
    static __device__ __forceinline__ uint4 store(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
    static __device__ __forceinline__ float one(const T *p) { return *p; }
};

template <>
struct Elems<true> {
    static constexpr int E = 8;
    typedef uint16_t T;
    static __device__ __forceinline__ void load(const uint4 &c, float (&f)[8]) {
        const unsigned w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 store(const float (&f)[8]) {
        unsigned w[4];  // the values are BF16: their low halves are zero
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = (__float_as_uint(f[2 * i]) >> 16) | (__float_as_uint(f[2 * i + 1]) & 0xFFFF0000u);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ float one(const T *p) {
        return __uint_as_float((unsigned)*p << 16);
    }
};

// z of a logit x <= m; -inf and undefined products give -inf.
__device__ __forceinline__ float z_of(float x, float m, float rt) {
    const float z = x == m ? 0.0f : __fmul_rn(__fadd_rn(x, -m), rt);
    return z <= 0.0f && x > -INFINITY ? z : -INFINITY;
}

__device__ __forceinline__ u64 mass_of(float w) { return __float2ull_rn(w * kWeightScale); }

__device__ __forceinline__ int bin_of(float z) {
    return z > -32.0f ? (int)(z * -kBinsPerZ) : kBins;
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <bool kBf16, bool kFilter>
struct Sampler {
    typedef Elems<kBf16> El;
    static constexpr int E = El::E;

    const SampleArgs &a;
    cg::cluster_group cl;
    Shared *sh;
    FilterShared *fs;
    uint4 *row;
    int C, rank, lane, warp;
    int c0, c1;  // this warp's chunks of the row
    int shift;   // elements before the row in its first chunk
    float m, rt, min_w;
    unsigned cut_key;
    int cut_idx;

    __device__ Sampler(const SampleArgs &args) : a(args), cl(cg::this_cluster()) {}

    // f(x, index) for every element of this warp's range.
    template <typename F>
    __device__ __forceinline__ void each(F f) {
        for (int c = c0 + lane; c < c1; c += 32) {
            float v[E];
            El::load(row[c - c0 + warp * a.chunks_per_warp], v);
#pragma unroll
            for (int e = 0; e < E; ++e) f(v[e], c * E + e - shift);
        }
    }

    // v of every rank into arr[rank] of every CTA, by thread 0 .. C-1.
    template <typename V>
    __device__ __forceinline__ void to_all(V *slot, V v) {
        if ((int)threadIdx.x < C) *cl.map_shared_rank(slot, threadIdx.x) = v;
    }

    __device__ __forceinline__ bool kept(float x, float w, int idx) const {
        if (x == -INFINITY) return false;
        if (!kFilter) return true;
        const unsigned k = key_of(x);
        return (k > cut_key || (k == cut_key && idx <= cut_idx)) && w >= min_w;
    }

    // Warp, CTA and cluster totals of a mass and a count; ends with a cluster
    // barrier, after which rank_mass / rank_cnt hold every CTA's totals.
    __device__ void totals(u64 mass, unsigned cnt) {
        mass = warp_sum(mass);
        cnt = __reduce_add_sync(0xffffffffu, cnt);
        if (lane == 0) {
            sh->warp_mass[warp] = mass;
            sh->warp_cnt[warp] = cnt;
        }
        __syncthreads();
        if ((int)threadIdx.x < C) {
            u64 t = 0;
            unsigned n = 0;
            for (int i = 0; i < kSaWarps; ++i) {
                t += sh->warp_mass[i];
                n += sh->warp_cnt[i];
            }
            to_all(&sh->rank_mass[rank], t);
            to_all(&sh->rank_cnt[rank], n);
        }
        cl.sync();
    }

    __device__ u64 all_mass() const {
        u64 t = 0;
        for (int r = 0; r < C; ++r) t += sh->rank_mass[r];
        return t;
    }
    __device__ unsigned all_cnt() const {
        unsigned t = 0;
        for (int r = 0; r < C; ++r) t += sh->rank_cnt[r];
        return t;
    }

    // Histogram of this CTA's elements of an interval of keys (level > 0), or
    // of all by the step of z (level 0).
    __device__ void histogram(int level, unsigned lo, unsigned hi, int sft) {
        for (int i = threadIdx.x; i < kBins; i += kSaThreads) {
            fs->mass[i] = 0;
            fs->cnt[i] = 0;
        }
        __syncthreads();
        each([&](float x, int) {
            if (x == -INFINITY) return;
            const float z = z_of(x, m, rt);
            int b;
            if (level == 0) {
                b = bin_of(z);
            } else {
                const unsigned k = key_of(x);
                b = k >= lo && k <= hi ? (int)((hi - k) >> sft) : kBins;
            }
            if (b < kBins) {
                atomicAdd(&fs->cnt[b], 1u);
                const u64 w = mass_of(expf(z));
                if (w) atomicAdd(&fs->mass[b], w);
            }
        });
        cl.sync();
    }

    // The first bin whose end reaches the target (a count or a mass), given
    // what lies before the histogram; its place goes to every CTA.
    __device__ void select(bool by_mass, unsigned target_cnt, double target_mass, unsigned base_cnt,
                           u64 base_mass) {
        const int seg = kBins / C;                         // bins this CTA merges
        const int per = seg > kSaThreads ? seg / kSaThreads : 1;
        u64 bm[kBins / kSaThreads];
        unsigned bc[kBins / kSaThreads];
        u64 tm = 0;
        unsigned tc = 0;
        const int first = rank * seg + (int)threadIdx.x * per;
        const bool active = (int)threadIdx.x * per < seg;
#pragma unroll
        for (int j = 0; j < kBins / kSaThreads; ++j) {
            bm[j] = 0;
            bc[j] = 0;
            if (active && j < per) {
                for (int r = 0; r < C; ++r) {
                    const FilterShared *o = cl.map_shared_rank(fs, r);
                    bm[j] += o->mass[first + j];
                    bc[j] += o->cnt[first + j];
                }
                tm += bm[j];
                tc += bc[j];
            }
        }
        u64 im = tm;  // inclusive over the CTA's threads
        unsigned ic = tc;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 q = __shfl_up_sync(0xffffffffu, im, o);
            const unsigned n = __shfl_up_sync(0xffffffffu, ic, o);
            if (lane >= o) {
                im += q;
                ic += n;
            }
        }
        if (lane == 31) {
            sh->scan_mass[warp] = im;
            sh->scan_cnt[warp] = ic;
        }
        if (threadIdx.x == 0) {
            sh->sel_bin = kBins;
            sh->list_n = 0;
            sh->best = 0;
        }
        __syncthreads();
        u64 sm = 0;
        unsigned sc = 0;
        for (int w = 0; w < kSaWarps; ++w) {
            if (w < warp) {
                im += sh->scan_mass[w];
                ic += sh->scan_cnt[w];
            }
            sm += sh->scan_mass[w];
            sc += sh->scan_cnt[w];
        }
        to_all(&sh->seg_mass[rank], sm);
        to_all(&sh->seg_cnt[rank], sc);
        cl.sync();
        u64 pm = base_mass + im - tm;
        unsigned pc = base_cnt + ic - tc;
        for (int r = 0; r < rank; ++r) {
            pm += sh->seg_mass[r];
            pc += sh->seg_cnt[r];
        }
#pragma unroll
        for (int j = 0; j < kBins / kSaThreads; ++j) {
            if (active && j < per) {
                const u64 em = pm + bm[j];
                const unsigned ec = pc + bc[j];
                const bool before = by_mass ? (double)pm < target_mass : pc < target_cnt;
                const bool after = by_mass ? (double)em < target_mass : ec < target_cnt;
                if (before && !after) {
                    for (int r = 0; r < C; ++r) {
                        Shared *o = cl.map_shared_rank(sh, r);
                        o->sel_bin = first + j;
                        o->sel_before = pc;
                        o->sel_mass = pm;
                        o->sel_cnt = bc[j];
                    }
                }
                pm = em;
                pc = ec;
            }
        }
        cl.sync();
    }

    // The cut among tokens of one logit: the first `n` of them in index order.
    __device__ void cut_ties(unsigned key, unsigned n, u64 mass) {
        unsigned mine = 0;
        each([&](float x, int) { mine += x > -INFINITY && key_of(x) == key; });
        totals(0, mine);
        unsigned before = 0;
        for (int r = 0; r < rank; ++r) before += sh->rank_cnt[r];
        for (int w = 0; w < warp; ++w) before += sh->warp_cnt[w];
        const unsigned own = sh->warp_cnt[warp];
        if (before < n && n <= before + own) {  // one warp of the cluster
            for (int base = c0; base < c1; base += 32) {
                const int c = base + lane;
                float v[E];
                unsigned t = 0;
                if (c < c1) {
                    El::load(row[c - c0 + warp * a.chunks_per_warp], v);
#pragma unroll
                    for (int e = 0; e < E; ++e) t += v[e] > -INFINITY && key_of(v[e]) == key;
                }
                unsigned inc = t;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned q = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += q;
                }
                if (before + inc - t < n && n <= before + inc) {
                    unsigned at = before + inc - t;
                    int idx = 0;
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (v[e] > -INFINITY && key_of(v[e]) == key && ++at == n)
                            idx = c * E + e - shift;
                    for (int r = 0; r < C; ++r) {
                        Shared *o = cl.map_shared_rank(sh, r);
                        o->cut_key = key;
                        o->cut_idx = idx;
                        o->cut_mass = mass;
                    }
                }
                before += __shfl_sync(0xffffffffu, inc, 31);
            }
        }
        cl.sync();
        cut_key = sh->cut_key;
        cut_idx = sh->cut_idx;
    }

    // The cut of a filter: the last token whose rank is below target_cnt, or
    // the mass before which is below target_mass.  The caller has checked that
    // the target lies inside the row.  Returns the kept mass.
    __device__ u64 cut(bool by_mass, unsigned target_cnt, double target_mass) {
        unsigned lo = 0, hi = 0xFFFFFFFFu, base_cnt = 0;
        u64 base_mass = 0;
        int sft = 0;
        for (int level = 0;; ++level) {
            histogram(level, lo, hi, sft);
            select(by_mass, target_cnt, target_mass, base_cnt, base_mass);
            const int bin = sh->sel_bin;
            unsigned n = sh->sel_cnt;
            if (bin < kBins) {
                base_cnt = sh->sel_before;
                base_mass = sh->sel_mass;
            } else {  // level 0 only: past the steps, among weights that round to zero
                for (int r = 0; r < C; ++r) {
                    base_cnt += sh->seg_cnt[r];
                    base_mass += sh->seg_mass[r];
                }
                n = 0xFFFFFFFFu;
            }
            auto in_bin = [&](float x) {
                if (x == -INFINITY) return false;
                if (level == 0) return bin_of(z_of(x, m, rt)) == bin;
                const unsigned k = key_of(x);
                return k >= lo && k <= hi && (int)((hi - k) >> sft) == bin;
            };
            if (n <= kListCap) {
                Shared *s0 = cl.map_shared_rank(sh, 0);
                FilterShared *f0 = cl.map_shared_rank(fs, 0);
                each([&](float x, int idx) {
                    if (in_bin(x)) {
                        const unsigned at = atomicAdd(&s0->list_n, 1u);
                        if (at < kListCap)
                            f0->list[at] = {key_of(x), idx, mass_of(expf(z_of(x, m, rt)))};
                    }
                });
                cl.sync();
                if (rank == 0) {
                    for (unsigned i = threadIdx.x; i < n; i += kSaThreads) {
                        const Entry me = fs->list[i];
                        unsigned ahead = 0;
                        u64 before = 0;
                        for (unsigned j = 0; j < n; ++j) {
                            const Entry o = fs->list[j];
                            if (o.key > me.key || (o.key == me.key && o.idx < me.idx)) {
                                ++ahead;
                                before += o.w;
                            }
                        }
                        const bool in = by_mass ? (double)(base_mass + before) < target_mass
                                                : base_cnt + ahead < target_cnt;
                        if (in) atomicMax(&sh->best, ((u64)(ahead + 1) << 32) | i);
                    }
                    __syncthreads();
                    const Entry last = fs->list[(unsigned)sh->best];
                    u64 part = 0;  // mass of the list up to and including the last
                    for (unsigned i = threadIdx.x; i < n; i += kSaThreads) {
                        const Entry o = fs->list[i];
                        if (o.key > last.key || (o.key == last.key && o.idx <= last.idx)) part += o.w;
                    }
                    part = warp_sum(part);
                    if (lane == 0) sh->scan_mass[warp] = part;
                    __syncthreads();
                    u64 total = base_mass;
                    for (int w = 0; w < kSaWarps; ++w) total += sh->scan_mass[w];
                    to_all(&sh->cut_key, last.key);
                    to_all(&sh->cut_idx, last.idx);
                    to_all(&sh->cut_mass, total);
                }
                cl.sync();
                cut_key = sh->cut_key;
                cut_idx = sh->cut_idx;
                return sh->cut_mass;
            }
            // too many to rank: the bin's own interval of keys
            unsigned klo = 0xFFFFFFFFu, khi = 0;
            each([&](float x, int) {
                if (in_bin(x)) {
                    klo = min(klo, key_of(x));
                    khi = max(khi, key_of(x));
                }
            });
            klo = __reduce_min_sync(0xffffffffu, klo);
            khi = __reduce_max_sync(0xffffffffu, khi);
            if (lane == 0) {
                sh->warp_lo[warp] = klo;
                sh->warp_hi[warp] = khi;
            }
            __syncthreads();
            if ((int)threadIdx.x < C) {
                for (int w = 0; w < kSaWarps; ++w) {
                    klo = min(klo, sh->warp_lo[w]);
                    khi = max(khi, sh->warp_hi[w]);
                }
                to_all(&sh->rank_lo[rank], klo);
                to_all(&sh->rank_hi[rank], khi);
            }
            cl.sync();
            lo = 0xFFFFFFFFu;
            hi = 0;
            for (int r = 0; r < C; ++r) {
                lo = min(lo, sh->rank_lo[r]);
                hi = max(hi, sh->rank_hi[r]);
            }
            if (lo == hi) {  // one logit: the first so many in index order
                const float x = __uint_as_float(lo ^ ((lo >> 31) ? 0x80000000u : 0xFFFFFFFFu));
                const u64 w = mass_of(expf(z_of(x, m, rt)));
                unsigned q;
                if (!by_mass) {
                    q = target_cnt - base_cnt;
                } else {  // token i of them is kept when base + i w < target
                    const double at = w ? (target_mass - (double)base_mass) / (double)w : 1.0;
                    q = at < 1.0 ? 1u : (unsigned)at;
                    while (q > 1 && (double)(base_mass + (q - 1) * w) >= target_mass) --q;
                    while (w && q < n && (double)(base_mass + q * w) < target_mass) ++q;
                }
                const u64 mass = base_mass + q * w;
                cut_ties(lo, q, mass);
                return mass;
            }
            const unsigned range = hi - lo;
            sft = max(0, 32 - __clz((int)range) - 11);  // range >> sft < 2048
        }
    }

    __device__ void run(int64_t b) {
        const int V = a.V;
        const typename El::T *x = static_cast<const typename El::T *>(a.x) + b * a.ld;
        shift = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(typename El::T));
        const int chunks = (shift + V + E - 1) / E;
        c0 = min((rank * kSaWarps + warp) * a.chunks_per_warp, chunks);
        c1 = min(c0 + a.chunks_per_warp, chunks);
        // the row into shared memory, and its maximum
        const uint4 *src = reinterpret_cast<const uint4 *>(x - shift);
        float mx = -INFINITY;
        constexpr int kLoads = 4;
        for (int base = c0; base < c1; base += 32 * kLoads) {
            uint4 t[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int c = base + 32 * i + lane;
                if (c < c1 && c * E >= shift && (c + 1) * E - shift <= V) t[i] = src[c];
            }
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int c = base + 32 * i + lane;
                if (c >= c1) break;
                float v[E];
                if (c * E >= shift && (c + 1) * E - shift <= V) {
                    El::load(t[i], v);
                } else {  // the row's ragged ends
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int idx = c * E + e - shift;
                        v[e] = idx >= 0 && idx < V ? El::one(x + idx) : -INFINITY;
                    }
                }
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    v[e] = clean(v[e]);
                    mx = fmaxf(mx, v[e]);
                }
                row[c - c0 + warp * a.chunks_per_warp] = El::store(v);
            }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (lane == 0) sh->warp_max[warp] = mx;
        __syncthreads();
        if ((int)threadIdx.x < C) {
            for (int w = 0; w < kSaWarps; ++w) mx = fmaxf(mx, sh->warp_max[w]);
            to_all(&sh->rank_max[rank], mx);
        }
        cl.sync();
        m = -INFINITY;
        for (int r = 0; r < C; ++r) m = fmaxf(m, sh->rank_max[r]);
        if (m == -INFINITY) {  // nothing can be drawn
            if (rank == 0 && threadIdx.x == 0) {
                a.token[b] = -1;
                a.logp[b] = __int_as_float(0x7FC00000);
                a.logp_all[b] = __int_as_float(0x7FC00000);
                a.kept[b] = 0;
            }
            return;
        }
        const float T = a.temperature ? a.temperature[b] : 1.0f;
        const bool greedy = !(T > 0.0f);
        rt = __fdiv_rn(1.0f, greedy ? 1.0f : T);
        u64 mass = 0;
        unsigned cnt = 0;
        each([&](float xv, int) {
            mass += mass_of(expf(z_of(xv, m, rt)));
            cnt += xv > -INFINITY;
        });
        totals(mass, cnt);
        const u64 S_all = all_mass();
        u64 S = S_all;
        unsigned n_kept = all_cnt();
        min_w = 0.0f;
        cut_key = 0;
        cut_idx = 0x7FFFFFFF;
        if (kFilter) {
            const int k = greedy ? 1 : a.top_k && a.top_k[b] > 0 ? a.top_k[b] : 0x7FFFFFFF;
            const float p = a.top_p ? a.top_p[b] : 1.0f;
            const float mp = a.min_p ? a.min_p[b] : 0.0f;
            min_w = mp > 0.0f ? fminf(mp, 1.0f) : 0.0f;
            const unsigned finite = n_kept;
            bool cut_any = min_w > 0.0f;
            if (k == 1) {
                cut_ties(key_of(m), 1, mass_of(1.0f));
                cut_any = true;
            } else {
                u64 S_k = S_all;
                if ((unsigned)k < finite) {
                    S_k = cut(false, (unsigned)k, 0.0);
                    cut_any = true;
                }
                if (p < 1.0f) {
                    const double target = (double)fmaxf(p, 0.0f) * (double)S_k;
                    if (target > 0.0) cut(true, 0, target);
                    else cut_ties(key_of(m), 1, mass_of(1.0f));
                    cut_any = true;
                }
            }
            if (cut_any) {
                mass = 0;
                cnt = 0;
                each([&](float xv, int idx) {
                    const float w = expf(z_of(xv, m, rt));
                    if (kept(xv, w, idx)) {
                        mass += mass_of(w);
                        ++cnt;
                    }
                });
                totals(mass, cnt);
                S = all_mass();
                n_kept = all_cnt();
            }
        }
        // the draw: the CTA, the warp, then the lane and element at which the
        // running sum exceeds u S
        float u = a.u[b];
        u = u >= 0.0f ? fminf(u, 0x1.fffffep-1f) : 0.0f;
        const double target = (double)u * (double)S;
        u64 before = 0;
        for (int r = 0; r < rank; ++r) before += sh->rank_mass[r];
        for (int w = 0; w < warp; ++w) before += sh->warp_mass[w];
        if ((double)before > target || !((double)(before + sh->warp_mass[warp]) > target)) return;
        for (int base = c0; base < c1; base += 32) {
            const int c = base + lane;
            u64 w[E], t = 0;
            if (c < c1) {
                float v[E];
                El::load(row[c - c0 + warp * a.chunks_per_warp], v);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float wf = expf(z_of(v[e], m, rt));
                    w[e] = kept(v[e], wf, c * E + e - shift) ? mass_of(wf) : 0;
                    t += w[e];
                }
            }
            u64 inc = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 q = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += q;
            }
            u64 at = before + inc - t;
            if (!((double)at > target) && (double)(at + t) > target) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (!((double)at > target) && (double)(at + w[e]) > target) {
                        a.token[b] = c * E + e - shift;
                        a.logp[b] = log_share(w[e], S);
                        a.logp_all[b] = log_share(w[e], S_all);
                        a.kept[b] = (int)n_kept;
                    }
                    at += w[e];
                }
            }
            before += __shfl_sync(0xffffffffu, inc, 31);
            if ((double)before > target) break;
        }
    }

    // log(w / s), through log1p where the share is near one.
    static __device__ __forceinline__ float log_share(u64 w, u64 s) {
        const float sf = __ull2float_rn(s);
        return 2 * w > s ? log1pf(-__fdiv_rn(__ull2float_rn(s - w), sf))
                         : logf(__fdiv_rn(__ull2float_rn(w), sf));
    }
};

template <bool kBf16, bool kFilter>
__global__ void __launch_bounds__(kSaThreads) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    jet::griddep_launch_dependents();
    jet::griddep_wait();
    Sampler<kBf16, kFilter> s(a);
    s.C = (int)s.cl.num_blocks();
    s.rank = (int)s.cl.block_rank();
    s.lane = threadIdx.x & 31;
    s.warp = threadIdx.x >> 5;
    s.sh = reinterpret_cast<Shared *>(smem);
    s.fs = reinterpret_cast<FilterShared *>(smem + (sizeof(Shared) + 15) / 16 * 16);
    s.row = reinterpret_cast<uint4 *>(smem + (sizeof(Shared) + 15) / 16 * 16 +
                                      (kFilter ? sizeof(FilterShared) : 0));
    s.run(blockIdx.x / s.C);
}

template <int kBytes>
bool aligned_to(const void *p) { return (reinterpret_cast<uintptr_t>(p) & (kBytes - 1)) == 0; }

}  // namespace

jet_status jet_sample(const void *logits, int dtype, int64_t B, int64_t V, int64_t ld,
                      const float *u, const float *temperature, const int32_t *top_k,
                      const float *top_p, const float *min_p, int64_t *token, float *logp,
                      float *logp_all, int32_t *kept, jet_stream_t stream) {
    JET_REQUIRE(B >= 0 && V >= 0, JET_ERR_SHAPE);
    JET_REQUIRE(B == 0 || (logits && u && token && logp && logp_all && kept), JET_ERR_NULL);
    JET_REQUIRE((B == 0 || V >= 1) && V <= kSaMaxV && B < ((int64_t)1 << 28) && ld >= V &&
                    ld < ((int64_t)1 << 40) && (dtype == JET_BF16 || dtype == JET_FP32),
                JET_ERR_SHAPE);
    JET_REQUIRE(jet::aligned16(logits) && aligned_to<4>(u) && aligned_to<4>(temperature) &&
                    aligned_to<4>(top_k) && aligned_to<4>(top_p) && aligned_to<4>(min_p) &&
                    aligned_to<8>(token) && aligned_to<4>(logp) && aligned_to<4>(logp_all) &&
                    aligned_to<4>(kept),
                JET_ERR_ALIGN);
    jet::DeviceInfo dev;
    jet_status st = jet::current_device(&dev);
    if (st != JET_OK) return st;
    if (B == 0) return JET_OK;
    const bool bf16 = dtype == JET_BF16;
    const bool filter = temperature || top_k || top_p || min_p;
    const int E = bf16 ? 8 : 4;
    const int64_t chunks = (V + E - 1 + E - 1) / E;  // a row may start inside a chunk
    // CTAs per row: all eight while the rows alone cannot fill the SMs, else
    // the fewest that keep a slice within 72 KB; a slice has 512 chunks at least.
    int C = B * kMaxCluster <= 2 * (int64_t)dev.num_sms ? kMaxCluster : 1;
    while (C < kMaxCluster && chunks * 16 > (int64_t)C * 72 * 1024) C *= 2;
    while (C > 1 && chunks < (int64_t)C * kSaThreads) C /= 2;
    SampleArgs a = {};
    a.x = logits;
    a.ld = ld;
    a.B = B;
    a.V = (int)V;
    a.u = u;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.token = token;
    a.logp = logp;
    a.logp_all = logp_all;
    a.kept = kept;
    const int64_t parts = (int64_t)C * kSaWarps;
    a.chunks_per_warp = (int)(((chunks + parts - 1) / parts + 31) / 32 * 32);
    const size_t smem = (sizeof(Shared) + 15) / 16 * 16 + (filter ? sizeof(FilterShared) : 0) +
                        (size_t)kSaWarps * a.chunks_per_warp * 16;
    void (*kernel)(SampleArgs) = bf16 ? (filter ? sample_kernel<true, true> : sample_kernel<true, false>)
                                      : (filter ? sample_kernel<false, true> : sample_kernel<false, false>);
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
        cudaSuccess) {
        cudaGetLastError();
        return JET_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * C));
    cfg.blockDim = dim3(kSaThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = jet::as_stream(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return JET_ERR_CUDA;
    }
    return jet::launch_status();
}
