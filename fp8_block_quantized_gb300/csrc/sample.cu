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
// once (cp.async); each warp owns a contiguous range of the row, so that a
// running sum in index order needs only one total per warp.  Without a filter
// two passes over shared memory (maximum, weights) and two cluster barriers
// lead to the draw.
//
// The filters' cut (the last kept token) is found without a sort of the row.
// A bound z_lo is taken below which it cannot lie (top-k: a group of z up to
// which k of the threads' own maxima lie; top-p: all tokens below w = (1 - p)
// S / V together weigh less than (1 - p) S; min-p: its own weight).  When at
// most kListMax tokens lie above it, they go to the first CTA, which sorts
// them in registers, finds the cut and draws, while the others end.  Flat
// distributions and large k take the general way: a histogram of counts and
// masses over 2048 steps of z finds the step the cut lies in, and the few
// tokens of that step are ranked against each other; a step with too many of
// them is split again on the bits of the logits, and one of equal logits by
// counting.
#include <cooperative_groups.h>

#include "jet_common.cuh"

namespace {

namespace cg = cooperative_groups;

constexpr int kMaxCluster = 8;
constexpr int kMaxWarps = 16;
constexpr int kBins = 2048;           // steps of 1/64 of z; z <= -32 is bin kBins
constexpr float kBinsPerZ = 64.0f;
constexpr int kGroups = 128;          // groups of 16 steps: 1/4 of z
constexpr float kGroupsPerZ = 4.0f;
constexpr int kListMax = 4096;        // tokens sorted by the first CTA
constexpr int64_t kSaMaxV = 262144;   // so that the sum of 2^45-scaled weights fits 64 bits

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

// What a CTA of the cluster holds besides its slice of the row.  Arrays over
// ranks are written by the peers and read after a cluster barrier.
struct Shared {
    u64 warp_mass[kMaxWarps], rank_mass[kMaxCluster], seg_mass[kMaxCluster];
    u64 scan[2][kMaxWarps], sel_mass, cut_entry;
    unsigned warp_cnt[kMaxWarps], rank_cnt[kMaxCluster];
    float warp_max[kMaxWarps], rank_max[kMaxCluster];
    unsigned warp_lo[kMaxWarps], warp_hi[kMaxWarps], rank_lo[kMaxCluster], rank_hi[kMaxCluster];
    int sel_bin;  // the selected bin
    int cut_idx;
};

// The general way's histogram, or the list the first CTA sorts.
struct FilterShared {
    union {
        // counts, or masses in three 15-bit parts: shared-memory atomics on 32
        // bits run in hardware, and 2^17 tokens of one CTA cannot overflow a part
        unsigned hist[3][kBins];
        u64 sorted[kListMax];  // ~key, index
    };
    unsigned grp[kMaxCluster][kGroups];  // threads' maxima by group of z
};

__device__ __forceinline__ unsigned key_of(float x) {  // orders as the logit does, zeros alike
    const unsigned b = __float_as_uint(x + 0.0f);
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ float logit_of(unsigned key) {
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// A logit as the kernel uses it: NaN is never drawn.
__device__ __forceinline__ float clean(float x) { return fmaxf(x, -INFINITY); }

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

__device__ __forceinline__ u64 mass_of(float w) { return __float2ull_rn(w * 0x1p45f); }

// floor(f s) and ceil(f s) for 0 <= f < 1, exact: f = mant 2^-sh.
__device__ __forceinline__ u64 share(float f, u64 s, bool up) {
    const unsigned bits = __float_as_uint(f), e = bits >> 23;
    const u64 mant = e ? (bits & 0x7FFFFFu) | 0x800000u : bits;
    const int sh = 150 - (e ? (int)e : 1);  // 24 .. 149
    const u64 lo = mant * s, hi = __umul64hi(mant, s);
    u64 q, rest;
    if (sh < 64) {
        q = (hi << (64 - sh)) | (lo >> sh);
        rest = lo << (64 - sh);
    } else if (sh < 128) {
        q = sh == 64 ? hi : hi >> (sh - 64);
        rest = lo | (sh == 64 ? 0 : hi << (128 - sh));
    } else {
        q = 0;
        rest = lo | hi;
    }
    return q + (up && rest != 0);
}

// Sums of round(w 2^45) of one thread, in two 32-bit halves (weights of 1 at
// most, 512 of them at most): adding 2^23 to w 2^22 leaves its integer part
// `hi` in the low bits; what is left, times 2^23, is rounded the same way.
// Exact, and without the 64-bit conversion, whose rate is a quarter of the
// multiply-adds'.
struct MassSum {
    unsigned hi = 0, lo = 0;
    __device__ __forceinline__ void add2(float w0, float w1) {
        const float2 w = make_float2(w0, w1), up = make_float2(0x1p22f, 0x1p22f);
        const float2 big = make_float2(0x1p23f, 0x1p23f);
        const float2 t = __ffma2_rn(w, up, big);
        const float2 whole = __fadd2_rn(t, make_float2(-0x1p23f, -0x1p23f));
        const float2 r = __ffma2_rn(w, up, make_float2(-whole.x, -whole.y));
        const float2 l = __ffma2_rn(r, big, make_float2(0x1.8p23f, 0x1.8p23f));
        hi += __float_as_uint(t.x) + __float_as_uint(t.y);
        lo += __float_as_uint(l.x) + __float_as_uint(l.y);
    }
    // n: how many weights were added
    __device__ __forceinline__ u64 total(unsigned n) const {
        return ((u64)(hi - n * 0x4B000000u) << 23) + (u64)(int64_t)(int)(lo - n * 0x4B400000u);
    }
};

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     (unsigned)__cvta_generic_to_shared(dst)),
                 "l"(src)
                 : "memory");
}

template <int kPending>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// A z below which every token weighs less than w (-inf when past the steps).
__device__ __forceinline__ float z_below(float w) {
    const float z = w > 0.0f ? fminf(logf(w) - 1e-3f, 0.0f) : -INFINITY;
    return z > -32.0f ? z : -INFINITY;
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 q = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += q;
    }
    return v;
}

template <bool kBf16, bool kFilter, int kThreads>
struct Sampler {
    typedef Elems<kBf16> El;
    static constexpr int E = El::E;
    static constexpr int kWarps = kThreads / 32;

    const SampleArgs &a;
    cg::cluster_group cl;
    Shared *sh;
    FilterShared *fs;
    uint4 *row;   // this warp's chunk c0 is row[0]
    int C, rank, lane, warp;
    int c0, c1;   // this warp's chunks of the row
    int shift;    // elements before the row in its first chunk
    float m, rt, min_w;
    bool regular;  // m and 1/T finite: z needs no care
    float cut_x;
    int cut_idx;

    __device__ Sampler(const SampleArgs &args) : a(args), cl(cg::this_cluster()) {}

    __device__ __forceinline__ float z(float x) const {
        return regular ? __fmul_rn(__fadd_rn(x, -m), rt) : z_of(x, m, rt);
    }

    // f(x, index) for every element of this warp's range.
    template <typename F>
    __device__ __forceinline__ void each(F f) {
#pragma unroll 1
        for (int c = c0 + lane; c < c1; c += 32) {
            float v[E];
            El::load(row[c - c0], v);
#pragma unroll
            for (int e = 0; e < E; ++e) f(clean(v[e]), c * E + e - shift);
        }
    }

    // v of every rank into arr[rank] of every CTA, by thread 0 .. C-1.
    template <typename V>
    __device__ __forceinline__ void to_all(V *slot, V v) {
        if ((int)threadIdx.x < C) *cl.map_shared_rank(slot, threadIdx.x) = v;
    }

    __device__ __forceinline__ bool kept(float x, float w, int idx) const {
        if (!kFilter) return true;  // weight 0 where it could matter
        return (x > cut_x || (x == cut_x && idx <= cut_idx)) && w >= min_w && x > -INFINITY;
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
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
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

    // The row into shared memory by this thread's own copies, four groups of
    // them in flight; the maximum of what this thread copied and how many of
    // them are logits that can be drawn.
    __device__ float load_row(const typename El::T *x, unsigned &finite) {
        const int V = a.V;
        const uint4 *src = reinterpret_cast<const uint4 *>(x - shift);
        uint4 *dst = row - c0;
        const int quarter = (a.chunks_per_warp / 32 + 3) / 4 * 32;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            for (int c = c0 + i * quarter + lane; c < min(c0 + (i + 1) * quarter, c1); c += 32) {
                if (c * E >= shift && (c + 1) * E - shift <= V) {
                    cp_async16(dst + c, src + c);
                } else {  // the row's ragged ends
                    float v[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int idx = c * E + e - shift;
                        v[e] = idx >= 0 && idx < V ? El::one(x + idx) : -INFINITY;
                    }
                    dst[c] = El::store(v);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        float mx = -INFINITY;
        unsigned n = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i == 0) cp_wait<3>();
            if (i == 1) cp_wait<2>();
            if (i == 2) cp_wait<1>();
            if (i == 3) cp_wait<0>();
            for (int c = c0 + i * quarter + lane; c < min(c0 + (i + 1) * quarter, c1); c += 32) {
                float v[E];
                El::load(dst[c], v);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    mx = fmaxf(mx, v[e]);  // a NaN leaves it as it is
                    n += v[e] > -INFINITY;
                }
            }
        }
        finite = n;
        return mx;
    }

    // This thread's weights.  Where m and 1/T are finite, x = -inf gives z =
    // -inf and weight 0 by itself.
    __device__ __forceinline__ u64 weigh() {
        MassSum s;
        unsigned n = 0;
        const float2 nm = make_float2(-m, -m), r2 = make_float2(rt, rt);
        if (regular) {
            for (int c = c0 + lane; c < c1; c += 32) {
                float v[E];
                El::load(row[c - c0], v);
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float2 zz = __fmul2_rn(__fadd2_rn(make_float2(clean(v[e]), clean(v[e + 1])), nm), r2);
                    s.add2(expf(zz.x), expf(zz.y));
                }
                n += E;
            }
        } else {
#pragma unroll 1
            for (int c = c0 + lane; c < c1; c += 32) {
                float v[E];
                El::load(row[c - c0], v);
#pragma unroll
                for (int e = 0; e < E; e += 2)
                    s.add2(expf(z_of(clean(v[e]), m, rt)), expf(z_of(clean(v[e + 1]), m, rt)));
                n += E;
            }
        }
        return s.total(n);
    }

    // Exclusive sum of v over the CTA's threads, the total, and the total of o.
    __device__ u64 block_scan(u64 v, u64 &total, u64 o, u64 &total_o) {
        const u64 inc = warp_scan(v, lane);
        o = warp_sum(o);
        __syncthreads();  // the arrays may still be read
        if (lane == 31) {
            sh->scan[0][warp] = inc;
            sh->scan[1][warp] = o;
        }
        __syncthreads();
        u64 before = inc - v, t = 0;
        total_o = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) before += t;
            t += sh->scan[0][w];
            total_o += sh->scan[1][w];
        }
        total = t;
        return before;
    }

    // Bitonic sort of the first n of kThreads * N values (the others are ~0 and
    // stay), N consecutive ones a thread, ascending: strides inside a thread in registers, inside a warp by
    // shuffles, across warps through `buf` (value i of thread t at
    // buf[i kThreads + t]).
    template <int N>
    __device__ void sort(u64 (&r)[N], unsigned n, u64 *buf) {
        const int first = (int)threadIdx.x * N;
#pragma unroll 1
        for (int size = 2; size < 2 * (int)n; size *= 2) {  // up to the power of two that holds n
#pragma unroll 1
            for (int d = size / 2; d >= N; d /= 2) {
                const int dt = d / N;  // partner thread distance
                if (dt >= 32) {
                    __syncthreads();
#pragma unroll
                    for (int j = 0; j < N; ++j) buf[j * kThreads + threadIdx.x] = r[j];
                    __syncthreads();
                }
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const u64 o = dt >= 32 ? buf[j * kThreads + (threadIdx.x ^ dt)]
                                           : __shfl_xor_sync(0xffffffffu, r[j], dt);
                    const bool low = ((first + j) & d) == 0, up = ((first + j) & size) == 0;
                    r[j] = (low == up) == (r[j] < o) ? r[j] : o;
                }
            }
#pragma unroll
            for (int d = N / 2; d >= 1; d /= 2) {
                if (d >= size) continue;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    if (j & d) continue;
                    const bool up = ((first + j) & size) == 0;
                    if ((r[j] > r[j | d]) == up) {
                        const u64 t = r[j];
                        r[j] = r[j | d];
                        r[j | d] = t;
                    }
                }
            }
        }
        __syncthreads();
    }

    // The list's entries (N a thread) sorted by falling logit, their masses,
    // and the mass before this thread's.
    template <int N>
    __device__ u64 sorted_list(unsigned n, unsigned k, u64 (&r)[N], u64 (&w)[N], u64 &S_k) {
        const unsigned first = threadIdx.x * N;
#pragma unroll
        for (int j = 0; j < N; ++j) r[j] = first + j < n ? fs->sorted[first + j] : ~0ull;
        __syncthreads();
        sort<N>(r, n, fs->sorted);
        u64 own = 0, own_k = 0, total;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            w[j] = first + j < n ? mass_of(weight_of(~(unsigned)(r[j] >> 32))) : 0;
            own += w[j];
            own_k += first + j < k ? w[j] : 0;
        }
        return block_scan(own, total, own_k, S_k);
    }

    __device__ __forceinline__ float weight_of(unsigned key) const {
        return expf(z_of(logit_of(key), m, rt));
    }

    // The first CTA's part of the list way: n candidates in fs->sorted, which
    // hold the cut.  The kept prefix is sorted by index, and the draw is where
    // its running sum crosses u S.
    template <int N>
    __device__ void draw_from_list(int64_t b, unsigned n, unsigned k, bool k_on, float p, u64 S_all) {
        u64 r[N], w[N], S_k, S, nk, total;
        const unsigned first = threadIdx.x * N;
        u64 at = sorted_list<N>(n, k, r, w, S_k);
        const u64 target = p < 1.0f ? share(p, k_on ? S_k : S_all, true) : ~0ull;
        u64 own = 0, own_n = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const unsigned i = first + j;
            const bool in = i < n && i < k && (i == 0 || at < target) &&
                            weight_of(~(unsigned)(r[j] >> 32)) >= min_w;
            at += w[j];
            own += in ? w[j] : 0;
            own_n += in;
            r[j] = in ? (r[j] << 32) | (r[j] >> 32) : ~0ull;  // index, ~key
        }
        block_scan(own, S, own_n, nk);
        sort<N>(r, (unsigned)nk, fs->sorted);
        own = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            w[j] = first + j < (unsigned)nk ? mass_of(weight_of(~(unsigned)r[j])) : 0;
            own += w[j];
        }
        at = block_scan(own, total, 0, total);
        const u64 aim = share(uniform(b), S, false);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (at <= aim && at + w[j] > aim) put(b, (int)(r[j] >> 32), w[j], S, S_all, (unsigned)nk);
            at += w[j];
        }
    }

    // The first CTA's part of a filter's cut: n tokens in fs->sorted, one of
    // which is the last whose rank is below target_cnt or the mass before
    // which is below target_mass; it goes to every CTA.
    template <int N>
    __device__ void cut_from_list(unsigned n, bool by_mass, unsigned target_cnt, u64 target_mass,
                                  unsigned base_cnt, u64 base_mass) {
        u64 r[N], w[N], unused;
        const unsigned first = threadIdx.x * N;
        u64 at = base_mass + sorted_list<N>(n, 0, r, w, unused);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const unsigned rank_ = base_cnt + first + j;
            const u64 end = at + w[j];
            const bool in = by_mass ? at < target_mass : rank_ < target_cnt;
            const bool next = by_mass ? end < target_mass : rank_ + 1 < target_cnt;
            if (first + j < n && in && (!next || first + j + 1 == n)) sh->cut_entry = r[j];
            at = end;
        }
        __syncthreads();
        const u64 entry = sh->cut_entry;
        to_all(&sh->cut_entry, entry);
    }

    // The tokens for which f(x) into the first CTA's list, if there are at most
    // kListMax; their number.  Ends with a cluster barrier.
    template <typename F>
    __device__ unsigned gather(F f) {
        u64 hit[3] = {0, 0, 0};  // of this thread's elements, 136 at most
        unsigned mine = 0;
        int at = 0;
#pragma unroll 1
        for (int c = c0 + lane; c < c1; c += 32, at += E) {
            float v[E];
            El::load(row[c - c0], v);
            unsigned bits = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) bits |= f(clean(v[e])) ? 1u << e : 0u;
            mine += __popc(bits);
            if (at < 64) hit[0] |= (u64)bits << at;
            else if (at < 128) hit[1] |= (u64)bits << (at - 64);
            else hit[2] |= (u64)bits << (at - 128);
        }
        totals(0, mine);
        const unsigned n = all_cnt();
        if (n <= kListMax) {
            unsigned to = (unsigned)warp_scan(mine, lane) - mine;
            for (int r = 0; r < rank; ++r) to += sh->rank_cnt[r];
            for (int w = 0; w < warp; ++w) to += sh->warp_cnt[w];
            u64 *list = cl.map_shared_rank(fs, 0)->sorted;
            for (int i0 = 0; i0 < 192; i0 += 64) {
                u64 bits = i0 == 0 ? hit[0] : i0 == 64 ? hit[1] : hit[2];
                for (; bits; bits &= bits - 1) {
                    const int i = i0 + __ffsll((long long)bits) - 1;
                    const int c = c0 + lane + 32 * (i / E), e = i % E;
                    const float xv = El::one(reinterpret_cast<const typename El::T *>(row + (c - c0)) + e);
                    list[to++] = ((u64)~key_of(xv) << 32) | (unsigned)(c * E + e - shift);
                }
            }
            cl.sync();
        }
        return n;
    }

    __device__ __forceinline__ float uniform(int64_t b) const {
        const float u = a.u[b];
        return u >= 0.0f ? fminf(u, 0x1.fffffep-1f) : 0.0f;
    }

    // log(w / s), through log1p where the share is near one.
    static __device__ __forceinline__ float log_share(u64 w, u64 s) {
        const float sf = __ull2float_rn(s);
        return 2 * w > s ? log1pf(-__fdiv_rn(__ull2float_rn(s - w), sf))
                         : logf(__fdiv_rn(__ull2float_rn(w), sf));
    }

    __device__ void put(int64_t b, int idx, u64 w, u64 S, u64 S_all, unsigned n_kept) {
        a.token[b] = idx;
        a.logp[b] = log_share(w, S);
        a.logp_all[b] = log_share(w, S_all);
        a.kept[b] = (int)n_kept;
    }

    // Histogram of this CTA's elements with z > z_lo by the step of z (level
    // 0), or of those of an interval of keys: masses or counts.
    __device__ void histogram(bool by_mass, int level, float z_lo, unsigned lo, unsigned hi, int sft) {
        for (int i = threadIdx.x; i < 3 * kBins; i += kThreads) (&fs->hist[0][0])[i] = 0;
        __syncthreads();
        const float x_lo = logit_of(lo), x_hi = logit_of(hi);
        each([&](float x, int) {
            const float zx = z(x);
            if (level == 0 ? zx > z_lo : x >= x_lo && x <= x_hi && x > -INFINITY) {
                const int b = level == 0 ? (int)(zx * -kBinsPerZ) : (int)((hi - key_of(x)) >> sft);
                if (by_mass) {
                    const u64 w = mass_of(expf(zx));
                    atomicAdd(&fs->hist[0][b], (unsigned)w & 0x7FFFu);
                    atomicAdd(&fs->hist[1][b], (unsigned)(w >> 15) & 0x7FFFu);
                    atomicAdd(&fs->hist[2][b], (unsigned)(w >> 30));
                } else {
                    atomicAdd(&fs->hist[0][b], 1u);
                }
            }
        });
        cl.sync();
    }

    // The first bin whose end reaches the target, given what lies before the
    // histogram, with what lies before the bin, at every CTA.
    __device__ void select(bool by_mass, u64 target, u64 base) {
        constexpr int kPer = kBins / kThreads;           // bins a thread at most
        const int seg = kBins / C;                       // bins this CTA merges
        const int per = seg > kThreads ? seg / kThreads : 1;
        u64 bin[kPer], own = 0;
        const int first = rank * seg + (int)threadIdx.x * per;
        const bool active = (int)threadIdx.x * per < seg;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            bin[j] = 0;
            if (active && j < per) {
                // a peer past the cluster is read as this one and not counted, so
                // that all the loads are in flight together
                unsigned part[kMaxCluster];
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    if (i > 0 && !by_mass) break;
#pragma unroll
                    for (int r = 0; r < kMaxCluster; ++r)
                        part[r] = cl.map_shared_rank(fs, r < C ? r : rank)->hist[i][first + j];
                    u64 sum = 0;
#pragma unroll
                    for (int r = 0; r < kMaxCluster; ++r) sum += r < C ? part[r] : 0;
                    bin[j] += sum << (15 * i);
                }
                own += bin[j];
            }
        }
        u64 total, unused;
        u64 at = base + block_scan(own, total, 0, unused);
        if (threadIdx.x == 0) sh->sel_bin = kBins;
        to_all(&sh->seg_mass[rank], total);
        cl.sync();
        for (int r = 0; r < rank; ++r) at += sh->seg_mass[r];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (active && j < per) {
                if (at < target && at + bin[j] >= target) {
                    for (int r = 0; r < C; ++r) {
                        Shared *o = cl.map_shared_rank(sh, r);
                        o->sel_bin = first + j;
                        o->sel_mass = at;
                    }
                }
                at += bin[j];
            }
        }
        cl.sync();
    }

    // The cut among tokens of one logit: the first `n` of them in index order.
    __device__ void cut_ties(float x, unsigned n) {
        unsigned mine = 0;
        each([&](float v, int) { mine += v == x; });
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
                    El::load(row[c - c0], v);
#pragma unroll
                    for (int e = 0; e < E; ++e) t += v[e] == x;
                }
                const unsigned inc = (unsigned)warp_scan(t, lane);
                if (before + inc - t < n && n <= before + inc) {
                    unsigned at = before + inc - t;
                    int idx = 0;
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (v[e] == x && ++at == n) idx = c * E + e - shift;
                    for (int r = 0; r < C; ++r) cl.map_shared_rank(sh, r)->cut_idx = idx;
                }
                before += __shfl_sync(0xffffffffu, inc, 31);
            }
        }
        cl.sync();
        cut_x = x;
        cut_idx = sh->cut_idx;
    }

    // The cut of a filter: the last token whose rank is below the target (a
    // count), or the mass before which is.  The caller has checked that the
    // target lies inside the row, at z > z_lo.
    __device__ void cut(bool by_mass, u64 target, float z_lo) {
        unsigned lo = 0, hi = 0xFFFFFFFFu;
        u64 base = 0;  // mass or count before the interval
        int sft = 0;
        // Step b is exactly -(b + 1) / 64 < z <= -b / 64 (the product with 64 is
        // exact); whole steps are counted.
        z_lo = ceilf(fmaxf(z_lo, -32.0f) * -kBinsPerZ) * (-1.0f / kBinsPerZ);
        for (int level = 0;; ++level) {
            histogram(by_mass, level, z_lo, lo, hi, sft);
            select(by_mass, target, base);
            const int bin = sh->sel_bin;
            if (bin < kBins) {
                base = sh->sel_mass;
            } else {  // level 0 only: past the steps, among weights that round to zero
                for (int r = 0; r < C; ++r) base += sh->seg_mass[r];
            }
            // the bin's tokens: an interval of z, or of logits
            const float z0 = bin < kBins ? (float)(bin + 1) * (-1.0f / kBinsPerZ) : -INFINITY;
            const float z1 = (float)bin * (-1.0f / kBinsPerZ);
            const unsigned span = (unsigned)min((u64)(bin + 1) << sft, (u64)(hi - lo) + 1) - 1;
            const float x0 = logit_of(hi - span), x1 = logit_of(hi - ((unsigned)bin << sft));
            auto in_bin = [&](float x) {
                if (level > 0) return x >= x0 && x <= x1 && x > -INFINITY;
                const float zx = z(x);
                return zx <= z1 && (zx > z0 || bin == kBins) && x > -INFINITY;
            };
            const unsigned n = gather(in_bin);
            if (n <= kListMax) {
                if (rank == 0) {
                    const unsigned bc = by_mass ? 0 : (unsigned)base, tc = by_mass ? 0 : (unsigned)target;
                    const u64 bm = by_mass ? base : 0;
                    if (n <= kThreads) cut_from_list<1>(n, by_mass, tc, target, bc, bm);
                    else cut_from_list<kListMax / kThreads>(n, by_mass, tc, target, bc, bm);
                }
                cl.sync();
                cut_x = logit_of(~(unsigned)(sh->cut_entry >> 32));
                cut_idx = (int)(unsigned)sh->cut_entry;
                return;
            }
            // too many to sort: the bin's own interval of keys
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
                for (int w = 0; w < kWarps; ++w) {
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
                const u64 w = mass_of(weight_of(lo));
                // by mass, token i of them is kept when base + i w < target
                const u64 q = !by_mass ? target - base : w ? (target - base + w - 1) / w : 1;
                cut_ties(logit_of(lo), (unsigned)q);
                return;
            }
            sft = max(0, 32 - __clz((int)(hi - lo)) - 11);  // (hi - lo) >> sft < 2048
        }
    }

    // Mass and number of the kept tokens (all of them at every CTA).
    __device__ u64 kept_totals() {
        MassSum s;
        unsigned n = 0, cnt = 0;
#pragma unroll 1
        for (int c = c0 + lane; c < c1; c += 32, n += E) {
            float v[E], w[E];
            El::load(row[c - c0], v);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float x = clean(v[e]);
                w[e] = expf(z(x));
                const bool in = kept(x, w[e], c * E + e - shift);
                w[e] = in ? w[e] : 0.0f;
                cnt += in;
            }
#pragma unroll
            for (int e = 0; e < E; e += 2) s.add2(w[e], w[e + 1]);
        }
        totals(s.total(n), cnt);
        return all_mass();
    }

    __device__ void run(int64_t b) {
        const typename El::T *x = static_cast<const typename El::T *>(a.x) + b * a.ld;
        shift = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(typename El::T));
        const int chunks = (shift + a.V + E - 1) / E;
        c0 = min((rank * kWarps + warp) * a.chunks_per_warp, chunks);
        c1 = min(c0 + a.chunks_per_warp, chunks);
        unsigned cnt;
        const float own_max = load_row(x, cnt);
        float mx = own_max;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (lane == 0) sh->warp_max[warp] = mx;
        if (kFilter)
            for (int i = threadIdx.x; i < kGroups; i += kThreads) fs->grp[rank][i] = 0;
        __syncthreads();
        if ((int)threadIdx.x < C) {
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sh->warp_max[w]);
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
        const float T = kFilter && a.temperature ? a.temperature[b] : 1.0f;
        const bool greedy = !(T > 0.0f);
        rt = __fdiv_rn(1.0f, greedy ? 1.0f : T);
        regular = m < INFINITY && rt > 0.0f && rt < INFINITY;
        int k = 0x7FFFFFFF;
        float p = 1.0f;
        min_w = 0.0f;
        cut_x = -INFINITY;
        cut_idx = 0;
        if (kFilter) {
            k = greedy ? 1 : a.top_k && a.top_k[b] > 0 ? a.top_k[b] : 0x7FFFFFFF;
            if (a.top_p && a.top_p[b] < 1.0f) p = a.top_p[b];
            if (a.min_p) min_w = fminf(fmaxf(a.min_p[b], 0.0f), 1.0f);
        }
        if (kFilter && k > 1 && k < 0x7FFFFFFF) {  // the threads' maxima, to every CTA
            const float zx = z_of(own_max, m, rt);
            if (zx > -32.0f) atomicAdd(&fs->grp[rank][(int)(zx * -kGroupsPerZ)], 1u);
            __syncthreads();
            for (int i = threadIdx.x; i < C * kGroups; i += kThreads)
                if (i / kGroups != rank)
                    cl.map_shared_rank(fs, i / kGroups)->grp[rank][i % kGroups] = fs->grp[rank][i % kGroups];
        }
        totals(weigh(), cnt);
        const u64 S_all = all_mass();
        u64 S = S_all;
        unsigned n_kept = all_cnt();
        if (kFilter && (k < 0x7FFFFFFF || p < 1.0f || min_w > 0.0f)) {
            const unsigned finite = n_kept;
            const bool k_on = (unsigned)k < finite;
            bool cut_any = min_w > 0.0f;
            if (k == 1 || p <= 0.0f) {
                cut_ties(m, 1);
                cut_any = true;
            } else if (k_on || p < 1.0f || cut_any) {
                // no token at or below z_lo matters: the highest of the filters' bounds
                float z_lo = min_w > 0.0f ? z_below(min_w) : -INFINITY;
                float z_p = -INFINITY;
                if (!k_on && p < 1.0f)
                    z_p = z_below(0.999f * (1.0f - p) * (__ull2float_rn(S_all) * 0x1p-45f) / (float)a.V);
                z_lo = fmaxf(z_lo, z_p);
                if (k_on) {
                    unsigned g4[kGroups / 32], sum = 0;  // every warp scans the groups itself
#pragma unroll
                    for (int j = 0; j < kGroups / 32; ++j) {
                        g4[j] = 0;
                        for (int r = 0; r < C; ++r) g4[j] += fs->grp[r][lane * (kGroups / 32) + j];
                        sum += g4[j];
                    }
                    unsigned upto = (unsigned)warp_scan(sum, lane) - sum;
                    int g = kGroups;
#pragma unroll
                    for (int j = kGroups / 32 - 1; j >= 0; --j) {
                        unsigned t = upto;
                        for (int i = 0; i <= j; ++i) t += g4[i];
                        if (t >= (unsigned)k) g = lane * (kGroups / 32) + j;
                    }
                    g = __reduce_min_sync(0xffffffffu, g);
                    const float z_k = g < kGroups ? (float)(g + 1) * (-1.0f / kGroupsPerZ) : -INFINITY;
                    // with top-p the mass of all k counts, whatever min-p cuts
                    z_lo = p < 1.0f ? z_k : fmaxf(z_lo, z_k);
                }
                const bool everything = finite <= kListMax;
                if (everything || z_lo > -INFINITY) {
                    auto in_list = [&](float xv) {
                        return everything ? xv > -INFINITY : z(xv) > z_lo;
                    };
                    const unsigned n_c = gather(in_list);
                    if (n_c <= kListMax) {
                        if (rank != 0) return;
                        const unsigned kk = k_on ? (unsigned)k : finite;
                        if (n_c <= kThreads) draw_from_list<1>(b, n_c, kk, k_on, p, S_all);
                        else if (n_c <= 4 * kThreads) draw_from_list<4>(b, n_c, kk, k_on, p, S_all);
                        else draw_from_list<kListMax / kThreads>(b, n_c, kk, k_on, p, S_all);
                        return;
                    }
                }
                for (int by_mass = 0; by_mass < 2; ++by_mass) {
                    if (by_mass ? p >= 1.0f : !k_on) continue;
                    u64 target = (u64)(unsigned)k;
                    if (by_mass) {
                        const float own_min = min_w;  // min-p does not count here
                        min_w = 0.0f;
                        target = share(p, k_on ? kept_totals() : S_all, true);
                        min_w = own_min;
                    }
                    cut(by_mass, target, by_mass ? z_p : -INFINITY);
                    cut_any = true;
                }
            }
            if (cut_any) {
                S = kept_totals();
                n_kept = all_cnt();
            }
        }
        // the draw: the CTA and the warp range in which the running sum exceeds
        // u S; then all warps sum a part of that range, then a lane its own
        const u64 aim = share(uniform(b), S, false);
        u64 before = 0;
        for (int r = 0; r < rank; ++r) before += sh->rank_mass[r];
        if (before > aim || before + sh->rank_mass[rank] <= aim) return;
        int wi = 0;
        while (wi < kWarps - 1 && before + sh->warp_mass[wi] <= aim) before += sh->warp_mass[wi++];
        const typename El::T *src =
            reinterpret_cast<const typename El::T *>(row + (wi - warp) * a.chunks_per_warp);
        const int r0 = min((rank * kWarps + wi) * a.chunks_per_warp, chunks);
        const int n = (min(r0 + a.chunks_per_warp, chunks) - r0) * E;  // elements of the range
        const int per = (n + kThreads - 1) / kThreads;
        const int l0 = min((int)threadIdx.x * per, n), l1 = min(l0 + per, n);
        auto weight = [&](int i) -> u64 {
            const float xv = clean(El::one(src + i)), w = expf(z(xv));
            return kept(xv, w, r0 * E + i - shift) ? mass_of(w) : 0;
        };
        u64 own = 0, all;
#pragma unroll 1
        for (int i = l0; i < l1; ++i) own += weight(i);
        before += block_scan(own, all, 0, all);
        if (before > aim || before + own <= aim) return;
#pragma unroll 1
        for (int i = l0; i < l1; ++i) {
            const u64 w = weight(i);
            if (before <= aim && before + w > aim) put(b, r0 * E + i - shift, w, S, S_all, n_kept);
            before += w;
        }
    }
};

template <bool kBf16, bool kFilter, int kThreads>
__global__ void __launch_bounds__(kThreads, (kThreads == 256 ? 3 : 2) - kFilter)
sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    jet::griddep_launch_dependents();
    jet::griddep_wait();
    Sampler<kBf16, kFilter, kThreads> s(a);
    s.C = (int)s.cl.num_blocks();
    s.rank = (int)s.cl.block_rank();
    s.lane = threadIdx.x & 31;
    s.warp = threadIdx.x >> 5;
    constexpr size_t kHead = (sizeof(Shared) + 15) / 16 * 16;
    s.sh = reinterpret_cast<Shared *>(smem);
    s.fs = reinterpret_cast<FilterShared *>(smem + kHead);
    s.row = reinterpret_cast<uint4 *>(smem + kHead + (kFilter ? sizeof(FilterShared) : 0)) +
            s.warp * a.chunks_per_warp;
    s.run(blockIdx.x / s.C);
}

template <int kThreads>
void (*kernel_for(bool bf16, bool filter))(SampleArgs) {
    return bf16 ? (filter ? sample_kernel<true, true, kThreads> : sample_kernel<true, false, kThreads>)
                : (filter ? sample_kernel<false, true, kThreads> : sample_kernel<false, false, kThreads>);
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
    // the fewest that keep a slice within 64 KB or so; a slice has 256 chunks at least.
    int C = B * kMaxCluster <= 2 * (int64_t)dev.num_sms ? kMaxCluster : 1;
    while (C < kMaxCluster && chunks * 16 > (int64_t)C * 64 * 1024 + 2048) C *= 2;
    while (C > 1 && chunks < (int64_t)C * 256) C /= 2;
    // 512 threads a CTA where the SMs are not full anyway
    const int threads = B * C <= (int64_t)dev.num_sms ? 512 : 256;
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
    const int64_t parts = (int64_t)C * (threads / 32);
    a.chunks_per_warp = (int)(((chunks + parts - 1) / parts + 31) / 32 * 32);
    const size_t smem = (sizeof(Shared) + 15) / 16 * 16 + (filter ? sizeof(FilterShared) : 0) +
                        (size_t)(threads / 32) * a.chunks_per_warp * 16;
    void (*kernel)(SampleArgs) =
        threads == 512 ? kernel_for<512>(bf16, filter) : kernel_for<256>(bf16, filter);
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
        cudaSuccess) {
        cudaGetLastError();
        return JET_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * C));
    cfg.blockDim = dim3((unsigned)threads);
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
