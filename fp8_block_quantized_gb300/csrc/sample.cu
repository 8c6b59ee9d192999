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
// A cluster of 1 to 8 CTAs takes one row; each warp owns a contiguous range of
// it, so that a running sum in index order needs only one total per warp.
// Without a filter the row is read twice, for the maximum and for the weights
// (the second time mostly from L2), and two cluster barriers lead to the draw.
// With one the CTAs hold the row in shared memory, read from HBM once
// (cp.async).
//
// The filters' cut (the last kept token) is found without a sort of the row.
// A bound z_lo is taken below which it cannot lie (top-k: a group of z up to
// which k of the threads' own maxima lie; top-p: all tokens below w = (1 - p)
// S / V together have less weight than (1 - p) S; min-p: its own weight).  When
// at most kListMax tokens lie above it, they go to the first CTA, which finds
// the cut and draws, while the others end.  Flat distributions and large k take
// the general way: a histogram of counts and masses over 2048 steps of z finds
// the step the cut lies in, and the first CTA finds it among the tokens of that
// step; a step with too many of them is split again on the bits of the logits,
// and one of equal logits by counting.
//
// Without a filter, 256 rows of 128256 binary32 logits take 44.3 us (2.96 TB/s,
// 44% of a copy's rate), in BF16 38.3: 26 instructions a logit in two passes with
// a barrier behind each.  With them, few rows are bound by those barriers and the
// passes over shared memory (15 such rows in BF16, one wave of clusters: 13 us
// where short lists suffice, 19 with long ones, 28 for flat nuclei).
#include <cooperative_groups.h>

#include <algorithm>

#include "jet_common.cuh"

namespace {

namespace cg = cooperative_groups;

constexpr int kMaxCluster = 8;
constexpr int kMaxWarps = 16;
constexpr int kBins = 2048;           // steps of 1/64 of z; z <= -32 is bin kBins
constexpr float kBinsPerZ = 64.0f;
constexpr int kGroups = 128;          // groups of 16 steps: 1/4 of z
constexpr float kGroupsPerZ = 4.0f;
constexpr int kListMax = 2048;        // tokens the first CTA takes
constexpr int kRankMax = 256;         // values sorted by counting
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
// ranks are written by the peers and read after a cluster barrier, and between
// those reads and the peers' next writes lies another one.  The totals have no
// barrier of their own there: consecutive ones go to two copies in turn, so that
// the barrier of each parts the reads of its copy's last use from the next writes.
struct Shared {
    u64 warp_mass[kMaxWarps], rank_mass[2][kMaxCluster], seg_mass[kMaxCluster];
    u64 scan[2][kMaxWarps], sel_mass, cut_entry;
    unsigned list_range[4][kMaxWarps], list_left;
    unsigned warp_cnt[kMaxWarps], rank_cnt[2][kMaxCluster];
    float warp_max[kMaxWarps], rank_max[kMaxCluster];
    unsigned lo, hi, rank_lo[kMaxCluster], rank_hi[kMaxCluster];
    int sel_bin;  // the selected bin
    int cut_idx;
};

// With a filter.
static_assert(kListMax >= kBins, "the list's room takes the peers' bins, in rounded parts");
struct FilterShared {
    // counts, or masses in three 15-bit parts: shared-memory atomics on 32 bits
    // run in hardware, and 2^17 tokens of one CTA cannot overflow a part
    unsigned hist[3][kBins];
    u64 list[kListMax + 8 * kMaxCluster];  // ~key, index; at the first CTA
    alignas(16) unsigned grp[kMaxCluster][kGroups];  // threads' maxima by group of z
};

constexpr size_t kHead = (sizeof(Shared) + 15) / 16 * 16;

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
    static __device__ __forceinline__ float largest() { return 0x1.fffffep127f; }
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
    static __device__ __forceinline__ float largest() { return 0x1.fep127f; }
};

__device__ __forceinline__ u64 mass_of(float w) { return __float2ull_rn(w * 0x1p45f); }

// floor(f s) and ceil(f s) for 0 <= f < 1, exact: f = mant 2^-sh.
__device__ __noinline__ u64 share(float f, u64 s, bool up) {
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

// Sums of round(w 2^45) of one thread, weights of 1 at most, in two 32-bit halves
// that are carried into 64 bits before kRun weights could overflow them: adding
// 2^23 to w 2^22 leaves its integer part `hi` in the low bits; what is left,
// times 2^23, is rounded the same way.  Exact, and without the 64-bit
// conversion, whose rate is a quarter of the multiply-adds'.
struct MassSum {
    static constexpr unsigned kRun = 256;  // 2^8 2^22 in either half
    u64 sum = 0;
    unsigned hi = 0, lo = 0, n = 0;
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
    // After `added` more weights, 32 at most.
    __device__ __forceinline__ void count(unsigned added) {
        n += added;
        if (n >= kRun) carry();
    }
    __device__ __forceinline__ void carry() {
        sum += ((u64)(hi - n * 0x4B000000u) << 23) + (u64)(int64_t)(int)(lo - n * 0x4B400000u);
        hi = lo = n = 0;
    }
    __device__ __forceinline__ u64 total() {
        carry();
        return sum;
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

// The code of a row runs once, and fetching it takes time: what is used in
// several places is not inlined.

struct Scan {
    u64 before, total, other;
};

// Sums over the CTA: of v over the threads before this one and over all, and of
// o over all.
__device__ __noinline__ Scan block_scan(u64 v, u64 o, u64 (*sums)[kMaxWarps]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    const u64 inc = warp_scan(v, lane);
    o = warp_sum(o);
    __syncthreads();  // the sums may still be read
    if (lane == 31) {
        sums[0][warp] = inc;
        sums[1][warp] = o;
    }
    __syncthreads();
    const u64 w = warp_scan(lane < nwarps ? sums[0][lane] : 0, lane);
    Scan r;
    r.total = __shfl_sync(0xffffffffu, w, 31);
    const u64 ahead = __shfl_sync(0xffffffffu, w, warp == 0 ? 0 : warp - 1);
    r.before = inc - v + (warp == 0 ? 0 : ahead);
    r.other = warp_sum(lane < nwarps ? sums[1][lane] : 0);
    return r;
}

// Sort of the first n values (distinct; the others are ~0 and stay), one a
// thread, ascending.  Up to kRankMax of them: a value's place is the number of
// smaller ones, counted by neighbouring threads in turn.  Else bitonic: inside a
// warp by shuffles, across warps through `buf`.
template <int kThreads>
__device__ __noinline__ u64 block_sort(u64 r, unsigned n, u64 *buf) {
    const int i = threadIdx.x;
    if (n <= kRankMax) {
        const int sh = n <= kThreads / 8 ? 3 : n <= kThreads / 4 ? 2 : 1;  // 2^sh threads a value
        __syncthreads();
        buf[i] = r;
        __syncthreads();
        const u64 own = buf[i >> sh];
        unsigned at = 0;
#pragma unroll 8
        for (unsigned j = i & ((1 << sh) - 1); j < n; j += 1 << sh) at += buf[j] < own;
        for (int d = 1; d < 1 << sh; d *= 2) at += __shfl_xor_sync(0xffffffffu, at, d);
        __syncthreads();
        if ((i & ((1 << sh) - 1)) == 0 && (unsigned)(i >> sh) < n) buf[at] = own;
        __syncthreads();
        r = buf[i];
        __syncthreads();
        return r;
    }
#pragma unroll 1
    for (int size = 2; size < 2 * (int)n; size *= 2) {  // up to the power of two that holds n
#pragma unroll 1
        for (int d = size / 2; d >= 1; d /= 2) {
            u64 o;
            if (d >= 32) {
                __syncthreads();
                buf[i] = r;
                __syncthreads();
                o = buf[i ^ d];
            } else {
                o = __shfl_xor_sync(0xffffffffu, r, d);
            }
            const bool low = (i & d) == 0, up = (i & size) == 0;
            r = (low == up) == (r < o) ? r : o;
        }
    }
    __syncthreads();
    return r;
}

// log(w / s), through log1p where the share is near one.
__device__ __noinline__ float log_share(u64 w, u64 s) {
    const float sf = __ull2float_rn(s);
    return 2 * w > s ? log1pf(-__fdiv_rn(__ull2float_rn(s - w), sf))
                     : logf(__fdiv_rn(__ull2float_rn(w), sf));
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
    uint4 *row;   // with a filter: this warp's chunk c0 is row[0]
    const typename El::T *x;  // the row in global memory
    bool infinite;  // the row holds +inf
    bool odd;       // this thread's part of it holds a NaN
    int C, rank, lane, warp;
    int c0, c1;   // this warp's chunks of the row
    int shift;    // elements before the row in its first chunk
    float m, rt, min_w;
    float cut_x;
    int cut_idx;
    int copy;     // of the last totals, the same in every thread of the cluster

    __device__ Sampler(const SampleArgs &args) : a(args), cl(cg::this_cluster()), infinite(false), odd(false), copy(1) {}

    // m is finite and rt a normal number, so x = -inf gives -inf and nothing else
    // is undefined.
    __device__ __forceinline__ float z(float x) const { return __fmul_rn(__fadd_rn(x, -m), rt); }

    // A chunk of the row in shared memory.
    __device__ __forceinline__ void chunk(int c, float (&v)[E]) const {
        El::load(row[c - c0], v);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = clean(v[e]);
    }

    // Whether all of a chunk lies inside the row.
    __device__ __forceinline__ bool whole(int c) const {
        return c * E >= shift && (c + 1) * E - shift <= a.V;
    }

    // A chunk at the row's ends, element by element.
    __device__ __forceinline__ void ragged(int c, float (&v)[E]) const {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int idx = c * E + e - shift;
            v[e] = idx >= 0 && idx < a.V ? El::one(x + idx) : -INFINITY;
        }
    }

    // +inf counts as the type's largest finite number.
    static __device__ __forceinline__ void lower(float (&v)[E]) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = v[e] == INFINITY ? El::largest() : v[e];
    }

    // A row that holds +inf: lowered, in shared memory by the threads that
    // copied it.  Its new maximum.
    __device__ float lower_infinities() {
        infinite = true;
        if (kFilter) {
            for (int c = c0 + lane; c < c1; c += 32) {
                float v[E];
                El::load(row[c - c0], v);
                lower(v);
                row[c - c0] = El::store(v);
            }
        }
        return El::largest();
    }

    // f(values) for every chunk of this warp's range, the values as they are in
    // global memory: whole chunks several loads ahead, then the row's ragged
    // ends.  After some of them, done(their number).
    template <typename F, typename G>
    __device__ __forceinline__ void global_chunks(F f, G done) {
        const int first = shift > 0, past = (shift + a.V) / E;  // the whole chunks
        int c = max(c0, first) + lane;
        const int end = min(c1, past);
        const uint4 *p = reinterpret_cast<const uint4 *>(x - shift) + c;
        float v[E];
        constexpr int kN = 32 / E;  // loads ahead: 256 x 128256 binary32 take 44.2 us with 8, 46.1 with 4
        for (; c + 32 * (kN - 1) < end; c += 32 * kN, p += 32 * kN) {
            uint4 t[kN];
#pragma unroll
            for (int i = 0; i < kN; ++i) t[i] = p[32 * i];
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                El::load(t[i], v);
                f(v);
            }
            done(kN);
        }
#pragma unroll 1
        for (; c < end; c += 32, p += 32) {
            El::load(*p, v);
            f(v);
            done(1);
        }
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {  // chunk 0 and chunk `past`, where they are not whole
            const int r = i == 0 ? 0 : past;
            if (lane == i && r >= c0 && r < c1 && !whole(r) && (i == 0 || past > 0)) {
                ragged(r, v);
                f(v);
                done(1);
            }
        }
    }

    // f(values, chunk) for every chunk of this warp's range in shared memory.
    template <typename F>
    __device__ __forceinline__ void chunks(F f) {
        for (int c = c0 + lane; c < c1; c += 32) {
            float v[E];
            chunk(c, v);
            f(v, c);
        }
    }

    // Element i of this warp's range in shared memory (its index is i - skip()).
    __device__ __forceinline__ float element(int i) const {
        return clean(El::one(reinterpret_cast<const typename El::T *>(row) + i));
    }
    __device__ __forceinline__ int elements() const { return (c1 - c0) * E; }
    __device__ __forceinline__ int skip() const { return shift - c0 * E; }

    // f(x, index) for every element of this warp's range in shared memory.
    template <typename F>
    __device__ __forceinline__ void each(F f) {
        chunks([&](const float (&v)[E], int c) {
#pragma unroll
            for (int e = 0; e < E; ++e) f(v[e], c * E + e - shift);
        });
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
    // barrier, after which this copy of rank_mass / rank_cnt holds every CTA's
    // totals.
    __device__ void totals(u64 mass, unsigned cnt) {
        copy ^= 1;
        mass = warp_sum(mass);
        cnt = __reduce_add_sync(0xffffffffu, cnt);
        if (lane == 0) {
            sh->warp_mass[warp] = mass;
            sh->warp_cnt[warp] = cnt;
        }
        __syncthreads();
        if (warp == 0) {
            const u64 t = warp_sum(lane < kWarps ? sh->warp_mass[lane] : 0);
            const unsigned n = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh->warp_cnt[lane] : 0);
            to_all(&sh->rank_mass[copy][rank], t);
            to_all(&sh->rank_cnt[copy][rank], n);
        }
        cl.sync();
    }

    __device__ u64 all_mass() const {
        u64 t = 0;
        for (int r = 0; r < C; ++r) t += sh->rank_mass[copy][r];
        return t;
    }
    __device__ unsigned all_cnt() const {
        unsigned t = 0;
        for (int r = 0; r < C; ++r) t += sh->rank_cnt[copy][r];
        return t;
    }

    // The maximum of this thread's part of the row and the number of logits in it
    // that can be drawn.  With a filter the part goes to shared memory by this
    // thread's own copies, four groups of them in flight.
    __device__ float load_row(unsigned &finite) {
        float mx = -INFINITY;
        unsigned n = 0;
        auto take = [&](const float (&v)[E]) {
            float sum = v[0];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                mx = fmaxf(mx, v[e]);  // a NaN leaves it as it is
                if (e > 0) sum += v[e];
            }
            n += E;
            if (!(fabsf(sum) < INFINITY)) {  // some may be -inf or NaN
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    n -= !(v[e] > -INFINITY);
                    odd |= v[e] != v[e];
                }
            }
        };
        if (!kFilter) {
            global_chunks([&](float (&v)[E]) { take(v); }, [](int) {});
            finite = n;
            return mx;
        }
        const uint4 *src = reinterpret_cast<const uint4 *>(x - shift);
        uint4 *dst = row - c0;
        const int quarter = (a.chunks_per_warp / 32 + 3) / 4 * 32;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            const int end = min(c0 + (i + 1) * quarter, c1);
#pragma unroll 1
            for (int c = c0 + i * quarter + lane; c < end; c += 32) {
                if (whole(c)) {
                    cp_async16(dst + c, src + c);
                } else {
                    float v[E];
                    ragged(c, v);
                    dst[c] = El::store(v);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            if (i == 0) cp_wait<3>();
            if (i == 1) cp_wait<2>();
            if (i == 2) cp_wait<1>();
            if (i == 3) cp_wait<0>();
            const int end = min(c0 + (i + 1) * quarter, c1);
#pragma unroll 2
            for (int c = c0 + i * quarter + lane; c < end; c += 32) {
                float v[E];
                El::load(dst[c], v);
                take(v);
            }
        }
        finite = n;
        return mx;
    }

    // This thread's weights.
    __device__ __forceinline__ u64 weigh() {
        MassSum s;
        const float2 nm = make_float2(-m, -m), r2 = make_float2(rt, rt);
        auto add = [&](const float (&v)[E]) {
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                float2 zz = __fadd2_rn(make_float2(v[e], v[e + 1]), nm);
                if (kFilter) zz = __fmul2_rn(zz, r2);  // without one r2 is 1
                s.add2(expf(zz.x), expf(zz.y));
            }
        };
        if (kFilter) {
            chunks([&](const float (&v)[E], int) {
                add(v);
                s.count(E);
            });
        } else if (!odd && !infinite) {  // nothing to clean
            global_chunks([&](float (&v)[E]) { add(v); }, [&](int n) { s.count(n * E); });
        } else {
            global_chunks([&](float (&v)[E]) {
                if (infinite) lower(v);
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] = clean(v[e]);
                add(v);
            }, [&](int n) { s.count(n * E); });
        }
        return s.total();
    }

    __device__ __forceinline__ Scan scan(u64 v, u64 o = 0) { return block_scan(v, o, sh->scan); }

    // A buffer of one value a thread.
    __device__ __forceinline__ u64 sort(u64 r, unsigned n) {
        return block_sort<kThreads>(r, n, reinterpret_cast<u64 *>(fs->hist));
    }

    __device__ __forceinline__ float weight_of(unsigned key) const {
        return expf(z(logit_of(key)));
    }

    // Mass of a list value: the key's complement is its upper half, or where the
    // list goes by index its lower.
    __device__ __forceinline__ u64 mass_in(u64 v, bool by_index) const {
        return mass_of(weight_of(~(unsigned)(by_index ? v : v >> 32)));
    }

    // The first CTA's part of the list way for a short list: n candidates in
    // fs->list, which hold the cut, one a thread.  Sorted by falling logit; the
    // kept prefix is then sorted by index, and the draw is where its running
    // sum crosses u S.
    __device__ void draw_from_short(int64_t b, unsigned n, unsigned k, bool k_on, float p, u64 S_all) {
        const unsigned i = threadIdx.x;
        u64 r = sort(i < n ? fs->list[i] : ~0ull, n);
        const float wf = i < n ? weight_of(~(unsigned)(r >> 32)) : 0.0f;
        u64 w = mass_of(wf);
        const Scan by_logit = scan(w, i < k ? w : 0);
        const u64 target = p < 1.0f ? share(p, k_on ? by_logit.other : S_all, true) : ~0ull;
        const bool in = i < n && i < k && (i == 0 || by_logit.before < target) && wf >= min_w;
        const Scan held = scan(in ? w : 0, in);
        const unsigned nk = (unsigned)held.other;
        r = sort(in ? (r << 32) | (r >> 32) : ~0ull, nk);  // index, ~key
        w = i < nk ? mass_in(r, true) : 0;
        const u64 before = scan(w).before;
        const u64 aim = share(uniform(b), held.total, false);
        if (before <= aim && before + w > aim) put(b, (int)(r >> 32), w, held.total, S_all, nk);
    }

    // The same for a long list: top-k, top-p and, by index, the draw are each a
    // cut of what is left.  A thread keeps to its own entries, ~0 where dropped.
    __device__ void draw_from_long(int64_t b, unsigned n, unsigned k, bool k_on, float p, u64 S_all) {
        u64 last = 0;
        Scan held = {0, 0, n};
#pragma unroll 1
        for (int step = 0; step < 3; ++step) {
            u64 target = k;
            if (step == 0 && (!k_on || k >= n)) continue;
            if (step == 1 && p >= 1.0f) continue;
            if (step > 0) {
                // the mass of what is left (by step 2, of what min-p leaves)
                u64 own = 0, own_n = 0;
#pragma unroll 1
                for (unsigned i = threadIdx.x; i < n; i += kThreads) {
                    const u64 v = fs->list[i];
                    if (v == ~0ull) continue;
                    const float w = weight_of(~(unsigned)(v >> 32));
                    const bool out = step == 2 && w < min_w;
                    if (step == 2) fs->list[i] = out ? ~0ull : (v << 32) | (v >> 32);  // index, ~key
                    own += out ? 0 : mass_of(w);
                    own_n += !out;
                }
                held = scan(own, own_n);
                target = step == 1 ? share(p, k_on ? held.total : S_all, true)
                                   : share(uniform(b), held.total, false) + 1;
            }
            last = list_cut(n, step > 0, target, step == 2);
#pragma unroll 1
            for (unsigned i = threadIdx.x; step < 2 && i < n; i += kThreads)
                if (fs->list[i] > last) fs->list[i] = ~0ull;
        }
        if (threadIdx.x == 0)
            put(b, (int)(last >> 32), mass_in(last, true), held.total, S_all, (unsigned)held.other);
    }

    // Among the first n values of the list (distinct; ~0 for none), in rising
    // order, the last one before which less than `target` lies: their number, or
    // their mass.  A histogram of the values' range, then of its bin that holds
    // the target, until a bin's values can be sorted one a thread.
    __device__ u64 list_cut(unsigned n, bool by_mass, u64 target, bool by_index) {
        u64 lo = 0, hi = ~0ull - 1;
        unsigned left = n;
        const u64 *buf = fs->list;
        // f(v) for this thread's values in the range
        auto own = [&](auto f) {
#pragma unroll 1
            for (unsigned i = threadIdx.x; i < n; i += kThreads) {
                const u64 v = fs->list[i];
                if (v >= lo && v <= hi) f(v);
            }
        };
        while (left > kThreads) {
            // their range: by the upper halves, or the lower where those are equal
            unsigned r[4] = {~0u, 0, ~0u, 0};
            own([&](u64 v) {
                r[0] = min(r[0], (unsigned)(v >> 32));
                r[1] = max(r[1], (unsigned)(v >> 32));
                r[2] = min(r[2], (unsigned)v);
                r[3] = max(r[3], (unsigned)v);
            });
            __syncthreads();  // what is shared may still be read
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                r[q] = q % 2 ? __reduce_max_sync(0xffffffffu, r[q]) : __reduce_min_sync(0xffffffffu, r[q]);
                if (lane == 0) sh->list_range[q][warp] = r[q];
            }
            if (threadIdx.x == 0) sh->list_left = 0;
            clear_histogram();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const unsigned w = sh->list_range[q][lane % kWarps];
                r[q] = q % 2 ? __reduce_max_sync(0xffffffffu, w) : __reduce_min_sync(0xffffffffu, w);
            }
            lo = (u64)r[0] << 32 | (r[0] == r[1] ? r[2] : 0);
            hi = (u64)r[1] << 32 | (r[0] == r[1] ? r[3] : by_index ? ~0u : 0x7FFFFFFFu);
            const int sft = max(0, 64 - __clzll((long long)(hi - lo)) - 11);
            own([&](u64 v) {
                count_in((int)((v - lo) >> sft), by_mass, by_mass ? mass_in(v, by_index) : 0);
            });
            __syncthreads();
            constexpr int kPer = kBins / kThreads;
            u64 bin[kPer], sum = 0;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int i = threadIdx.x * kPer + j;
                bin[j] = fs->hist[0][i] + ((u64)fs->hist[1][i] << 15) + ((u64)fs->hist[2][i] << 30);
                sum += bin[j];
            }
            const Scan s = scan(sum);
            if (s.total < target) return hi;  // all of them
            u64 at = s.before;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                if (at < target && at + bin[j] >= target) {
                    sh->sel_bin = threadIdx.x * kPer + j;
                    sh->sel_mass = at;
                }
                at += bin[j];
            }
            __syncthreads();
            target -= sh->sel_mass;
            lo += (u64)sh->sel_bin << sft;
            hi = min(hi, lo + ((1ull << sft) - 1));
            // the bin's values, in any order: they are sorted next
            u64 *some = reinterpret_cast<u64 *>(fs->hist) + kThreads;  // past the sort's
            own([&](u64 v) {
                const unsigned to = atomicAdd(&sh->list_left, 1u);
                if (to < kThreads) some[to] = v;
            });
            __syncthreads();
            left = sh->list_left;
            buf = some;
        }
        const u64 v = sort(threadIdx.x < left ? buf[threadIdx.x] : ~0ull, left);
        const u64 w = threadIdx.x >= left ? 0 : by_mass ? mass_in(v, by_index) : 1;
        const u64 at = scan(w).before;
        if (threadIdx.x < left && at < target && (at + w >= target || threadIdx.x + 1 == left))
            sh->cut_entry = v;
        __syncthreads();
        return sh->cut_entry;
    }

    __device__ void clear_histogram() {
        for (int i = threadIdx.x; i < 3 * kBins; i += kThreads) (&fs->hist[0][0])[i] = 0;
        __syncthreads();
    }

    // One token into a bin of the histogram.
    __device__ __forceinline__ void count_in(int bin, bool by_mass, u64 w) {
        if (by_mass) {
            atomicAdd(&fs->hist[0][bin], (unsigned)w & 0x7FFFu);
            atomicAdd(&fs->hist[1][bin], (unsigned)(w >> 15) & 0x7FFFu);
            atomicAdd(&fs->hist[2][bin], (unsigned)(w >> 30));
        } else {
            atomicAdd(&fs->hist[0][bin], 1u);
        }
    }

    // The tokens for which f(x) into the first CTA's list, if there are at most
    // kListMax; their number.  Ends with a cluster barrier.
    template <typename F>
    __device__ unsigned gather(F f) {
        u64 hit[3] = {0, 0, 0};  // of this thread's elements, 192 at most
        int at = 0;
        chunks([&](const float (&v)[E], int) {
            unsigned bits = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) bits |= f(v[e]) ? 1u << e : 0u;
            if (at < 64) hit[0] |= (u64)bits << at;
            else if (at < 128) hit[1] |= (u64)bits << (at - 64);
            else hit[2] |= (u64)bits << (at - 128);
            at += E;
        });
        const unsigned mine = __popcll(hit[0]) + __popcll(hit[1]) + __popcll(hit[2]);
        totals(0, mine);
        const unsigned n = all_cnt();
        if (n <= kListMax) {
            unsigned to = (unsigned)warp_scan(mine, lane) - mine;
            for (int r = 0; r < rank; ++r) to += sh->rank_cnt[copy][r];
            to += __reduce_add_sync(0xffffffffu, lane < warp ? sh->warp_cnt[lane] : 0);
            u64 *list = cl.map_shared_rank(fs, 0)->list;
#pragma unroll 1
            for (int j0 = 0; j0 < 192; j0 += 64) {
                u64 bits = j0 == 0 ? hit[0] : j0 == 64 ? hit[1] : hit[2];
#pragma unroll 1
                for (; bits; bits &= bits - 1) {
                    const int j = j0 + __ffsll((long long)bits) - 1;
                    const int i = (lane + 32 * (j / E)) * E + j % E;
                    list[to++] = ((u64)~key_of(element(i)) << 32) | (unsigned)(i - skip());
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

    __device__ void put(int64_t b, int idx, u64 w, u64 S, u64 S_all, unsigned n_kept) {
        a.token[b] = idx;
        a.logp[b] = log_share(w, S);
        a.logp_all[b] = log_share(w, S_all);
        a.kept[b] = (int)n_kept;
    }

    // Histogram of this CTA's elements with z > z_lo by the step of z (level
    // 0), or of those of an interval of keys: masses or counts.
    __device__ void histogram(bool by_mass, int level, float z_lo, unsigned lo, unsigned hi, int sft) {
        clear_histogram();
        const float x_lo = logit_of(lo), x_hi = logit_of(hi);
        each([&](float x, int) {
            const float zx = z(x);
            if (level == 0 ? zx > z_lo : x >= x_lo && x <= x_hi && x > -INFINITY) {
                const int b = level == 0 ? (int)(zx * -kBinsPerZ) : (int)((hi - key_of(x)) >> sft);
                count_in(b, by_mass, by_mass ? mass_of(expf(zx)) : 0);
            }
        });
        __syncthreads();
    }

    // The first bin whose end reaches the target, given what lies before the
    // histogram, with what lies before the bin, at every CTA.  Every CTA sends
    // its bins to the CTA that adds them, kBins / C or so each (sent: stores
    // into the peers' shared memory, a third of the time of loads from it).
    __device__ void select(bool by_mass, u64 target, u64 base) {
        constexpr int kPer = kBins / kThreads;  // bins a thread
        const int seg = (kBins / kPer + C - 1) / C * kPer, first = (int)threadIdx.x * kPer;
        ulonglong2 *to = reinterpret_cast<ulonglong2 *>(
            cl.map_shared_rank(fs, first / seg)->list + rank * seg + first % seg);
#pragma unroll
        for (int j = 0; j < kPer; j += 2) {
            u64 v[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int i = first + j + q;
                v[q] = fs->hist[0][i];
                if (by_mass) v[q] += ((u64)fs->hist[1][i] << 15) + ((u64)fs->hist[2][i] << 30);
            }
            to[j / 2] = make_ulonglong2(v[0], v[1]);
        }
        cl.sync();
        // this CTA's bins: `per` a thread, from every rank
        const int past = min(seg, kBins - rank * seg);
        const int per = (seg + kThreads - 1) / kThreads;
        const int at0 = (int)threadIdx.x * per;
        u64 bin[kPer], own = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            bin[j] = 0;
            if (j < per && at0 + j < past)
                for (int r = 0; r < C; ++r) bin[j] += fs->list[r * seg + at0 + j];
            own += bin[j];
        }
        const Scan s = scan(own);
        u64 at = base + s.before;
        if (threadIdx.x == 0) sh->sel_bin = kBins;
        to_all(&sh->seg_mass[rank], s.total);
        cl.sync();
        for (int r = 0; r < rank; ++r) at += sh->seg_mass[r];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (j < per && at0 + j < past && at < target && at + bin[j] >= target) {
                for (int r = 0; r < C; ++r) {
                    Shared *o = cl.map_shared_rank(sh, r);
                    o->sel_bin = rank * seg + at0 + j;
                    o->sel_mass = at;
                }
            }
            at += bin[j];
        }
        cl.sync();
    }

    // The cut among tokens of one logit: the first `n` of them in index order.
    __device__ void cut_ties(float logit, unsigned n) {
        unsigned mine = 0;
        each([&](float v, int) { mine += v == logit; });
        totals(0, mine);
        unsigned before = 0;
        for (int r = 0; r < rank; ++r) before += sh->rank_cnt[copy][r];
        before += __reduce_add_sync(0xffffffffu, lane < warp ? sh->warp_cnt[lane] : 0);
        const unsigned own = sh->warp_cnt[warp];
        if (before < n && n <= before + own) {  // one warp of the cluster
#pragma unroll 1
            for (int i = lane; i - lane < elements(); i += 32) {
                const bool tie = i < elements() && element(i) == logit;
                const unsigned ties = __ballot_sync(0xffffffffu, tie);
                if (tie && before + __popc(ties & ((1u << lane) - 1)) + 1 == n) {
                    for (int r = 0; r < C; ++r) cl.map_shared_rank(sh, r)->cut_idx = i - skip();
                }
                before += __popc(ties);
            }
        }
        cl.sync();
        cut_x = logit;
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
            const float z0 = (float)(bin + 1) * (-1.0f / kBinsPerZ);
            const float z1 = (float)bin * (-1.0f / kBinsPerZ);
            const unsigned span = (unsigned)min((u64)(bin + 1) << sft, (u64)(hi - lo) + 1) - 1;
            const float x0 = logit_of(hi - span), x1 = logit_of(hi - ((unsigned)bin << sft));
            const float below = level > 0 ? nextafterf(x0, -INFINITY) : bin < kBins ? z0 : NAN;
            const float top = level > 0 ? x1 : z1;
            const float off = level > 0 ? 0.0f : -m, mul = level > 0 ? 1.0f : rt;
            auto in_bin = [&](float x) {
                const float v = __fmul_rn(__fadd_rn(x, off), mul);
                return v <= top && !(v <= below) && x > -INFINITY;
            };
            const unsigned n = gather(in_bin);
            if (n <= kListMax) {
                if (rank == 0) {
                    const u64 entry = list_cut(n, by_mass, target - base, false);
                    to_all(&sh->cut_entry, entry);
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
            if (threadIdx.x == 0) {
                sh->lo = 0xFFFFFFFFu;
                sh->hi = 0;
            }
            __syncthreads();
            atomicMin(&sh->lo, klo);
            atomicMax(&sh->hi, khi);
            __syncthreads();
            to_all(&sh->rank_lo[rank], sh->lo);
            to_all(&sh->rank_hi[rank], sh->hi);
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

    // Mass of the kept tokens; their totals at every CTA.
    __device__ u64 kept_totals() {
        MassSum s;
        unsigned cnt = 0;
        const float low = fmaxf(cut_x, -0x1.fffffep127f);  // no -inf is kept
        chunks([&](const float (&v)[E], int c) {
            float w[E];
            const int last = cut_idx - (c * E - shift);  // ties up to this element
#pragma unroll
            for (int e = 0; e < E; ++e) {
                w[e] = expf(z(v[e]));
                const bool in = v[e] >= low && (v[e] > cut_x || e <= last) && w[e] >= min_w;
                w[e] = in ? w[e] : 0.0f;
                cnt += in;
            }
#pragma unroll
            for (int e = 0; e < E; e += 2) s.add2(w[e], w[e + 1]);
            s.count(E);
        });
        totals(s.total(), cnt);
        return all_mass();
    }

    __device__ void run(int64_t b) {
        x = static_cast<const typename El::T *>(a.x) + b * a.ld;
        shift = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(typename El::T));
        const int chunks = (shift + a.V + E - 1) / E;
        c0 = min((rank * kWarps + warp) * a.chunks_per_warp, chunks);
        c1 = min(c0 + a.chunks_per_warp, chunks);
        unsigned cnt;
        const float own_max = load_row(cnt);
        float mx = own_max;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (lane == 0) sh->warp_max[warp] = mx;
        if (kFilter)
            for (int i = threadIdx.x; i < kGroups; i += kThreads) fs->grp[rank][i] = 0;
        __syncthreads();
        cl.barrier_wait();  // the peers have begun: their shared memory is there
        if (warp == 0) {
            mx = lane < kWarps ? sh->warp_max[lane] : -INFINITY;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            to_all(&sh->rank_max[rank], mx);
        }
        cl.sync();
        m = -INFINITY;
        for (int r = 0; r < C; ++r) m = fmaxf(m, sh->rank_max[r]);
        if (m == INFINITY) m = lower_infinities();
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
        rt = fminf(fmaxf(__fdiv_rn(1.0f, greedy ? 1.0f : T), 0x1p-126f), 0x1.fffffep127f);
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
        const bool filtered = kFilter && (k < 0x7FFFFFFF || p < 1.0f || min_w > 0.0f);
        if (filtered && k > 1) {  // the threads' maxima, to every CTA
            const float zx = z(fminf(own_max, m));
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
        if (filtered) {
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
                // every warp scans the groups itself, four a lane
                static_assert(kGroups == 4 * 32, "a quad a lane");
                unsigned g4[4] = {0, 0, 0, 0};
                for (int r = 0; r < C; ++r) {
                    const uint4 q = reinterpret_cast<const uint4 *>(fs->grp[r])[lane];
                    g4[0] += q.x;
                    g4[1] += q.y;
                    g4[2] += q.z;
                    g4[3] += q.w;
                }
                const unsigned sum = g4[0] + g4[1] + g4[2] + g4[3];
                if (k_on) {
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
                // the maxima in whole groups above z_lo: so many tokens at least (a
                // flat nucleus in each of 16 rows: 47 us, 52 with the vain gather)
                const int above = (int)(fmaxf(z_lo, -32.0f) * -kGroupsPerZ);
                unsigned sure = 0;
#pragma unroll
                for (int j = 0; j < kGroups / 32; ++j) sure += lane * (kGroups / 32) + j < above ? g4[j] : 0;
                sure = __reduce_add_sync(0xffffffffu, sure);
                if (everything || (z_lo > -INFINITY && sure <= kListMax)) {
                    auto in_list = [&](float xv) {
                        return everything ? xv > -INFINITY : z(xv) > z_lo;
                    };
                    const unsigned n_c = gather(in_list);
                    if (n_c <= kListMax) {
                        if (rank != 0) return;
                        const unsigned kk = k_on ? (unsigned)k : finite;
                        if (n_c <= kThreads) draw_from_short(b, n_c, kk, k_on, p, S_all);
                        else draw_from_long(b, n_c, kk, k_on, p, S_all);
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
        for (int r = 0; r < rank; ++r) before += sh->rank_mass[copy][r];
        if (before > aim || before + sh->rank_mass[copy][rank] <= aim) return;
        int wi = 0;
        while (wi < kWarps - 1 && before + sh->warp_mass[wi] <= aim) before += sh->warp_mass[wi++];
        const typename El::T *held =
            reinterpret_cast<const typename El::T *>(row + (wi - warp) * a.chunks_per_warp);
        const int r0 = min((rank * kWarps + wi) * a.chunks_per_warp, chunks);
        const int n = (min(r0 + a.chunks_per_warp, chunks) - r0) * E;  // elements of the range
        const int per = (n + kThreads - 1) / kThreads;
        const int l0 = min((int)threadIdx.x * per, n), l1 = min(l0 + per, n);
        auto weight = [&](int i) -> u64 {
            const int idx = r0 * E + i - shift;
            float xv = -INFINITY;
            if (kFilter) xv = clean(El::one(held + i));
            else if (idx >= 0 && idx < a.V) xv = clean(El::one(x + idx));
            if (!kFilter && xv == INFINITY) xv = El::largest();
            const float w = expf(z(xv));
            return kept(xv, w, idx) ? mass_of(w) : 0;
        };
        u64 own = 0;
#pragma unroll 1
        for (int i = l0; i < l1; ++i) own += weight(i);
        before += scan(own).before;
        if (before > aim || before + own <= aim) return;
#pragma unroll 1
        for (int i = l0; i < l1; ++i) {
            const u64 w = weight(i);
            if (before <= aim && before + w > aim) put(b, r0 * E + i - shift, w, S, S_all, n_kept);
            before += w;
        }
    }
};

template <bool kBf16, bool kFilter, int kThreads, int kPerSm>
__global__ void __launch_bounds__(kThreads, kPerSm)
sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    Sampler<kBf16, kFilter, kThreads> s(a);
    // Waited for before the first store to a peer, behind the row's loads.  Nothing
    // is written before it, so it orders nothing (256 x 128256 binary32: 44.5 us,
    // 45.3 with an arrival that does).
    __cluster_barrier_arrive_relaxed();
    jet::griddep_launch_dependents();
    jet::griddep_wait();
    s.C = (int)s.cl.num_blocks();
    s.rank = (int)s.cl.block_rank();
    s.lane = threadIdx.x & 31;
    s.warp = threadIdx.x >> 5;
    s.sh = reinterpret_cast<Shared *>(smem);
    s.fs = reinterpret_cast<FilterShared *>(smem + kHead);
    s.row = reinterpret_cast<uint4 *>(smem + kHead + (kFilter ? sizeof(FilterShared) : 0)) +
            s.warp * a.chunks_per_warp;
    s.run(blockIdx.x / s.C);
}

template <bool kFilter, int kThreads, int kPerSm>
void (*kernel_for(bool bf16))(SampleArgs) {
    return bf16 ? sample_kernel<true, kFilter, kThreads, kPerSm>
                : sample_kernel<false, kFilter, kThreads, kPerSm>;
}

// Chunks of 16 bytes that one warp takes, and the shared memory of a CTA of 512
// threads that holds its slice of the row.
int warp_chunks(int C, int threads, int64_t chunks) {
    const int64_t parts = (int64_t)C * (threads / 32);
    return (int)(((chunks + parts - 1) / parts + 31) / 32 * 32);
}
size_t filter_smem(int C, int64_t chunks) {
    return kHead + sizeof(FilterShared) + (size_t)16 * 16 * warp_chunks(C, 512, chunks);
}
// What one and two CTAs an SM may have of it.
constexpr size_t kOne = 227 * 1024, kHalf = 113 * 1024;

template <int kBytes>
bool aligned_to(const void *p) { return (reinterpret_cast<uintptr_t>(p) & (kBytes - 1)) == 0; }

jet_status sample(const void *logits, bool logits_aligned, int dtype, int64_t B, int64_t V,
                  int64_t ld, const float *u, const float *temperature, const int32_t *top_k,
                  const float *top_p, const float *min_p, int64_t *token, float *logp,
                  float *logp_all, int32_t *kept, jet_stream_t stream) {
    JET_REQUIRE(B >= 0 && V >= 0, JET_ERR_SHAPE);
    JET_REQUIRE(B == 0 || (logits && u && token && logp && logp_all && kept), JET_ERR_NULL);
    JET_REQUIRE((B == 0 || V >= 1) && V <= kSaMaxV && B < ((int64_t)1 << 28) && ld >= V &&
                    ld < ((int64_t)1 << 40) && (dtype == JET_BF16 || dtype == JET_FP32),
                JET_ERR_SHAPE);
    JET_REQUIRE(logits_aligned && aligned_to<4>(u) && aligned_to<4>(temperature) &&
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
    const int64_t sms = dev.num_sms;
    int C = kMaxCluster, threads = 512;
    bool pairs = true;  // two CTAs an SM
    if (!filter) {
        // CTAs per row and threads per CTA, with their times in us.  Few rows: two
        // CTAs of 512 threads an SM (128256 logits in binary32: 1 row 6.9 with
        // 8 x 512, 8.3 with 8 x 256; 16 rows 9.0 and 12.6, 11.9 with 4 x 512; 64
        // rows 16.4 with 4 x 512, 19.1 with 8 x 512), so up to two rows an SM one
        // of 512 a row (300 rows of 32000: 16.5, 19.6 with 2 x 256), except that
        // five of 256 run on an SM (160 rows of 32000: 12.8 with 4 x 256, 14.3
        // with 1 x 512).  More rows: CTAs of 256, as few a row as fill the SMs
        // with slices of 104 KB at most (128256 in BF16: 340 rows 48 with 4, 84
        // with 1; 1024 rows 116 and 146, 133 with 8; 1024 rows of 32000 in BF16:
        // 39 with 1, 41 with 2).  Rows past 384 KB: 8 x 256 (256 rows of 128256
        // in binary32: 44, 54 with 1 x 512).
        while (C > 1 && (B * C > 2 * sms || chunks < (int64_t)C * 256)) C /= 2;
        if (B > sms) {
            auto room = [&](int c) { return c <= kMaxCluster && chunks >= (int64_t)c * 128; };
            if (chunks * 16 > 384 * 1024) {
                C = kMaxCluster;
                threads = 256;
            } else if (B * 8 <= 9 * sms && room(4)) {
                C = 4;
                threads = 256;
            } else if (B > 2 * sms) {
                threads = 256;
                for (C = 1; room(2 * C) && (B * C < 4 * sms || chunks * 16 > (int64_t)C * 104 * 1024);) C *= 2;
            }
        }
    } else {
        // Few rows: the largest cluster with which they run in about one wave,
        // an SM a CTA.  The SMs' groups hold 15 clusters of 8 (and 15 of 7), 23
        // of 6, 28 of 5, 36 of 4 (128256 BF16 logits, us, mixed filters / flat
        // nuclei / top-k: 16 rows 30 / 47 / 23 with 8, 36 / 34 / 21 with 6; 20
        // rows 36 / 34 / 21 with 6, 30 / 50 / 28 with 8; 32 rows 43 / 42 / 23
        // with 4, 42 / 71 / 33 with 8).  More rows: two CTAs an SM of half the
        // registers, again in about one wave while that can be (64 rows 58 / 67
        // / 35, one CTA an SM 62 / 79 / 39; 256 rows 132 / 207 / 100 and 167 /
        // 281 / 125), else as few CTAs a row as its slices allow (300 rows of
        // 32000 binary32 82 / 80 / 65 with 2, 82 / 117 / 74 with 4).  Where
        // slices are too long for two an SM: as few as one CTA can hold (128
        // rows of 151937 binary32 119 / 178 / 81 with 4, 146 / 246 / 111 with 8).
        const int longest = (int)std::max<int64_t>(1, std::min<int64_t>(kMaxCluster, chunks / 256));
        const int64_t wave = sms * 12 / 13;
        auto fits = [&](int c, size_t room) { return c != 7 && filter_smem(c, chunks) <= room; };
        static_assert((kOne - kHead - sizeof(FilterShared)) / (512 * 16) * 8 <= 192, "a thread's bits in gather");
        pairs = false;
        for (C = longest; C > 0; --C)
            if (fits(C, kOne) && B * C <= wave && (C >= 4 || C == longest)) break;
        if (C == 0) {
            pairs = true;
            for (C = longest; C > 0; --C)
                if (fits(C, kHalf) && B * C <= 2 * wave) break;
            if (C == 0)
                for (C = 1; C < kMaxCluster && !fits(C, kHalf);) ++C;
            if (!fits(C, kHalf)) {
                pairs = false;
                for (C = 1; C < kMaxCluster && !fits(C, kOne);) ++C;
            }
        }
    }
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
    a.chunks_per_warp = warp_chunks(C, threads, chunks);
    const size_t smem = filter ? filter_smem(C, chunks) : kHead;
    void (*kernel)(SampleArgs) =
        filter ? (pairs ? kernel_for<true, 512, 2>(bf16) : kernel_for<true, 512, 1>(bf16))
               : (threads == 512 ? kernel_for<false, 512, 2>(bf16) : kernel_for<false, 256, 5>(bf16));
    // The limit is the kernel's, whatever this call needs: another thread may be
    // about to launch it with other sizes.
    if (filter && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)(pairs ? kHalf : kOne)) != cudaSuccess) {
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

}  // namespace

jet_status jet_sample(const void *logits, int dtype, int64_t B, int64_t V, int64_t ld,
                      const float *u, const float *temperature, const int32_t *top_k,
                      const float *top_p, const float *min_p, int64_t *token, float *logp,
                      float *logp_all, int32_t *kept, jet_stream_t stream) {
    return sample(logits, jet::aligned16(logits), dtype, B, V, ld, u, temperature, top_k, top_p,
                  min_p, token, logp, logp_all, kept, stream);
}

jet_status jet_sample_unaligned(const void *logits, int dtype, int64_t B, int64_t V, int64_t ld,
                                const float *u, const float *temperature, const int32_t *top_k,
                                const float *top_p, const float *min_p, int64_t *token,
                                float *logp, float *logp_all, int32_t *kept, jet_stream_t stream) {
    const bool aligned = dtype == JET_FP32 ? aligned_to<4>(logits) : aligned_to<2>(logits);
    return sample(logits, aligned, dtype, B, V, ld, u, temperature, top_k, top_p, min_p, token,
                  logp, logp_all, kept, stream);
}
