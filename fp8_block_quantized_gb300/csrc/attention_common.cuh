// What the attention kernels share: the call's arguments, the segments that a
// call is made of, and how each kernel cuts them into units and key tiles.
#pragma once

#include <cuda_bf16.h>

#include "jet_common.cuh"

namespace jet {
namespace attn {

constexpr int kTile = 128;         // keys of a wide tile
constexpr int kStep = 32;          // keys of a narrow tile
constexpr int kRows = 8;           // rows of a narrow unit
constexpr int kMaxCtas = 160;      // most CTAs of a launch (one on each SM)
constexpr int kNarrowWarps = 8;    // most of a CTA
constexpr int kNarrowWorkers = kMaxCtas * kNarrowWarps;
constexpr int kWideRows = 256;     // rows of a wide unit's pieces
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct Args {
    const uint16_t *q;
    int64_t ldq;
    int64_t T;
    int Hq, Hk, G;                 // G = Hq / Hk
    const uint8_t *kc, *vc;
    int64_t S;
    const float *ks, *vs;
    const int32_t *table;
    int64_t width, bs;
    int bs_shift;                  // log2 of bs, or -1
    const int64_t *off;
    const int32_t *len;
    int B;
    const int64_t *po;
    const int32_t *pl;
    int Ng;
    float scale;
    uint16_t *out;
    int64_t ldo;
    float *lse;
    // Which segments the wide kernel takes: requests' own parts, groups' prefixes.
    bool wide_own, wide_prefix;
    int ctas;                      // of a launch
    int heads, phases;             // narrow: KV heads a worker has, workers a CTA has
    // Workspace.  Partial results of pieces of units that several workers share, two
    // a worker (narrow: heads x kRows rows each, wide: kWideRows); with groups, whole
    // units by row (prefix, then own); and the plan.
    float *part, *part_ml, *wpart, *wpart_ml;
    float *whole, *whole_ml;       // [2][T * Hq][D], [..][2]
    struct Segment *segs;          // [B + Ng]
    int *order;                    // [2][B + Ng] the segments with work (narrow, wide)
    struct Start *starts;          // [kNarrowWorkers + kMaxCtas] of the workers' ranges
    struct Split *splits;          // [the same], in no order
    struct Plan *plan;
};

__device__ __forceinline__ int64_t clamp64(int64_t v, int64_t lo, int64_t hi) {
    return v < lo ? lo : (v > hi ? hi : v);
}

// The number of entries a[1 .. n] that are <= x: the interval of [a[i], a[i+1])
// that holds x, for x >= a[0].
__device__ __forceinline__ int upper(const int64_t *a, int n, int64_t x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a[mid + 1] <= x) lo = mid + 1; else hi = mid;
    }
    return lo;
}

// Keys request b has behind its table row.
__device__ __forceinline__ int keys_of(const Args &a, int b) {
    return (int)clamp64(a.len[b], 0, a.width * a.bs);
}

// The prefix length of group i: at most the keys of its first request.
__device__ __forceinline__ int prefix_of(const Args &a, int i) {
    const int64_t first = a.po[i];
    if (first < 0 || first >= a.B) return 0;
    return (int)clamp64(a.pl[i], 0, keys_of(a, (int)first));
}

// Segment s < B: the own part of request s; B + i: the prefix of group i.
struct Segment {
    int64_t t0;        // first token
    int64_t before;    // tiles of its kernel's segments before it
    int ntok;
    int k0, k1;        // keys
    int row;           // table row
    int r0, r1;        // requests r0 .. r1 - 1
    int base;          // own part: the first new token's position, if its queries see k0 and
                       // the last one's position is k1 - 1; else -1
    int group;         // own part: the request's group, or -1
};

// A worker's range: how many tiles, from which one of the segment order[at] = s on;
// what it needs at first in one read.
struct Start {
    Segment g;
    int64_t left, from;
    int at, s;
    int empty;         // the plan's
    int pad;
};

struct Plan {
    int64_t total[2];  // tiles (narrow, wide)
    int workers[2];    // none of them without a tile
    int empty;         // segments with tokens and no keys
    int splits;        // units that more than one worker has (without groups)
    int many;          // whether one of them has more than kManyPieces pieces
};
// A row of more pieces than this is joined by the eight warps of a CTA, not by one (one
// request of 4001 keys: 17.1 us, with one warp 36.2; two of 100000 to 131072: 87 and 102).
constexpr int kManyPieces = 8;

// A unit that more than one worker has, as the first worker that begins in its middle
// tells it the join.
struct Split {
    int64_t token;     // the unit's first row: token and query head within the KV head's group
    int sub;
    int head;          // its first KV head
    int rows;
    int n, c0, first;  // pieces: their number, the first one's worker and slot
};

// Position of token t of segment s.
__device__ __forceinline__ int position(const Args &a, const Segment &g, int s, int64_t t) {
    if (g.base >= 0) return g.base + (int)(t - g.t0);
    int b = s;
    if (s >= a.B) b = min(g.r0 + upper(a.off + g.r0, g.r1 - g.r0, t), a.B - 1);
    return (int)clamp64((int64_t)a.len[b] - (a.off[b + 1] - t), -1, 0x7FFFFFFF);
}

// Narrow units: 8 rows of each of `heads` KV heads, whose keys lie side by side.
struct Narrow {
    int rtiles, groups, ktiles;  // row tiles, groups of heads, key tiles
    __device__ Narrow(const Args &a, const Segment &g) {
        rtiles = (int)(((int64_t)g.ntok * a.G + kRows - 1) / kRows);
        groups = (a.Hk + a.heads - 1) / a.heads;
        ktiles = (int)(((int64_t)g.k1 - g.k0 + kStep - 1) / kStep);
    }
    __device__ int64_t tiles() const { return (int64_t)rtiles * groups * ktiles; }
};

// Wide units: up to 256 rows of whole tokens with tiles of 128 keys, or, where a
// segment has at most 128 rows, all of them with pairs of tiles.  Tiles past the
// last key that a row tile sees are not in the list.
struct Wide {
    int tokens;        // of a row tile
    int rtiles, keys;  // keys of a tile (or pair)
    __device__ Wide(const Args &a, const Segment &g) {
        const bool one = (int64_t)g.ntok * a.G <= 128;
        tokens = one ? (g.ntok > 0 ? g.ntok : 1) : kWideRows / a.G;
        keys = one ? 2 * kTile : kTile;
        rtiles = (g.ntok + tokens - 1) / tokens;
    }
    __device__ int ktiles(const Segment &g, int rt) const {
        const int64_t end = g.base >= 0 ? g.base + min((int64_t)g.ntok, (rt + 1) * (int64_t)tokens) : g.k1;
        return (int)((end - g.k0 + keys - 1) / keys);
    }
    // tiles of one head in the row tiles [r0, r1), every `step`th of them
    __device__ int64_t head_tiles(const Segment &g, int r0, int r1, int step = 1) const {
        if (g.base < 0) return r1 > r0 ? (int64_t)((r1 - r0 + step - 1) / step) * ktiles(g, 0) : 0;
        int64_t n = 0;
        for (int r = r0; r < r1; r += step) n += ktiles(g, r);
        return n;
    }
    __device__ int64_t tiles(const Args &a, const Segment &g) const { return head_tiles(g, 0, rtiles) * a.Hk; }
};

// The worker that has tile x when `total` tiles are dealt to `workers` in equal
// ranges (worker c: from total c / workers on).
__device__ __forceinline__ int worker_of(int64_t x, int64_t total, int64_t workers) {
    return (int)(((x + 1) * workers - 1) / total);
}

// The pieces of a unit of `tiles` tiles from u0 on, dealt to several workers: worker
// c's is its first piece (slot 2 c) where its range begins in the unit, else its last.
struct Pieces {
    int c0, n, first;  // the first worker and its slot; their number
    __device__ Pieces(int64_t u0, int64_t tiles, int64_t total, int64_t workers) {
        c0 = worker_of(u0, total, workers);
        n = worker_of(u0 + tiles - 1, total, workers) - c0 + 1;
        first = 2 * c0 + (total * c0 / workers >= u0 ? 0 : 1);
    }
    __device__ int64_t slot(int i) const { return i == 0 ? first : 2 * (c0 + i); }
};

// Adds the unit of `tiles` tiles that worker `me` begins in, `in` tiles from its start, to
// the splits, if it is the first to.
__device__ __forceinline__ void tell_split(const Args &a, bool wide, int me, const Segment &g, int64_t from,
                                           int in, int tiles, int64_t token, int sub, int head, int rows) {
    const int64_t total = a.plan->total[wide], workers = a.plan->workers[wide], u0 = g.before + from - in;
    if (in == 0 || total * (me - 1) / workers > u0) return;
    const Pieces p(u0, tiles, total, workers);
    Split sp;
    sp.token = token, sp.sub = sub, sp.head = head, sp.rows = rows;
    sp.n = p.n, sp.c0 = p.c0, sp.first = p.first;
    if (p.n > kManyPieces) a.plan->many = 1;
    a.splits[atomicAdd(&a.plan->splits, 1)] = sp;
}

// Block of key p and the key's place in it.
__device__ __forceinline__ uint32_t block_of(const Args &a, uint32_t p, uint32_t &at) {
    const uint32_t b = a.bs_shift >= 0 ? p >> a.bs_shift : p / (uint32_t)a.bs;
    at = p - b * (uint32_t)a.bs;
    return b;
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t codes_f16(uint32_t two) {  // low two codes -> f16x2
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
        : "=r"(r)
        : "r"(two));
    return r;
}
__device__ __forceinline__ uint32_t codes_f16_hi(uint32_t two) {  // high two codes
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
        : "=r"(r)
        : "r"(two));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Bits 0x80 where one of the four times four codes is NaN (0x7F or 0xFF).
__device__ __forceinline__ uint32_t nan_bits(uint4 v) {
    auto top = [](uint32_t w) { return (w & 0x7F7F7F7Fu) + 0x01010101u; };
    return (top(v.x) | top(v.y) | top(v.z) | top(v.w)) & 0x80808080u;
}

// lse in natural units and the factor of an output from a row's reference and sum: no
// key, no weight.  A NaN scale of the keys comes in here: the scores' factors are held
// above 2^-126, which leaves a NaN out.
__device__ __forceinline__ float nan_or_zero(float ks) { return ks == ks ? 0.0f : ks; }
__device__ __forceinline__ float row_lse(float m, float l, float ks) {
    return l == 0.0f ? -INFINITY : kLn2 * (m + log2f(l)) + nan_or_zero(ks);
}
__device__ __forceinline__ float row_factor(float vs, float l, float ks) {
    return l == 0.0f ? 0.0f : vs / l + nan_or_zero(ks);
}

// The power of two that brings a row's largest channel to [2^14, 2^15).
__device__ __forceinline__ float row_power(float top) {
    const int e = min(254, 268 - (int)(__float_as_uint(top) >> 23));
    return top == 0.0f ? 1.0f : __uint_as_float((uint32_t)max(e, 1) << 23);
}

// 1 / v of a power of two from 2^-126 to 2^127.
__device__ __forceinline__ float inverse_power(float v) {
    const uint32_t e = __float_as_uint(v) >> 23;
    return __uint_as_float(e == 254 ? 1u << 22 : (254u - e) << 23);
}

// The rows of the segments without keys, where no join writes them (without
// groups).
template <int D>
__device__ __forceinline__ void clear_rows(const Args &a, int tid, int threads) {
    for (int s = blockIdx.x; s < a.B; s += gridDim.x) {
        const Segment &g = a.segs[s];
        if (g.k1 > g.k0) continue;
        const int64_t n = (int64_t)g.ntok * a.Hq * (D / 8);
        for (int64_t i = tid; i < n; i += threads) {
            const int64_t t = g.t0 + i / (a.Hq * (D / 8)), c = i % (a.Hq * (D / 8));
            *reinterpret_cast<uint4 *>(a.out + t * a.ldo + c * 8) = make_uint4(0, 0, 0, 0);
        }
        if (a.lse)
            for (int64_t i = tid; i < (int64_t)g.ntok * a.Hq; i += threads)
                a.lse[g.t0 * a.Hq + i] = -INFINITY;
    }
}

}  // namespace attn

// The wide kernel's launch (attention_wide.cu); D is 64 or 128.
jet_status launch_attention_wide(const DeviceInfo &dev, const attn::Args &a, int D, cudaStream_t stream);
}  // namespace jet
