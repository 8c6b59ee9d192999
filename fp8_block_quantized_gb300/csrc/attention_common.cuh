// What the attention kernels share: the call's arguments, the segments that a
// call is made of, and how each kernel cuts them into units and key tiles.
#pragma once

#include <cuda_bf16.h>

#include "jet_common.cuh"

namespace jet {
namespace attn {

constexpr int kTile = 128;         // keys of a tile
constexpr int kRows = 16;          // rows of a narrow unit
constexpr int kNarrowCtas = 320;   // most CTAs of the narrow kernel (two on each SM)
constexpr int kWideRows = 256;     // rows of a wide unit's pieces
constexpr int kWideCtas = 160;     // most CTAs of the wide kernel (one on each SM)
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
    int narrow_ctas, wide_ctas;    // CTAs of each launch
    // Workspace.  Pieces of units that several CTAs share, two a CTA (narrow:
    // kRows rows each, wide: kWideRows); with groups, whole units by row (prefix,
    // then own); the tiles of the same kernel before each segment, and their totals
    // (narrow, wide).
    float *part, *part_ml, *wpart, *wpart_ml;
    float *whole, *whole_ml;       // [2][T * Hq][D], [..][2]
    int64_t *before, *total;       // [B + Ng], [2]
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
    int ntok;
    int k0, k1;        // keys
    int row;           // table row
    int base;          // own part: the first new token's position, if its queries see k0 and
                       // the last one's position is k1 - 1; else -1
};

__device__ inline Segment segment(const Args &a, int s) {
    Segment g;
    int64_t r0, r1;
    g.base = -1;
    g.k0 = 0;
    if (s < a.B) {
        r0 = s;
        r1 = s + 1;
        g.row = s;
        g.k1 = keys_of(a, s);
        if (a.Ng > 0 && s >= a.po[0]) {
            const int i = upper(a.po, a.Ng, s);
            if (i < a.Ng) g.k0 = min(prefix_of(a, i), g.k1);
        }
    } else {
        const int i = s - a.B;
        r0 = clamp64(a.po[i], 0, a.B);
        r1 = clamp64(a.po[i + 1], r0, a.B);
        g.row = (int)r0;
        g.k1 = r1 > r0 ? prefix_of(a, i) : 0;
    }
    const int64_t o0 = a.off[r0], o1 = a.off[r1];
    const int64_t t0 = clamp64(o0, 0, a.T), t1 = clamp64(o1, t0, a.T);
    g.t0 = t0;
    g.ntok = (int)(t1 - t0);
    if (s < a.B && o0 == t0 && o1 == t1 && g.k1 == a.len[s] && g.k1 - g.ntok >= g.k0)
        g.base = g.k1 - g.ntok;
    return g;
}

// Position of token t of request b.
__device__ __forceinline__ int position(const Args &a, int b, int64_t t) {
    return (int)clamp64((int64_t)a.len[b] - (a.off[b + 1] - t), -1, 0x7FFFFFFF);
}

// Narrow units: 16 rows, a row tile of one KV head; all tiles of a head's row
// tiles one after another.
struct Narrow {
    int rtiles, ktiles;
    __device__ Narrow(const Args &a, const Segment &g) {
        rtiles = (int)(((int64_t)g.ntok * a.G + kRows - 1) / kRows);
        ktiles = (int)(((int64_t)g.k1 - g.k0 + kTile - 1) / kTile);
    }
    __device__ int64_t tiles(const Args &a) const { return (int64_t)rtiles * ktiles * a.Hk; }
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

// The CTA that has tile x when `total` tiles are dealt to `ctas` CTAs in equal
// ranges (CTA c: from total c / ctas on).
__device__ __forceinline__ int cta_of(int64_t x, int64_t total, int64_t ctas) {
    return (int)(((x + 1) * ctas - 1) / total);
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

// The power of two that brings a row's largest channel to [2^14, 2^15).
__device__ __forceinline__ float row_power(float top) {
    const int e = min(254, 268 - (int)(__float_as_uint(top) >> 23));
    return top == 0.0f ? 1.0f : __uint_as_float((uint32_t)max(e, 1) << 23);
}

// The tiles before each of a CTA's threads' stretches of the segments [s0, s1),
// in pre[0 .. N] (shared memory); CTA 0 leaves those before each segment and the
// total in the workspace.  tiles(s) is the segment's.  Returns the stretch.
template <int N, typename F>
__device__ int deal_segments(int s0, int s1, int64_t *pre, int64_t *before, int64_t *total, F tiles) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (s1 - s0 + N - 1) / N;
    const int b = min(s1, s0 + tid * per), e = min(s1, b + per);
    int64_t mine = 0;
    for (int s = b; s < e; ++s) mine += tiles(s);
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t v = __shfl_up_sync(~0u, incl, d);
        if (lane >= d) incl += v;
    }
    if (lane == 31) pre[warp] = incl;
    __syncthreads();
    int64_t at = 0;
    for (int w = 0; w < warp; ++w) at += pre[w];
    __syncthreads();
    pre[tid + 1] = at + incl;
    if (tid == 0) pre[0] = 0;
    __syncthreads();
    if (blockIdx.x == 0) {
        at += incl - mine;
        for (int s = b; s < e; ++s) {
            before[s] = at;
            at += tiles(s);
        }
        if (tid == 0) *total = pre[N];
    }
    return per;
}

// The last of the N stretches that begins at or before tile x.
template <int N>
__device__ __forceinline__ int stretch_of(const int64_t *pre, int64_t x) {
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

}  // namespace attn

// The wide kernel's launch (attention_wide.cu); D is 64 or 128.
jet_status launch_attention_wide(const DeviceInfo &dev, const attn::Args &a, int D, cudaStream_t stream);
}  // namespace jet
