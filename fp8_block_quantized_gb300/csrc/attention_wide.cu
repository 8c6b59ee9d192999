// Attention over the paged FP8 cache for many rows a KV head: chunks of a prompt,
// and prefixes that a group of requests shares.  The mathematics, the segments
// and the deal of the key tiles are those of attention.cu; here a tile is two
// 128 x 128 score products on the 5th-generation tensor core.
//
// One CTA an SM, 13 warps:
//   warps 0-3, 4-7  two halves (A, B), one thread a row: the row's query to FP16 in
//                   shared memory, then for every tile its scores from TMEM,
//                   maxima, weights e^(x - max) as FP16 back to TMEM over the
//                   scores, and at a piece's end its output;
//   warps 8-11      the tiles' codes: read through the block table a tile ahead
//                   (32 KB in flight), turned to FP16 (exact) and laid out in
//                   shared memory, K and V alike as rows of keys with the 128-byte
//                   swizzle: K-major for the scores, MN-major for the values;
//   warp 12         issues the MMAs: scores S = Q K^T (both operands in shared
//                   memory) and O += P V (P in TMEM).
// In a wide unit A and B are the two halves of 256 rows at the same keys; a unit
// of at most 128 rows has them at alternate tiles of the same rows, whose results
// are added at the end.  While one half's weights are computed the tensor core
// works for the other.  A row's output is rescaled in TMEM only when its maximum
// has grown by more than 2^8 since the last time: weights then reach 2^8 at most,
// within FP16, and are summed in binary32.
//
// Every wait is bounded (jet_common.cuh); a role that gives up sets the CTA's abort
// flag, MMAs in flight are awaited and TMEM is freed.
#include <cuda.h>
#include <cuda_fp16.h>

#include <mutex>

#include "attention_common.cuh"
#include "tcgen05_f16.cuh"

namespace {

using namespace jet;
using namespace jet::attn;
using namespace jet::ptx;

constexpr int kThreads = 416;
constexpr int kStages = 2;
// Wait sites in the status word (after those of head.cu).
constexpr unsigned kSiteLoad = 24, kSiteQuery = 25, kSiteTile = 26, kSiteWeights = 27, kSiteScores = 28,
                   kSiteOutput = 29, kSiteDrain = 30;

template <int D>
struct Cfg {
    static constexpr int kQBytes = 128 * D * 2;
    static constexpr int kKBytes = 128 * D * 2;
    static constexpr int kStageBytes = 2 * kKBytes;
    static constexpr int kUsed = 2 * kQBytes + kStages * kStageBytes + 1024;
    // at least half of an SM's, so that no second CTA waits there for TMEM
    static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

// One stretch of a unit in a CTA's range; the same for all roles.
struct Piece {
    Segment g;
    int s, h, rt;
    int kt0, n;        // first tile (or pair) and their number
    int ktiles;        // of the unit
    bool pairs;        // A and B at alternate tiles
    bool both;         // B takes part
    int64_t row0;      // the unit's first row
    int rows;
    bool first;        // of this CTA
};

struct Walk {
    int64_t x, x0, x1, at;  // tiles: next, the CTA's range, the segment's first
    int s;
    __device__ bool next(const Args &a, Piece &p) {
        if (x >= x1) return false;
        p.g = segment(a, s);
        Wide w(a, p.g);
        int64_t tiles = w.tiles(a, p.g);
        while (at + tiles <= x) {
            at += tiles;
            p.g = segment(a, ++s);
            w = Wide(a, p.g);
            tiles = w.tiles(a, p.g);
        }
        int64_t u = at;
        int rt = 0;
        if (p.g.base < 0) {
            rt = (int)((x - u) / ((int64_t)w.ktiles(p.g, 0) * a.Hk));
            u += (int64_t)rt * w.ktiles(p.g, 0) * a.Hk;
        } else {
            while (u + (int64_t)w.ktiles(p.g, rt) * a.Hk <= x) u += (int64_t)w.ktiles(p.g, rt++) * a.Hk;
        }
        p.s = s;
        p.rt = rt;
        p.ktiles = w.ktiles(p.g, rt);
        p.h = (int)((x - u) / p.ktiles);
        p.kt0 = (int)((x - u) - (int64_t)p.h * p.ktiles);
        p.n = (int)min((int64_t)(p.ktiles - p.kt0), x1 - x);
        p.pairs = w.keys != kTile;
        p.row0 = (int64_t)rt * w.tokens * a.G;
        p.rows = (int)min((int64_t)w.tokens * a.G, (int64_t)p.g.ntok * a.G - p.row0);
        p.both = p.pairs || p.rows > 128;
        p.first = x == x0;
        x += p.n;
        return true;
    }
};

// Without groups nobody else writes the rows of a segment without keys.
template <int D>
__device__ void no_keys(const Args &a, const Segment &g) {
    for (int64_t t = g.t0; t < g.t0 + g.ntok; ++t) {
        for (int64_t i = 0; i < (int64_t)a.Hq * D; i += 8)
            *reinterpret_cast<uint4 *>(a.out + t * a.ldo + i) = make_uint4(0, 0, 0, 0);
        for (int h = 0; h < a.Hq && a.lse; ++h) a.lse[t * a.Hq + h] = -INFINITY;
    }
}

__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}

// Place of 16-byte chunk c (8 FP16 channels) of row r in a [D / 64][128][128 bytes]
// operand with the 128-byte swizzle.
__device__ __forceinline__ uint32_t place(int r, int c) {
    return (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attention_wide_kernel(const Args a, unsigned *status) {
    using C = Cfg<D>;
    extern __shared__ uint8_t dyn[];
    __shared__ int64_t sh_pre[kThreads + 1];
    __shared__ uint64_t q_full, kv_full[kStages], kv_empty[kStages], s_full[2], p_full[2], o_full[2],
        ml_full, drain_bar;
    __shared__ uint32_t sh_mask[kStages][4];
    __shared__ float sh_m[128], sh_l[128];
    __shared__ uint32_t tmem_sh;
    __shared__ int abort_sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t smem = (smem_u32(dyn) + 1023u) & ~1023u;
    volatile int *abort = &abort_sh;

    if (tid == 0) {
        mbar_init(&q_full, 256);
        mbar_init(&ml_full, 128);
        mbar_init(&drain_bar, 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&kv_full[i], 128);
            mbar_init(&kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 128);
            mbar_init(&o_full[i], 1);
        }
        abort_sh = 0;
        fence_mbar_init();
    }
    if (warp == 12) {
        tmem_alloc(&tmem_sh, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_sh;
    griddep_launch_dependents();
    griddep_wait();

    const int lo = a.wide_own ? 0 : a.B, hi = a.wide_prefix ? a.B + a.Ng : a.B;
    const int per = deal_segments<kThreads>(lo, hi, sh_pre, a.before, a.total + 1, [&](int s) {
        const Segment g = segment(a, s);
        if (blockIdx.x == 0 && a.Ng == 0 && g.k1 <= g.k0) no_keys<D>(a, g);
        return Wide(a, g).tiles(a, g);
    });
    const int64_t total = sh_pre[kThreads], ctas = min((int64_t)a.wide_ctas, total);
    Walk walk;
    walk.x = walk.x0 = walk.x1 = walk.at = 0, walk.s = lo;
    if (blockIdx.x < ctas) {
        walk.x = walk.x0 = total * blockIdx.x / ctas;
        walk.x1 = total * (blockIdx.x + 1) / ctas;
        const int stretch = stretch_of<kThreads>(sh_pre, walk.x);
        walk.s = lo + stretch * per;
        walk.at = sh_pre[stretch];
    }
    // A wait of a whole warp for the n-th phase of a barrier; all lanes leave alike.
    auto wait = [&](uint64_t *bar, uint32_t n, unsigned site) -> bool {
        return __all_sync(~0u, mbar_wait(bar, n & 1u, abort, status, site));
    };
    const uint32_t q_s = smem, kv_s = smem + 2 * C::kQBytes;
    Piece p;

    if (warp >= 8 && warp < 12) {
        // ------------------------------------------------------------- codes
        constexpr int CH = D / 16;          // 16-byte chunks of a key's codes
        constexpr int RW = 32 / CH;         // rows a warp reads at once
        constexpr int NI = 32 / RW;
        const int w = warp - 8;
        uint32_t n = 0;                     // tiles so far
        bool ok = true;
        while (ok && walk.next(a, p)) {
            const int tiles = p.n * (p.pairs ? 2 : 1), t0 = p.kt0 * (p.pairs ? 2 : 1);
            const int32_t *tab = a.table + (int64_t)p.g.row * a.width;
            // the cache row of key 32 w + lane of tile kt, or -1
            auto slot_of = [&](int i) -> int {
                const int64_t at = (int64_t)p.g.k0 + (int64_t)(t0 + i) * kTile + 32 * w + lane;
                if (i >= tiles || at >= p.g.k1) return -1;
                const uint32_t blk = (uint32_t)at / (uint32_t)a.bs;
                const int64_t id = tab[blk];
                if (id < 0) return -1;
                const int64_t slot = id * a.bs + ((uint32_t)at - blk * (uint32_t)a.bs);
                return slot < a.S ? (int)slot : -1;
            };
            uint4 kr[NI], vr[NI];
            const int c = lane % CH, rq = lane / CH;
            auto load = [&](int slot) {
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int sl = __shfl_sync(~0u, slot, RW * i + rq);
                    kr[i] = vr[i] = make_uint4(0, 0, 0, 0);
                    if (sl >= 0) {
                        const int64_t from = ((int64_t)sl * a.Hk + p.h) * D + c * 16;
                        kr[i] = *reinterpret_cast<const uint4 *>(a.kc + from);
                        vr[i] = *reinterpret_cast<const uint4 *>(a.vc + from);
                    }
                }
            };
            auto store = [&](uint32_t dst, const uint4 (&v)[NI]) {
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int r = 32 * w + RW * i + rq;
                    uint32_t lo8[4] = {codes_f16(v[i].x), codes_f16_hi(v[i].x), codes_f16(v[i].y),
                                       codes_f16_hi(v[i].y)};
                    uint32_t hi8[4] = {codes_f16(v[i].z), codes_f16_hi(v[i].z), codes_f16(v[i].w),
                                       codes_f16_hi(v[i].w)};
                    // chunks 2 c and 2 c + 1; the lanes of the upper half of a row (and of odd
                    // rows where a row has four chunks) write the odd one first, so that
                    // eight lanes touch every bank once
                    const bool swap = D == 128 ? c >= 4 : (rq & 1);
                    const uint32_t e = dst + place(r, 2 * c), o = dst + place(r, 2 * c + 1);
                    if (!swap) {
                        sts16(e, lo8[0], lo8[1], lo8[2], lo8[3]);
                        sts16(o, hi8[0], hi8[1], hi8[2], hi8[3]);
                    } else {
                        sts16(o, hi8[0], hi8[1], hi8[2], hi8[3]);
                        sts16(e, lo8[0], lo8[1], lo8[2], lo8[3]);
                    }
                }
            };
            int cur = slot_of(0);
            load(cur);
            int nxt = slot_of(1);
            for (int i = 0; i < tiles; ++i, ++n) {
                const int st = n % kStages;
                if (!wait(&kv_empty[st], n / kStages + 1, kSiteLoad)) {
                    ok = false;
                    break;
                }
                const uint32_t mask = __ballot_sync(~0u, cur >= 0);
                if (lane == 0) sh_mask[st][w] = mask;
                const uint32_t dst = kv_s + st * C::kStageBytes;
                store(dst, kr);
                store(dst + C::kKBytes, vr);
                fence_proxy_async();
                mbar_arrive(&kv_full[st]);
                cur = nxt;
                if (i + 1 < tiles) load(cur);
                nxt = slot_of(i + 2);
            }
        }
    } else if (warp == 12) {
        // -------------------------------------------------------------- MMAs
        constexpr uint32_t kS = idesc_16bit(128, 128, false, false, false);
        constexpr uint32_t kO = idesc_16bit(128, D, false, false, true);
        uint32_t n = 0, piece = 0, np[2] = {0, 0};  // tiles, pieces, weights so far
        bool ok = true;
        while (ok && walk.next(a, p)) {
            if (!wait(&q_full, piece, kSiteQuery)) break;
            ++piece;
            const int each = p.pairs ? 2 : 1;
            // scores of half hf in its i-th tile
            auto scores = [&](int hf, int i) -> bool {
                const uint32_t t = n + i * each + (p.pairs ? hf : 0), st = t % kStages;
                if (!wait(&kv_full[st], t / kStages, kSiteTile)) return false;
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t qa = q_s + (p.pairs ? 0 : hf) * C::kQBytes;
                    const uint32_t kb = kv_s + st * C::kStageBytes;
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t o = (ks >> 2) * 16384 + (ks & 3) * 32;
                        mma_16bit(tmem + hf * 128, smem_desc(qa + o, 16, 1024, kSwizzle128B),
                                  smem_desc(kb + o, 16, 1024, kSwizzle128B), kS, ks > 0);
                    }
                    mma_commit(&s_full[hf]);
                }
                __syncwarp();
                return true;
            };
            const int halves = p.both ? 2 : 1;
            for (int hf = 0; ok && hf < halves; ++hf) ok = scores(hf, 0);
            for (int i = 0; ok && i < p.n; ++i) {
                for (int hf = 0; ok && hf < halves; ++hf) {
                    if (!wait(&p_full[hf], np[hf], kSiteWeights)) {
                        ok = false;
                        break;
                    }
                    ++np[hf];
                    tc_fence_after();
                    const uint32_t t = n + i * each + (p.pairs ? hf : 0), st = t % kStages;
                    if (lane == 0) {
                        const uint32_t vb = kv_s + st * C::kStageBytes + C::kKBytes;
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            mma_16bit_ta(tmem + 256 + hf * D, tmem + hf * 128 + 64 + ks * 8,
                                         smem_desc(vb + ks * 2048, 16384, 1024, kSwizzle128B), kO,
                                         i > 0 || ks > 0);
                        if (p.pairs || hf == halves - 1) mma_commit(&kv_empty[st]);
                        if (i + 1 == p.n) mma_commit(&o_full[hf]);
                    }
                    __syncwarp();
                    if (i + 1 < p.n) ok = scores(hf, i + 1);
                }
            }
            n += p.n * each;
        }
        if (lane == 0) mma_commit(&drain_bar);
        __syncwarp();
        mbar_wait(&drain_bar, 0, nullptr, status, kSiteDrain);
    } else if (warp < 8) {
        // ----------------------------------------------- weights and outputs
        const int hf = warp >> 2, r = tid & 127;  // half, its row = TMEM lane
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_t = lanes + hf * 128, o_t = lanes + 256 + hf * D;
        uint32_t n = 0, nt = 0, no[2] = {0, 0}, nml = 0;  // tiles, scores, outputs, merges so far
        bool ok = true;
        while (ok && walk.next(a, p)) {
            // the query
            const int64_t lr = r + (p.pairs ? 0 : 128 * hf);
            const bool row_ok = lr < p.rows;
            const int64_t rr = p.row0 + (row_ok ? lr : 0);
            const int64_t t = p.g.t0 + rr / a.G;
            const int hq = p.h * a.G + (int)(rr % a.G);
            const uint4 *src = reinterpret_cast<const uint4 *>(a.q + t * a.ldq + (int64_t)hq * D);
            float top = 0.0f;
            if (row_ok) {
#pragma unroll 4
                for (int i = 0; i < D / 8; ++i) {
                    const uint4 v = src[i];
                    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[k] << 16)),
                                               fabsf(__uint_as_float(u[k] & 0xFFFF0000u))));
                }
            }
            float up = row_power(top);
            float f = a.scale * a.ks[p.h] * kLog2e / up;
            if (f < 0.0f) f = -f, up = -up;  // maxima are of the raw scores
            f = fmaxf(f, 0x1p-126f);
            int pos = 0x7FFFFFFF;  // a row past the unit's last hides no key
            if (row_ok) pos = position(a, p.s < a.B ? p.s : min(upper(a.off, a.B, t), a.B - 1), t);
            if (!p.pairs || hf == 0) {
                const uint32_t dst = q_s + hf * C::kQBytes;
#pragma unroll 4
                for (int i = 0; i < D / 8; ++i) {
                    const uint4 v = row_ok ? src[i] : make_uint4(0, 0, 0, 0);
                    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = pack_f16(__uint_as_float(u[k] << 16) * up,
                                        __uint_as_float(u[k] & 0xFFFF0000u) * up);
                    sts16(dst + place(r, i), w[0], w[1], w[2], w[3]);
                }
                fence_proxy_async();
            }
            tc_fence_before();  // the last piece's reads of TMEM
            mbar_arrive(&q_full);
            const int each = p.pairs ? 2 : 1;
            if (hf == 1 && !p.both && !wait(&q_full, no[0], kSiteQuery)) break;  // its next arrival is the next piece's
            float m = -INFINITY, l = 0.0f;  // reference of the weights (a power of two), their sum
            const bool active = hf == 0 || p.both;
            for (int i = 0; active && i < p.n; ++i) {
                const int kt = each * (p.kt0 + i) + (p.pairs ? hf : 0);
                const uint32_t seq = n + i * each + (p.pairs ? hf : 0), st = seq % kStages;
                if (!wait(&s_full[hf], nt, kSiteScores) ||
                    !wait(&kv_full[st], seq / kStages, kSiteScores)) {
                    ok = false;
                    break;
                }
                ++nt;
                __syncwarp();
                tc_fence_after();
                // the keys that the row sees, where some are hidden
                uint32_t see[4];
                bool all = true;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int64_t left = pos - ((int64_t)p.g.k0 + (int64_t)kt * kTile + 32 * c);
                    see[c] = sh_mask[st][c];
                    if (left < 31) see[c] &= left < 0 ? 0u : (2u << (int)left) - 1u;
                    all = all && see[c] == ~0u;
                }
                const bool hidden = __any_sync(~0u, !all);
                auto hide = [&](uint32_t (&v)[32], uint32_t bits, float with) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (!((bits >> k) & 1u)) v[k] = __float_as_uint(with);
                };
                uint32_t v0[32], v1[32];
                float top0 = -INFINITY, top1 = -INFINITY;
                auto largest = [&](uint32_t (&v)[32]) {
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        top0 = fmaxf(top0, fmaxf(__uint_as_float(v[k]), __uint_as_float(v[k + 1])));
                        top1 = fmaxf(top1, fmaxf(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])));
                    }
                };
                tmem_ld32(s_t, v0);
                tmem_ld32(s_t + 32, v1);
                tmem_wait32(v0);
                tmem_wait32(v1);
                if (hidden) hide(v0, see[0], -INFINITY), hide(v1, see[1], -INFINITY);
                largest(v0);
                largest(v1);
                __syncwarp();
                tmem_ld32(s_t + 64, v0);
                tmem_ld32(s_t + 96, v1);
                tmem_wait32(v0);
                tmem_wait32(v1);
                if (hidden) hide(v0, see[2], -INFINITY), hide(v1, see[3], -INFINITY);
                largest(v0);
                largest(v1);
                const float tile = fmaxf(top0, top1) * f;
                const bool grown = i > 0 && tile > m + 8.0f;
                if (i == 0) m = tile;
                if (__any_sync(~0u, grown)) {
                    const float c = grown ? ex2(m - tile) : 1.0f;
                    if (grown) m = tile;
                    l *= c;
#pragma unroll 1
                    for (int ch = 0; ch < D / 16; ++ch) {
                        uint32_t o[16];
                        tmem_ld16(o_t + ch * 16, o);
                        tmem_ld_wait(o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * c);
                        tmem_st16(o_t + ch * 16, o);
                    }
                }
                __syncwarp();
                const float2 f2 = make_float2(f, f);
                const float nm = m == -INFINITY ? 0.0f : -m;
                const float2 nm2 = make_float2(nm, nm);
                float2 s0 = make_float2(0.0f, 0.0f), s1 = s0;
                // weights of 32 keys, to 16 columns over the upper half of the scores
                auto weigh = [&](uint32_t (&v)[32], uint32_t bits, int col) {
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float2 x = __ffma2_rn(
                            make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), f2, nm2);
                        float2 e = make_float2(ex2(x.x), ex2(x.y));
                        if (hidden) {
                            if (!((bits >> (2 * k)) & 1u)) e.x = 0.0f;
                            if (!((bits >> (2 * k + 1)) & 1u)) e.y = 0.0f;
                        }
                        if (k & 1) s1 = __fadd2_rn(s1, e); else s0 = __fadd2_rn(s0, e);
                        w[k] = pack_f16(e.x, e.y);
                    }
                    __syncwarp();
                    tmem_st16(s_t + 64 + col, w);
                };
                weigh(v0, see[2], 32);
                tmem_ld32(s_t, v0);
                weigh(v1, see[3], 48);
                tmem_ld32(s_t + 32, v1);
                tmem_wait32(v0);
                weigh(v0, see[0], 0);
                tmem_wait32(v1);
                weigh(v1, see[1], 16);
                l += (s0.x + s0.y) + (s1.x + s1.y);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&p_full[hf]);
            }
            n += p.n * each;
            if (!ok) break;
            // the output
            if (active) {
                if (!wait(&o_full[hf], no[hf], kSiteOutput)) break;
                if (p.pairs && hf == 1) {
                    sh_m[r] = m;
                    sh_l[r] = l;
                    mbar_arrive(&ml_full);
                } else {
                    float ca = 1.0f, cb = 0.0f;
                    if (p.pairs) {
                        if (!wait(&o_full[1], no[1], kSiteOutput) ||
                            !wait(&ml_full, nml, kSiteOutput))
                            break;
                        const float mb = sh_m[r], both = fmaxf(m, mb), use = both == -INFINITY ? 0.0f : both;
                        ca = ex2(m - use);
                        cb = ex2(mb - use);
                        l = l * ca + sh_l[r] * cb;
                        m = both;
                    }
                    __syncwarp();
                    tc_fence_after();
                    const bool full = p.n == p.ktiles, direct = full && a.Ng == 0;
                    const int64_t slot = full ? ((p.s < a.B ? a.T : 0) + t) * a.Hq + hq
                                              : (int64_t)(2 * blockIdx.x + (p.first ? 0 : 1)) * kWideRows + lr;
                    float *po = (full ? a.whole : a.wpart) + slot * D;
                    const float inv = l > 0.0f ? a.vs[p.h] / l : 0.0f;
                    uint16_t *out = a.out + t * a.ldo + (int64_t)hq * D;
#pragma unroll 1
                    for (int ch = 0; ch < D / 32; ++ch) {
                        uint32_t v[32];
                        __syncwarp();
                        tmem_ld32(o_t + ch * 32, v);
                        tmem_wait32(v);
                        if (p.pairs) {
                            uint32_t w[32];
                            tmem_ld32(o_t + D + ch * 32, w);
                            tmem_wait32(w);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                v[k] = __float_as_uint(ca * __uint_as_float(v[k]) + cb * __uint_as_float(w[k]));
                        }
                        if (!row_ok) continue;
                        if (direct) {
#pragma unroll
                            for (int k = 0; k < 32; k += 8) {
                                uint32_t w[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const __nv_bfloat162 b = __floats2bfloat162_rn(
                                        __uint_as_float(v[k + 2 * e]) * inv, __uint_as_float(v[k + 2 * e + 1]) * inv);
                                    w[e] = *reinterpret_cast<const uint32_t *>(&b);
                                }
                                *reinterpret_cast<uint4 *>(out + ch * 32 + k) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < 32; k += 4)
                                *reinterpret_cast<uint4 *>(po + ch * 32 + k) =
                                    make_uint4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                        }
                    }
                    if (row_ok) {
                        if (!direct) {
                            float *ml = (full ? a.whole_ml : a.wpart_ml) + slot * 2;
                            ml[0] = m;
                            ml[1] = l;
                        } else if (a.lse) {
                            a.lse[t * a.Hq + hq] = l > 0.0f ? kLn2 * (m + log2f(l)) : -INFINITY;
                        }
                    }
                }
            }
            ++no[0];
            if (p.both) ++no[1];
            if (p.pairs) ++nml;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D>
jet_status launch(const DeviceInfo &dev, const Args &a, cudaStream_t stream) {
    {
        // the same limit for every call: attributes are shared by a process's threads
        static std::mutex mu;
        static void *done[64] = {};
        std::lock_guard<std::mutex> lock(mu);
        if (dev.context == nullptr || done[dev.ordinal] != dev.context) {
            if (cudaFuncSetAttribute(attention_wide_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     Cfg<D>::kSmem) != cudaSuccess) {
                cudaGetLastError();
                return JET_ERR_CUDA;
            }
            done[dev.ordinal] = dev.context;
        }
    }
    return launch_pdl(attention_wide_kernel<D>, dim3((unsigned)a.wide_ctas), dim3(kThreads), Cfg<D>::kSmem,
                      stream, a, dev.status_word);
}

}  // namespace

namespace jet {
jet_status launch_attention_wide(const DeviceInfo &dev, const attn::Args &a, int D, cudaStream_t stream) {
    return D == 64 ? launch<64>(dev, a, stream) : launch<128>(dev, a, stream);
}
}  // namespace jet
