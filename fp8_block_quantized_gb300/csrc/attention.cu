// Attention of new tokens' queries over the paged FP8 KV cache.
//
// For the query of token t of request b at position pos, with the request's
// keys p = 0 .. len - 1 behind its block table:
//   x_p = scale ks (q . k_p), p <= pos;  lse = ln sum_p e^x_p,
//   out = vs sum_p e^(x_p - lse) v_p.
// k_p and v_p are E4M3 codes, ks and vs the head's scales.  The keys below a
// group's prefix length are read through its first request's table row, once for
// all of the group's queries.
//
// The work is a list of key tiles: a segment is the own part of a request or
// the prefix of a group, a unit one 16-row tile (rows = (token, query head of
// the KV head's group)) of a segment and one KV head, and a unit's keys come in
// tiles of 128.  Every CTA takes an equal range of the tiles of all units in
// order, so the loads are even whatever the lengths; each stretch of one unit
// in a CTA's range (a piece) ends in a partial result, joined by a second kernel
// in a fixed order.  A unit that one CTA has whole is written at once.
//
// In a tile each of four warps takes 32 keys on its own: a ring of cp.async
// stages (K and V codes, 16 bytes a copy, so any page size and order), scores
// and values by 16-bit tensor core instructions.  E4M3 codes are exact in FP16;
// the queries are brought to FP16 by a power of two a row that puts their
// largest channel at 2^14, so that a channel's rounding is below 2^-38 of that
// (BF16 has eight bits, FP16 eleven: only channels 2^-25 of the largest lose
// any).  Weights e^(x - max) are rounded to FP16 (2^-11 relative, below the output's
// 2^-8 BF16 step); maxima, sums and outputs are in binary32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <mutex>

#include "attention_common.cuh"
#include "jet_common.cuh"
#include "sm100_ptx.cuh"

namespace {

using namespace jet;
using jet::ptx::smem_u32;

using namespace jet::attn;

constexpr int kThreads = 128;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16-byte copy global -> shared, zeros where !ok.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? 16u : 0u)
                 : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a));
    return v;
}

// Shared-memory place of 16-byte chunk c of key row r: the chunks of a 128-byte
// line are permuted so that the reads below touch every bank once.  K is read by
// two rows and four neighbouring chunks at a time, V by four rows of two chunks.
template <int D, bool V>
__device__ __forceinline__ uint32_t place(int r, int c) {
    if (D == 64) {
        const int line = r >> 1;
        return line * 128 + ((((r & 1) * 4 + c) ^ ((line & 3) << 1)) << 4);
    }
    const int s = V ? ((r >> 1) & 3) << 1 : (r & 1) << 2;
    return r * D + ((c ^ s) << 4);
}

template <int D>
struct Cfg {
    static constexpr int kStageBytes = 2 * 32 * D;             // a warp's K and V
    static constexpr int kStages = D == 64 ? 4 : D == 128 ? 3 : 2;
    static constexpr int kWarpBytes = kStages * kStageBytes;
    static constexpr int kQBytes = D > 128 ? kRows * D * 2 : 0;  // query fragments
    static constexpr int kSmem = 4 * kWarpBytes + kQBytes;
    static constexpr int kCtasPerSm = D > 128 ? 1 : 2;
    static_assert(kSmem * kCtasPerSm <= 227 * 1024, "shared memory");
    static_assert(4 * kWarpBytes >= 4 * kRows * D * 4, "the warps' join reuses the ring");
};

// The rows of a segment without keys (only without groups: with them the join
// writes every row).
template <int D>
__device__ void no_keys(const Args &a, const Segment &g) {
    for (int64_t t = g.t0; t < g.t0 + g.ntok; ++t) {
        for (int64_t i = 0; i < (int64_t)a.Hq * D; i += 8)
            *reinterpret_cast<uint4 *>(a.out + t * a.ldo + i) = make_uint4(0, 0, 0, 0);
        for (int h = 0; h < a.Hq && a.lse; ++h) a.lse[t * a.Hq + h] = -INFINITY;
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, Cfg<D>::kCtasPerSm) attention_kernel(const Args a) {
    using C = Cfg<D>;
    constexpr int ST = C::kStages, KS = D / 16, NT = D / 8, H = D / 64;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int64_t sh_pre[kThreads + 1];
    __shared__ uint32_t sh_mask[4][ST];
    __shared__ float sh_m[4][kRows], sh_l[4][kRows];
    griddep_launch_dependents();
    griddep_wait();

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
    const int lo = a.wide_own ? a.B : 0, hi = a.wide_prefix ? a.B : a.B + a.Ng;
    const int per = deal_segments<kThreads>(lo, hi, sh_pre, a.before, a.total, [&](int s) {
        const Segment g = segment(a, s);
        const Narrow n(a, g);
        if (blockIdx.x == 0 && a.Ng == 0 && n.ktiles == 0) no_keys<D>(a, g);
        return n.tiles(a);
    });
    const int64_t total = sh_pre[kThreads];
    const int64_t ctas = min((int64_t)a.narrow_ctas, total);  // none of them without a tile
    if (blockIdx.x >= ctas) return;
    const int64_t x0 = total * blockIdx.x / ctas, x1 = total * (blockIdx.x + 1) / ctas;
    const int stretch = stretch_of<kThreads>(sh_pre, x0);
    int s = lo + stretch * per;
    int64_t at = sh_pre[stretch];  // first tile of segment s
    const uint32_t ring = smem_u32(smem) + warp * C::kWarpBytes;
    uint2 *qs = reinterpret_cast<uint2 *>(smem + 4 * C::kWarpBytes);  // [KS][kRows / 8][32] (D > 128)

    int64_t x = x0;
    while (x < x1) {
        Segment sg = segment(a, s);
        Narrow nw(a, sg);
        while (at + nw.tiles(a) <= x) {
            at += nw.tiles(a);
            sg = segment(a, ++s);
            nw = Narrow(a, sg);
        }
        const int unit = (int)((x - at) / nw.ktiles);
        const int kt0 = (int)((x - at) - (int64_t)unit * nw.ktiles);
        const int kt1 = (int)min((int64_t)nw.ktiles, kt0 + (x1 - x));
        const int h = unit / nw.rtiles, rt = unit - h * nw.rtiles;
        const int64_t nrows = (int64_t)sg.ntok * a.G, row0 = (int64_t)rt * kRows;

        // queries: rows g and g + 8 of the tile, channels 64 i + 16 j .. + 15
        uint32_t qf[D <= 128 ? KS : 1][4];
        float f[2];
        int pos[2];                // a row past the unit's last hides no key
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int64_t rr = row0 + g + 8 * r;
            const bool ok = rr < nrows;
            const int64_t t = sg.t0 + (ok ? rr / a.G : 0);
            const int hq = h * a.G + (ok ? (int)(rr % a.G) : 0);
            const uint16_t *src = a.q + t * a.ldq + (int64_t)hq * D + 16 * j;
            uint4 w[2 * H];
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 2 * H; ++i) {
                w[i] = make_uint4(0, 0, 0, 0);
                if (ok) w[i] = *reinterpret_cast<const uint4 *>(src + 64 * (i >> 1) + 8 * (i & 1));
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[k] << 16)),
                                           fabsf(__uint_as_float(u[k] & 0xFFFF0000u))));
            }
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
            const float up = row_power(top);
            f[r] = a.scale * a.ks[h] * kLog2e / up;
            pos[r] = 0x7FFFFFFF;
            if (ok) pos[r] = position(a, s < a.B ? s : min(upper(a.off, a.B, t), a.B - 1), t);
#pragma unroll
            for (int i = 0; i < 2 * H; ++i) {
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                uint32_t v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[k] = pack_f16(__uint_as_float(u[k] << 16) * up,
                                    __uint_as_float(u[k] & 0xFFFF0000u) * up);
                // step 4 (i / 2) + 2 (i % 2) + {0, 1}: channels 4 at a time
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int ks = 4 * (i >> 1) + 2 * (i & 1) + k;
                    if constexpr (D <= 128) {
                        qf[ks][r] = v[2 * k];
                        qf[ks][2 + r] = v[2 * k + 1];
                    } else if (warp == 0) {
                        qs[(ks * 2 + r) * 32 + lane] = make_uint2(v[2 * k], v[2 * k + 1]);
                    }
                }
            }
        }
        if (D > 128) __syncthreads();
        const bool causal = __any_sync(~0u, min(pos[0], pos[1]) < sg.k1 - 1);

        const int32_t *tab = a.table + (int64_t)sg.row * a.width;
        // this lane's key of tile kt: its cache row, or -1
        auto slot_of = [&](int kt) -> int {
            const int64_t p = (int64_t)sg.k0 + (int64_t)kt * kTile + warp * 32 + lane;
            if (kt >= kt1 || p >= sg.k1) return -1;
            const uint32_t blk = (uint32_t)p / (uint32_t)a.bs;
            const int64_t id = tab[blk];
            if (id < 0) return -1;
            const int64_t slot = id * a.bs + ((uint32_t)p - blk * (uint32_t)a.bs);
            return slot < a.S ? (int)slot : -1;
        };
        auto issue = [&](int kt, int slot) {
            const int st = kt % ST;
            const uint32_t mask = __ballot_sync(~0u, slot >= 0);
            if (lane == 0) sh_mask[warp][st] = mask;
            const uint32_t dst = ring + st * C::kStageBytes;
            if (kt < kt1) {
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    const int idx = i * 32 + lane, key = idx / KS, c = idx % KS;
                    const int sl = __shfl_sync(~0u, slot, key);
                    const int64_t from = ((int64_t)(sl < 0 ? 0 : sl) * a.Hk + h) * D + c * 16;
                    copy16(dst + place<D, false>(key, c), a.kc + from, sl >= 0);
                    copy16(dst + 32 * D + place<D, true>(key, c), a.vc + from, sl >= 0);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };

        float o[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < ST - 1; ++i) issue(kt0 + i, slot_of(kt0 + i));
        int next = slot_of(kt0 + ST - 1);
        for (int kt = kt0; kt < kt1; ++kt) {
            __syncwarp();  // the stage written below has been read by all lanes
            issue(kt + ST - 1, next);
            next = slot_of(kt + ST);
            asm volatile("cp.async.wait_group %0;" ::"n"(ST - 1) : "memory");
            __syncwarp();
            const int st = kt % ST;
            const uint32_t kb = ring + st * C::kStageBytes, vb = kb + 32 * D;
            const uint32_t mask = sh_mask[warp][st];
            if (mask == 0) continue;
            // scores of keys 8 t + 2 j, + 1 for rows g and g + 8
            float sc[4][4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.0f;
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const uint4 w = lds16(kb + place<D, false>(8 * t + g, 4 * i + j));
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int ks = 4 * i + k;
                        if constexpr (D <= 128) {
                            mma16816(sc[t], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3],
                                     codes_f16(u[k]), codes_f16_hi(u[k]));
                        } else {
                            const uint2 lo = qs[(ks * 2) * 32 + lane], hi = qs[(ks * 2 + 1) * 32 + lane];
                            mma16816(sc[t], lo.x, hi.x, lo.y, hi.y, codes_f16(u[k]),
                                     codes_f16_hi(u[k]));
                        }
                    }
                }
            }
            float top[2] = {-INFINITY, -INFINITY};
            // a key of the mask lies below 2^31, and so do its tile's others but for the last few
            const uint32_t p0 = (uint32_t)sg.k0 + (uint32_t)kt * kTile + warp * 32 + 2 * j;
            const bool all = mask == ~0u && !causal;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v = sc[t][e] * f[e >> 1];
                    if (!all) {
                        const int key = 8 * t + 2 * j + (e & 1);
                        if (!((mask >> key) & 1) || (int64_t)(p0 + 8 * t + (e & 1)) > pos[e >> 1])
                            v = -INFINITY;
                    }
                    sc[t][e] = v;
                    top[e >> 1] = fmaxf(top[e >> 1], v);
                }
            float use[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 1));
                top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 2));
                top[r] = fmaxf(top[r], m[r]);
                use[r] = top[r] == -INFINITY ? 0.0f : top[r];
            }
            if (__any_sync(~0u, top[0] != m[0] || top[1] != m[1])) {
                const float c0 = ex2(m[0] - use[0]), c1 = ex2(m[1] - use[1]);
                l[0] *= c0;
                l[1] *= c1;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    o[i][0] *= c0;
                    o[i][1] *= c0;
                    o[i][2] *= c1;
                    o[i][3] *= c1;
                }
                m[0] = top[0];
                m[1] = top[1];
            }
            uint32_t pw[4][2];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float e0 = ex2(sc[t][2 * r] - use[r]), e1 = ex2(sc[t][2 * r + 1] - use[r]);
                    l[r] += e0 + e1;
                    pw[t][r] = pack_f16(e0, e1);
                }
            // values: keys 16 u + {2j, 2j + 1, 2j + 8, 2j + 9}
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t a0 = pw[2 * u][0], a1 = pw[2 * u][1], a2 = pw[2 * u + 1][0],
                               a3 = pw[2 * u + 1][1];
                const int r0 = 16 * u + 2 * j;
                constexpr int HV = D == 256 ? 2 : 1, NW = D == 64 ? 2 : 4;
#pragma unroll
                for (int hv = 0; hv < HV; ++hv) {
                    uint32_t w[4][NW];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = r0 + (k & 1) + 8 * (k >> 1);
                        if constexpr (D == 64) {
                            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                                         : "=r"(w[k][0]), "=r"(w[k][1])
                                         : "r"(vb + place<D, true>(row, g >> 1) + 8 * (g & 1)));
                        } else {
                            const uint4 v = lds16(vb + place<D, true>(row, g + 8 * hv));
                            w[k][0] = v.x;
                            w[k][1] = v.y;
                            w[k][2] = v.z;
                            w[k][3] = v.w;
                        }
                    }
#pragma unroll
                    for (int c = 0; c < NW; ++c) {
                        const uint32_t l0 = __byte_perm(w[0][c], w[1][c], 0x5140),
                                       l1 = __byte_perm(w[0][c], w[1][c], 0x7362),
                                       h0 = __byte_perm(w[2][c], w[3][c], 0x5140),
                                       h1 = __byte_perm(w[2][c], w[3][c], 0x7362);
                        const int n = hv * 16 + c * 4;
                        mma16816(o[n], a0, a1, a2, a3, codes_f16(l0), codes_f16(h0));
                        mma16816(o[n + 1], a0, a1, a2, a3, codes_f16_hi(l0), codes_f16_hi(h0));
                        mma16816(o[n + 2], a0, a1, a2, a3, codes_f16(l1), codes_f16(h1));
                        mma16816(o[n + 3], a0, a1, a2, a3, codes_f16_hi(l1), codes_f16_hi(h1));
                    }
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        // join of the four warps in the ring's memory
        float *red = reinterpret_cast<float *>(smem);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(~0u, l[r], 1);
            l[r] += __shfl_xor_sync(~0u, l[r], 2);
            if (j == 0) {
                sh_m[warp][g + 8 * r] = m[r];
                sh_l[warp][g + 8 * r] = l[r];
            }
            float *dst = red + (warp * kRows + g + 8 * r) * D;
            constexpr int W = D == 64 ? 8 : 16;  // channels of one column of a fragment
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int base = (n / W) * 128 + n % W;
                dst[base + W * (2 * j)] = o[n][2 * r];
                dst[base + W * (2 * j + 1)] = o[n][2 * r + 1];
            }
        }
        __syncthreads();
        {
            const int r = tid >> 3, d0 = (tid & 7) * 4;
            const int64_t rr = row0 + r;
            if (rr < nrows) {
                float top = -INFINITY, wt[4], sum = 0.0f;
#pragma unroll
                for (int w = 0; w < 4; ++w) top = fmaxf(top, sh_m[w][r]);
                const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    wt[w] = ex2(sh_m[w][r] - base);
                    sum += wt[w] * sh_l[w][r];
                }
                const int64_t t = sg.t0 + rr / a.G;
                const int hq = h * a.G + (int)(rr % a.G);
                const bool full = kt1 - kt0 == nw.ktiles, direct = full && a.Ng == 0;
                const int64_t slot =
                    full ? ((s < a.B ? a.T : 0) + t) * a.Hq + hq
                         : (int64_t)(2 * blockIdx.x + (x == x0 ? 0 : 1)) * kRows + r;
                float *po = (full ? a.whole : a.part) + slot * D;
                float *ml = (full ? a.whole_ml : a.part_ml) + slot * 2;
                const float inv = sum > 0.0f ? a.vs[h] / sum : 0.0f;
#pragma unroll
                for (int d = d0; d < D; d += 32) {
                    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const float4 p = *reinterpret_cast<const float4 *>(red + (w * kRows + r) * D + d);
                        v.x += wt[w] * p.x;
                        v.y += wt[w] * p.y;
                        v.z += wt[w] * p.z;
                        v.w += wt[w] * p.w;
                    }
                    if (direct) {
                        const __nv_bfloat162 b0 = __floats2bfloat162_rn(v.x * inv, v.y * inv),
                                             b1 = __floats2bfloat162_rn(v.z * inv, v.w * inv);
                        uint2 w;
                        w.x = *reinterpret_cast<const uint32_t *>(&b0);
                        w.y = *reinterpret_cast<const uint32_t *>(&b1);
                        *reinterpret_cast<uint2 *>(a.out + t * a.ldo + (int64_t)hq * D + d) = w;
                    } else {
                        *reinterpret_cast<float4 *>(po + d) = v;
                    }
                }
                if ((tid & 7) == 0) {
                    if (!direct) {
                        ml[0] = top;
                        ml[1] = sum;
                    } else if (a.lse) {
                        a.lse[t * a.Hq + hq] = sum > 0.0f ? kLn2 * (top + log2f(sum)) : -INFINITY;
                    }
                }
            }
        }
        __syncthreads();
        x += kt1 - kt0;
    }
}

// One row's join: the running maximum, sum and output of a warp (channels lane +
// 32 e).
template <int D>
struct Row {
    static constexpr int E = D / 32;
    float m = -INFINITY, l = 0.0f, o[E] = {};
    // n partial results; piece(i) is the row of the i-th in o and ml
    template <typename F>
    __device__ void add(const float *po, const float *ml, int n, F piece) {
        const int lane = threadIdx.x & 31;
        for (int b = 0; b < n; b += 32) {
            float mi = -INFINITY, li = 0.0f;
            if (b + lane < n) {
                const float2 v = *reinterpret_cast<const float2 *>(ml + 2 * piece(b + lane));
                mi = v.x, li = v.y;
            }
            float top = fmaxf(m, mi);
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
            const float use = top == -INFINITY ? 0.0f : top, c = ex2(m - use), w = ex2(mi - use);
            li *= w;
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) li += __shfl_xor_sync(~0u, li, d);
            l = l * c + li;
            m = top;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] *= c;
            const int cnt = min(32, n - b);
#pragma unroll 4
            for (int i = 0; i < cnt; ++i) {
                const float wi = __shfl_sync(~0u, w, i);
                const float *src = po + piece(b + i) * D + lane;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] += wi * src[32 * e];
            }
        }
    }
    __device__ void write(const Args &a, int64_t t, int hq) const {
        const int lane = threadIdx.x & 31;
        const float inv = l > 0.0f ? a.vs[hq / a.G] / l : 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const __nv_bfloat16 v = __float2bfloat16_rn(o[e] * inv);
            a.out[t * a.ldo + (int64_t)hq * D + lane + 32 * e] = *reinterpret_cast<const uint16_t *>(&v);
        }
        if (a.lse && lane == 0) a.lse[t * a.Hq + hq] = l > 0.0f ? kLn2 * (m + log2f(l)) : -INFINITY;
    }
};

// The pieces of a unit of `n` tiles from u0 on, dealt to several CTAs: CTA c's is
// its first piece (slot 2 c) where its range begins in the unit, else its last.
struct Pieces {
    int c0, n, first;  // CTAs, and the first one's slot
    __device__ Pieces(int64_t u0, int64_t tiles, int64_t total, int64_t ctas) {
        c0 = cta_of(u0, total, ctas);
        n = cta_of(u0 + tiles - 1, total, ctas) - c0 + 1;
        first = 2 * c0 + (total * c0 / ctas >= u0 ? 0 : 1);
    }
    __device__ int64_t slot(int i) const { return i == 0 ? first : 2 * (c0 + i); }
};

// Without groups: the rows of the units that more than one CTA had.  The ranges'
// borders are gone through; a unit is joined at the first border inside it.  A
// CTA takes kJoinRows rows of a border's unit.
constexpr int kJoinRows = 16;

template <int D>
__global__ void __launch_bounds__(256, 4) attention_join_split_kernel(const Args a) {
    griddep_launch_dependents();
    griddep_wait();
    const bool wide = a.wide_own;
    const int rows = wide ? kWideRows : kRows, per = rows / kJoinRows;
    const int border = blockIdx.x / per + 1, r0 = (blockIdx.x % per) * kJoinRows;
    const int64_t total = a.total[wide], ctas = min((int64_t)(wide ? a.wide_ctas : a.narrow_ctas), total);
    if (border >= ctas) return;
    const int64_t x = total * border / ctas;
    int lo = 0, hi = a.B - 1;  // the last segment that begins at or before x (one with tiles)
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.before[mid] <= x) lo = mid; else hi = mid - 1;
    }
    const Segment g = segment(a, lo);
    int64_t u0 = a.before[lo], row0;
    int n, h, count;
    if (wide) {
        const Wide w(a, g);
        int rt = 0;
        while (u0 + (int64_t)w.ktiles(g, rt) * a.Hk <= x) u0 += (int64_t)w.ktiles(g, rt++) * a.Hk;
        n = w.ktiles(g, rt);
        h = (int)((x - u0) / n);
        row0 = (int64_t)rt * w.tokens * a.G;
        count = (int)min((int64_t)w.tokens * a.G, (int64_t)g.ntok * a.G - row0);
        u0 += (int64_t)h * n;
    } else {
        const Narrow w(a, g);
        n = w.ktiles;
        const int unit = (int)((x - u0) / n);
        h = unit / w.rtiles;
        row0 = (int64_t)(unit - h * w.rtiles) * kRows;
        count = (int)min((int64_t)kRows, (int64_t)g.ntok * a.G - row0);
        u0 += (int64_t)unit * n;
    }
    if (u0 == x || total * (border - 1) / ctas > u0) return;
    const Pieces p(u0, n, total, ctas);
    const float *po = wide ? a.wpart : a.part, *ml = wide ? a.wpart_ml : a.part_ml;
    for (int r = r0 + (threadIdx.x >> 5); r < min(count, r0 + kJoinRows); r += 8) {
        Row<D> row;
        row.add(po, ml, p.n, [&](int i) { return p.slot(i) * rows + r; });
        const int64_t rr = row0 + r;
        row.write(a, g.t0 + rr / a.G, h * a.G + (int)(rr % a.G));
    }
}

// With groups: every row, from its prefix and its request's own part.  One warp a
// row.
template <int D>
__global__ void __launch_bounds__(256, 4) attention_join_kernel(const Args a) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t first = clamp64(a.off[0], 0, a.T), last = clamp64(a.off[a.B], 0, a.T);
    for (int64_t i = blockIdx.x * 8ll + (threadIdx.x >> 5); i < a.T * a.Hq; i += gridDim.x * 8ll) {
        const int64_t t = i / a.Hq;
        const int hq = (int)(i - t * a.Hq), h = hq / a.G;
        if (t < first || t >= last) continue;
        const int b = upper(a.off, a.B, t);
        if (b >= a.B) continue;
        Row<D> row;
        for (int k = 0; k < 2; ++k) {
            int s = b;
            if (k == 0) {  // the prefix
                if (b < a.po[0]) continue;
                const int gi = upper(a.po, a.Ng, b);
                if (gi >= a.Ng) continue;
                s = a.B + gi;
            }
            const Segment g = segment(a, s);
            if (g.k1 <= g.k0 || t < g.t0 || t >= g.t0 + g.ntok) continue;
            const bool wide = s < a.B ? a.wide_own : a.wide_prefix;
            const int64_t rr = (t - g.t0) * a.G + hq % a.G;
            int64_t u0 = a.before[s];
            int n, r;
            if (wide) {
                const Wide w(a, g);
                const int rt = (int)((t - g.t0) / w.tokens);
                int64_t skip;
                if (g.base >= 0) {
                    skip = w.head_tiles(g, lane, rt, 32);
#pragma unroll
                    for (int d = 16; d >= 1; d >>= 1) skip += __shfl_xor_sync(~0u, skip, d);
                } else {
                    skip = w.head_tiles(g, 0, rt);
                }
                n = w.ktiles(g, rt);
                u0 += skip * a.Hk + (int64_t)h * n;
                r = (int)(rr - (int64_t)rt * w.tokens * a.G);
            } else {
                const Narrow w(a, g);
                n = w.ktiles;
                u0 += (h * (int64_t)w.rtiles + rr / kRows) * n;
                r = (int)(rr % kRows);
            }
            const int64_t total = a.total[wide], ctas = min((int64_t)(wide ? a.wide_ctas : a.narrow_ctas), total);
            const Pieces p(u0, n, total, ctas);
            if (p.n == 1) {
                const int64_t at = (s < a.B ? a.T * a.Hq : 0) + i;
                row.add(a.whole, a.whole_ml, 1, [&](int) { return at; });
            } else if (wide) {
                row.add(a.wpart, a.wpart_ml, p.n, [&](int j) { return p.slot(j) * kWideRows + r; });
            } else {
                row.add(a.part, a.part_ml, p.n, [&](int j) { return p.slot(j) * kRows + r; });
            }
        }
        row.write(a, t, hq);
    }
}

// Which segments go to the wide kernel, by the rows that a unit has on average:
// requests' own parts and prefixes.
constexpr int64_t kWideFrom = 32;

struct Layout {
    bool wide_own, wide_prefix;
    size_t part, part_ml, wpart, wpart_ml, whole, whole_ml, before, total, bytes;
};

Layout layout(int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t B, int64_t Ng) {
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    const int64_t G = Hq / Hk;
    Layout w;
    const bool can = D <= 128 && G <= 128;
    w.wide_own = can && T * G >= kWideFrom * B;
    w.wide_prefix = can && Ng > 0 && T * G >= kWideFrom * Ng;
    const size_t slots = !w.wide_own || (Ng > 0 && !w.wide_prefix) ? 2 * kNarrowCtas * kRows : 0,
                 wslots = w.wide_own || w.wide_prefix ? 2 * kWideCtas * kWideRows : 0,
                 rows = Ng > 0 ? (size_t)(2 * T * Hq) : 0;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t p = at;
        at += up(n);
        return p;
    };
    w.part = take(slots * D * 4);
    w.part_ml = take(slots * 8);
    w.wpart = take(wslots * D * 4);
    w.wpart_ml = take(wslots * 8);
    w.whole = take(rows * D * 4);
    w.whole_ml = take(rows * 8);
    w.before = take((size_t)(B + Ng) * 8);
    w.total = take(16);
    w.bytes = at;
    return w;
}

bool shape_ok(int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t B, int64_t Ng) {
    if (T < 0 || Hq < 0 || Hk < 0 || B < 0 || Ng < 0) return false;
    if (Hq > 1024 || T >= (int64_t)1 << 24 || B > 8192 || Ng > B) return false;
    if (Hq > 0 && (Hk == 0 || Hq % Hk != 0)) return false;
    return D == 64 || D == 128 || D == 256;
}

template <int D>
jet_status launch(const DeviceInfo &dev, const Args &a, cudaStream_t stream) {
    using C = Cfg<D>;
    {
        // the same limit for every call: attributes are shared by a process's threads
        static std::mutex mu;
        static void *done[64] = {};
        std::lock_guard<std::mutex> lock(mu);
        if (dev.context == nullptr || done[dev.ordinal] != dev.context) {
            if (cudaFuncSetAttribute(attention_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     C::kSmem) != cudaSuccess) {
                cudaGetLastError();
                return JET_ERR_CUDA;
            }
            done[dev.ordinal] = dev.context;
        }
    }
    jet_status st = JET_OK;
    if (!a.wide_own || (a.Ng > 0 && !a.wide_prefix))
        st = launch_pdl(attention_kernel<D>, dim3((unsigned)a.narrow_ctas), dim3(kThreads), C::kSmem,
                        stream, a);
    if (st == JET_OK && (a.wide_own || a.wide_prefix)) st = launch_attention_wide(dev, a, D, stream);
    if (st != JET_OK) return st;
    if (a.Ng > 0) {
        const int64_t want = (a.T * a.Hq + 7) / 8, cap = (int64_t)dev.num_sms * 8;
        return launch_pdl(attention_join_kernel<D>, dim3((unsigned)(want < cap ? want : cap)), dim3(256),
                          0, stream, a);
    }
    const int borders = (a.wide_own ? a.wide_ctas : a.narrow_ctas) - 1;
    const int per = (a.wide_own ? kWideRows : kRows) / kJoinRows;
    if (borders <= 0) return JET_OK;
    return launch_pdl(attention_join_split_kernel<D>, dim3((unsigned)(borders * per)), dim3(256), 0, stream, a);
}

inline bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

size_t jet_kv_attention_workspace(int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t B,
                                  int64_t n_prefix) {
    if (!shape_ok(T, Hq, Hk, D, B, n_prefix) || T == 0 || Hq == 0 || B == 0) return 0;
    return layout(T, Hq, Hk, D, B, n_prefix).bytes;
}

jet_status jet_kv_attention(const uint16_t *q, int64_t ldq, int64_t T, int64_t Hq, int64_t Hk,
                            int64_t D, const uint8_t *k_cache, const uint8_t *v_cache, int64_t S,
                            const float *k_scale, const float *v_scale, const int32_t *table,
                            int64_t width, int64_t block_size, const int64_t *offsets,
                            const int32_t *lengths, int64_t B, const int64_t *prefix_offsets,
                            const int32_t *prefix_lengths, int64_t n_prefix, float scale,
                            uint16_t *out, int64_t ldo, float *lse, void *ws, size_t ws_bytes,
                            jet_stream_t stream) {
    JET_REQUIRE(shape_ok(T, Hq, Hk, D, B, n_prefix), JET_ERR_SHAPE);
    const bool empty = T == 0 || Hq == 0 || B == 0;
    JET_REQUIRE(empty || (q && k_scale && v_scale && offsets && lengths && out), JET_ERR_NULL);
    JET_REQUIRE(S <= 0 || empty || (k_cache && v_cache), JET_ERR_NULL);
    JET_REQUIRE(width <= 0 || empty || table, JET_ERR_NULL);
    JET_REQUIRE(n_prefix == 0 || empty || (prefix_offsets && prefix_lengths), JET_ERR_NULL);
    JET_REQUIRE(S >= 0 && S < (int64_t)1 << 31 && width >= 0 && width < (int64_t)1 << 31 &&
                    block_size >= 1 && block_size < (int64_t)1 << 30,
                JET_ERR_SHAPE);
    JET_REQUIRE(scale > 0.0f && scale < INFINITY, JET_ERR_SHAPE);
    JET_REQUIRE(ldq >= Hq * D && ldo >= Hq * D && ldq < (int64_t)1 << 40 && ldo < (int64_t)1 << 40,
                JET_ERR_SHAPE);
    JET_REQUIRE(ldq % 8 == 0 && ldo % 8 == 0 && aligned16(q) && aligned16(k_cache) &&
                    aligned16(v_cache) && aligned16(out) && aligned16(ws),
                JET_ERR_ALIGN);
    JET_REQUIRE(aligned_to(k_scale, 4) && aligned_to(v_scale, 4) && aligned_to(table, 4) &&
                    aligned_to(offsets, 8) && aligned_to(lengths, 4) &&
                    aligned_to(prefix_offsets, 8) && aligned_to(prefix_lengths, 4) &&
                    aligned_to(lse, 4),
                JET_ERR_ALIGN);
    Layout w = {};
    if (!empty) w = layout(T, Hq, Hk, D, B, n_prefix);
    JET_REQUIRE(empty || (ws && ws_bytes >= w.bytes), JET_ERR_WORKSPACE);
    DeviceInfo dev;
    const jet_status st = current_device(&dev);
    if (st != JET_OK) return st;
    if (empty) return JET_OK;
    Args a;
    a.q = q, a.ldq = ldq, a.T = T, a.Hq = (int)Hq, a.Hk = (int)Hk, a.G = (int)(Hq / Hk);
    a.kc = k_cache, a.vc = v_cache, a.S = S, a.ks = k_scale, a.vs = v_scale;
    a.table = table, a.width = width, a.bs = block_size, a.off = offsets, a.len = lengths;
    a.B = (int)B, a.po = prefix_offsets, a.pl = prefix_lengths, a.Ng = (int)n_prefix;
    a.scale = scale, a.out = out, a.ldo = ldo, a.lse = lse;
    uint8_t *base = static_cast<uint8_t *>(ws);
    a.part = reinterpret_cast<float *>(base + w.part);
    a.part_ml = reinterpret_cast<float *>(base + w.part_ml);
    a.whole = reinterpret_cast<float *>(base + w.whole);
    a.whole_ml = reinterpret_cast<float *>(base + w.whole_ml);
    a.wpart = reinterpret_cast<float *>(base + w.wpart);
    a.wpart_ml = reinterpret_cast<float *>(base + w.wpart_ml);
    a.before = reinterpret_cast<int64_t *>(base + w.before);
    a.total = reinterpret_cast<int64_t *>(base + w.total);
    a.wide_own = w.wide_own, a.wide_prefix = w.wide_prefix;
    const int per_sm = D > 128 ? 1 : 2;  // narrow CTAs on an SM
    a.narrow_ctas = dev.num_sms * per_sm < kNarrowCtas ? dev.num_sms * per_sm : kNarrowCtas;
    a.wide_ctas = dev.num_sms < kWideCtas ? dev.num_sms : kWideCtas;
    const cudaStream_t s = as_stream(stream);
    return D == 64 ? launch<64>(dev, a, s) : D == 128 ? launch<128>(dev, a, s) : launch<256>(dev, a, s);
}
