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
// the prefix of a group, a unit one 8-row tile (rows = (token, query head of
// the KV head's group)) of a segment and one KV head, and a unit's keys come in
// tiles of 32.  Every worker takes an equal range of the tiles of all units in
// order, so the loads are even whatever the lengths; each stretch of one unit
// in a worker's range (a piece) ends in a partial result, joined by a last kernel
// in a fixed order.  A unit that one worker has whole is written at once.  The
// first kernel, one CTA, lists the segments with work and where each worker's
// range begins, so that the others find it with two reads.
//
// A narrow worker is up to eight warps, one for each of as many KV heads: they read the
// same tokens, whose heads lie side by side in memory, at about the same time (with
// a head's units one after another the rows of 128 bytes a kilobyte apart came at
// half the rate).  A CTA has as many workers as its warps allow.  A warp has its own ring of
// cp.async stages (K and V codes, 16 bytes a copy, so any page size and order);
// scores and values by 16-bit tensor core instructions.  E4M3 codes are exact in FP16;
// the queries are brought to FP16 by a power of two a row that puts their
// largest channel at 2^14, so that a channel's rounding is below 2^-38 of that
// (BF16 has eight bits, FP16 eleven: only channels 2^-25 of the largest lose
// any).  Weights e^(x - max) times 2^15 are rounded to FP16: 2^-11 relative (below the output's
// 2^-8 BF16 step) down to 2^-29 of a piece's largest, 2^-40 of it below; maxima, sums and outputs
// are in binary32, and the 2^15 is taken out at a piece's end.
//
// What bounds it: the read of the cache.  64 requests of 17 to 8192 tokens, 32 query and
// 8 KV heads of 128 channels: 538 MB in 91 us (5.9 TB/s; a copy runs at 6.8), 100 us with
// the plan and the join; two requests of 100000 to 131072 tokens with 64 query heads: 449
// MB in 77, with both 86.  A single request of 4001 tokens, 17 us, is three launches of
// dependent loads.
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

// The plan: every segment, the tiles before it in its kernel's list (narrow, wide),
// the lists without the segments that have none, and the workers' starts.
constexpr int kPlanThreads = 1024;
constexpr int kPlanHeld = 1024;  // groups, and segments of a list, that fit its shared memory

__global__ void __launch_bounds__(kPlanThreads) attention_plan_kernel(const Args a) {
    __shared__ int64_t sh_po[kPlanHeld + 1];
    __shared__ int64_t sh_before[2][kPlanHeld];
    __shared__ int64_t sh_tiles[2][kPlanThreads / 32];
    __shared__ int sh_count[2][kPlanThreads / 32];
    __shared__ int sh_empty;
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nseg = a.B + a.Ng;
    const bool held = a.Ng <= kPlanHeld;
    if (held && a.Ng > 0)
        for (int i = tid; i <= a.Ng; i += kPlanThreads) sh_po[i] = a.po[i];
    if (tid == 0) sh_empty = 0;
    __syncthreads();
    const int64_t *po = held ? sh_po : a.po;
    int64_t tiles0[2] = {0, 0};  // before the segments of this pass
    int count0[2] = {0, 0};
    int *order[2] = {a.order, a.order + nseg};
    for (int s0 = 0; s0 < nseg; s0 += kPlanThreads) {
        const int s = s0 + tid;
        int64_t mine[2] = {0, 0};
        Segment g;
        bool wide = false;
        if (s < nseg) {
            int64_t r0, r1;
            g.base = g.group = -1;
            g.k0 = 0;
            if (s < a.B) {
                r0 = s;
                r1 = s + 1;
                g.row = s;
                g.k1 = keys_of(a, s);
                if (a.Ng > 0 && s >= po[0]) {
                    const int i = upper(po, a.Ng, s);
                    if (i < a.Ng) g.group = i, g.k0 = min(prefix_of(a, i), g.k1);
                }
            } else {
                const int i = s - a.B;
                r0 = clamp64(po[i], 0, a.B);
                r1 = clamp64(po[i + 1], r0, a.B);
                g.row = (int)r0;
                g.k1 = r1 > r0 ? prefix_of(a, i) : 0;
            }
            g.r0 = (int)r0, g.r1 = (int)r1;
            const int64_t o0 = a.off[r0], o1 = a.off[r1];
            const int64_t t0 = clamp64(o0, 0, a.T), t1 = clamp64(o1, t0, a.T);
            g.t0 = t0;
            g.ntok = (int)(t1 - t0);
            if (s < a.B && o0 == t0 && o1 == t1 && g.k1 == a.len[s] && g.k1 - g.ntok >= g.k0)
                g.base = g.k1 - g.ntok;
            wide = s < a.B ? a.wide_own : a.wide_prefix;
            mine[wide] = wide ? Wide(a, g).tiles(a, g) : Narrow(a, g).tiles();
            if (g.ntok > 0 && g.k1 <= g.k0) atomicAdd(&sh_empty, 1);
        }
        int64_t incl[2];
        int cnt[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            incl[w] = mine[w];
            cnt[w] = mine[w] > 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t v = __shfl_up_sync(~0u, incl[w], d);
                const int c = __shfl_up_sync(~0u, cnt[w], d);
                if (lane >= d) incl[w] += v, cnt[w] += c;
            }
            if (lane == 31) sh_tiles[w][warp] = incl[w], sh_count[w][warp] = cnt[w];
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            // the warps' sums, scanned by every warp for itself
            int64_t v = sh_tiles[w][lane];
            int c = sh_count[w][lane];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t v1 = __shfl_up_sync(~0u, v, d);
                const int c1 = __shfl_up_sync(~0u, c, d);
                if (lane >= d) v += v1, c += c1;
            }
            const int64_t vb = __shfl_sync(~0u, v, warp > 0 ? warp - 1 : 0);
            const int cb = __shfl_sync(~0u, c, warp > 0 ? warp - 1 : 0);
            const int64_t before = tiles0[w] + (warp > 0 ? vb : 0);
            const int at = count0[w] + (warp > 0 ? cb : 0);
            tiles0[w] += __shfl_sync(~0u, v, 31);
            count0[w] += __shfl_sync(~0u, c, 31);
            if (s < nseg && wide == (w == 1)) g.before = before + incl[w] - mine[w];
            if (mine[w] > 0) {
                order[w][at + cnt[w] - 1] = s;
                if (at + cnt[w] <= kPlanHeld) sh_before[w][at + cnt[w] - 1] = before + incl[w] - mine[w];
            }
        }
        if (s < nseg) a.segs[s] = g;
        __syncthreads();
    }
    int workers[2];
    workers[0] = (int)min(tiles0[0], (int64_t)a.ctas * a.phases);
    workers[1] = (int)min(tiles0[1], (int64_t)a.ctas);
    if (tid == 0) {
        Plan p;
        p.total[0] = tiles0[0], p.total[1] = tiles0[1];
        p.workers[0] = workers[0], p.workers[1] = workers[1];
        p.empty = sh_empty;
        p.splits = p.many = 0;
        *a.plan = p;
    }
    __threadfence_block();  // the segments written above, before other threads read them
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int all = w == 0 ? a.ctas * a.phases : a.ctas;
        for (int c = tid; c < all; c += kPlanThreads) {
            Start &st = a.starts[w * kNarrowWorkers + c];
            st.empty = sh_empty;
            st.left = 0;
            if (c >= workers[w]) continue;
            const int64_t x = tiles0[w] * c / workers[w];
            int lo = 0, hi = count0[w] - 1;  // the last listed segment that begins at or before x
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if ((mid < kPlanHeld ? sh_before[w][mid] : a.segs[order[w][mid]].before) <= x) lo = mid;
                else hi = mid - 1;
            }
            st.at = lo;
            st.s = order[w][lo];
            st.g = a.segs[st.s];
            st.left = tiles0[w] * (c + 1) / workers[w] - x;
            st.from = x - st.g.before;
        }
    }
}

template <int D>
struct Cfg {
    static constexpr int kWarps = D > 128 ? 6 : kNarrowWarps;  // of a CTA
    static constexpr int kStageBytes = 2 * kStep * D;          // a warp's K and V
    static constexpr int kStages = D == 64 ? 5 : D == 128 ? 3 : 2;
    static constexpr int kWarpBytes = kStages * kStageBytes;
    static constexpr int kSmem = kWarps * kWarpBytes;
    static_assert(kSmem <= 227 * 1024, "shared memory");
};
constexpr float kUp = 0x1p15f;  // of a weight in FP16, whose normal range ends at 2^-14

template <int D>
__global__ void __launch_bounds__(32 * Cfg<D>::kWarps, 1) attention_kernel(const Args a) {
    using C = Cfg<D>;
    constexpr int ST = C::kStages, KS = D / 16, NT = D / 8, H = D / 64;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint32_t sh_mask[C::kWarps][ST];
    griddep_launch_dependents();
    griddep_wait();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
    // this warp's worker, and its head among the worker's
    const int me = blockIdx.x * a.phases + warp / a.heads, hw = warp % a.heads;
    if (warp >= a.phases * a.heads) return;
    const Start start = a.starts[me];
    if (a.Ng == 0 && start.empty > 0) clear_rows<D>(a, warp * 32 + lane, a.phases * a.heads * 32);
    int64_t left = start.left, from = start.from;  // tiles of the range; the next, in its segment
    int at = start.at, s = start.s;
    Segment sg = start.g;
    bool first = true;
    const uint32_t ring = smem_u32(smem) + warp * C::kWarpBytes;

    while (left > 0) {
        if (from < 0) {  // the next segment
            s = a.order[++at];
            sg = a.segs[s];
            from = 0;
        }
        const Narrow nw(a, sg);
        const int ktiles = nw.ktiles;
        const int unit = (int)(from / ktiles);
        const int kt0 = (int)(from - (int64_t)unit * ktiles);
        const int kt1 = (int)min((int64_t)ktiles, kt0 + left);
        const int rt = unit / nw.groups, h = (unit - rt * nw.groups) * a.heads + hw;
        const uint32_t nrows = (uint32_t)sg.ntok * a.G, row0 = (uint32_t)rt * kRows;
        if (first && a.Ng == 0 && hw == 0 && lane == 0)
            tell_split(a, false, me, sg, from, kt0, ktiles, sg.t0 + row0 / a.G, (int)(row0 % a.G), h,
                       (int)min((uint32_t)kRows, nrows - row0));
        left -= kt1 - kt0;
        from += kt1 - kt0;
        if (from == nw.tiles()) from = -1;
        const bool begins = first;
        first = false;
        if (h >= a.Hk) continue;  // (the last group of heads may be short)

        // the query: row g of the tile, channels 64 i + 16 j .. + 15
        uint32_t qf[KS][2];
        float f[2];                // of rows 2 j and 2 j + 1
        int pos[2];                // a row past the unit's last hides no key
        {
            const uint32_t rr = row0 + g, tok = rr < nrows ? rr / a.G : 0;
            const bool ok = rr < nrows;
            const int64_t t = sg.t0 + tok;
            const int hq = h * a.G + (ok ? (int)(rr - tok * a.G) : 0);
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
            float up = row_power(top);
            float mine = a.scale * a.ks[h] * kLog2e * inverse_power(up);
            if (mine < 0.0f) mine = -mine, up = -up;  // maxima are of the raw scores
            mine = fmaxf(mine, 0x1p-126f);
            const int place = ok ? position(a, sg, s, t) : 0x7FFFFFFF;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                f[r] = __shfl_sync(~0u, mine, 4 * (2 * j + r));
                pos[r] = __shfl_sync(~0u, place, 4 * (2 * j + r));
            }
#pragma unroll
            for (int i = 0; i < 2 * H; ++i) {
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                // steps 4 (i / 2) + 2 (i % 2) + {0, 1}: channels 4 at a time
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    qf[4 * (i >> 1) + 2 * (i & 1) + (k >> 1)][k & 1] =
                        pack_f16(__uint_as_float(u[k] << 16) * up, __uint_as_float(u[k] & 0xFFFF0000u) * up);
            }
        }
        const bool causal = __any_sync(~0u, min(pos[0], pos[1]) < sg.k1 - 1);

        const int32_t *tab = a.table + (int64_t)sg.row * a.width;
        // this lane's key of tile kt: its cache row, or -1
        auto slot_of = [&](int kt) -> int {
            const int64_t p = (int64_t)sg.k0 + (int64_t)kt * kStep + lane;
            if (kt >= kt1 || p >= sg.k1) return -1;
            uint32_t in;
            const int64_t id = tab[block_of(a, (uint32_t)p, in)];
            if (id < 0) return -1;
            const int64_t slot = id * a.bs + in;
            return slot < a.S ? (int)slot : -1;
        };
        auto issue = [&](int kt, int st, int slot) {
            const uint32_t mask = __ballot_sync(~0u, slot >= 0);
            if (lane == 0) sh_mask[warp][st] = mask;
            const uint32_t dst = ring + st * C::kStageBytes;
            if (kt < kt1) {
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    const int idx = i * 32 + lane, key = idx / KS, c = idx % KS;
                    const int sl = __shfl_sync(~0u, slot, key);
                    const int64_t at = (int64_t)(sl < 0 ? 0 : sl) * (a.Hk * D) + h * D + c * 16;
                    copy16(dst + place<D, false>(key, c), a.kc + at, sl >= 0);
                    copy16(dst + 32 * D + place<D, true>(key, c), a.vc + at, sl >= 0);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };

        // o[n]: channels 16 (or 8) g + 2 n, + 1 of each 128 (or 64), for rows 2 j, 2 j + 1
        float o[NT / 2][4];
#pragma unroll
        for (int i = 0; i < NT / 2; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < ST - 1; ++i) issue(kt0 + i, i, slot_of(kt0 + i));
        int next = slot_of(kt0 + ST - 1);
        int st = 0, fill = ST - 1;  // stages in turn
        for (int kt = kt0; kt < kt1; ++kt) {
            __syncwarp();  // the stage written below has been read by all lanes
            issue(kt + ST - 1, fill, next);
            next = slot_of(kt + ST);
            asm volatile("cp.async.wait_group %0;" ::"n"(ST - 1) : "memory");
            __syncwarp();
            const int use_st = st;
            st = st + 1 == ST ? 0 : st + 1;
            fill = fill + 1 == ST ? 0 : fill + 1;
            const uint32_t kb = ring + use_st * C::kStageBytes, vb = kb + 32 * D;
            const uint32_t mask = sh_mask[warp][use_st];
            if (mask == 0) continue;
            // scores of keys 16 t + g (and + 8) for rows 2 j and 2 j + 1: the keys are the
            // products' rows, so that eight of the sixteen are not wasted on a few queries
            float sc[2][4] = {};
#pragma unroll
            for (int i = 0; i < H; ++i) {
                uint32_t u[4][4];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint4 w = lds16(kb + place<D, false>(8 * t + g, 4 * i + j));
                    u[t][0] = w.x, u[t][1] = w.y, u[t][2] = w.z, u[t][3] = w.w;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        mma16816(sc[t], codes_f16(u[2 * t][k]), codes_f16(u[2 * t + 1][k]),
                                 codes_f16_hi(u[2 * t][k]), codes_f16_hi(u[2 * t + 1][k]),
                                 qf[4 * i + k][0], qf[4 * i + k][1]);
            }
            if (mask != ~0u || causal) {
                const uint32_t p0 = (uint32_t)sg.k0 + (uint32_t)kt * kStep;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = 16 * t + 8 * (e >> 1) + g;
                        // (a key of the mask lies below 2^31)
                        if (!((mask >> key) & 1) || (int64_t)(p0 + key) > pos[e & 1]) sc[t][e] = -INFINITY;
                    }
                // A NaN among the values of a key that some row does not see (weight 0) would
                // reach that row: taken out, and given to the rows that see the key.
                if (causal && __any_sync(~0u, (int64_t)p0 + (kStep - 1) > min(pos[0], pos[1]))) {
                    uint32_t bad = 0;
#pragma unroll 1
                    for (int i = lane; i < kStep * KS; i += 32) {
                        const uint32_t at = vb + place<D, true>(i / KS, i % KS);
                        if (nan_bits(lds16(at))) {
                            bad |= 1u << (i / KS);
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
                        }
                    }
                    bad = __reduce_or_sync(~0u, bad);
                    if (bad != 0) {
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const int64_t last = (int64_t)pos[r] - p0;  // the last key that the row sees
                            const uint32_t see = last < 0 ? 0u : last >= 31 ? ~0u : (2u << (int)last) - 1u;
                            if ((bad & mask & see) == 0) continue;
#pragma unroll
                            for (int n = 0; n < NT / 2; ++n) o[n][r] = o[n][2 + r] = __uint_as_float(0x7FFFFFFFu);
                        }
                        __syncwarp();
                    }
                }
            }
            float top[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                top[r] = fmaxf(fmaxf(sc[0][r], sc[0][r + 2]), fmaxf(sc[1][r], sc[1][r + 2]));
                top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 4));
                top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 8));
                top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 16));
                // A reference is the next value above any maximum so far (-inf and inf are their
                // own), so that no weight, whose score is not rounded, is above 1 (and FP16
                // holds it times 2^15).
                top[r] *= f[r];
                top[r] = top[r] >= m[r] ? fmaf(fminf(fabsf(top[r]), 0x1.fffffep127f), 0x1.2p-24f, top[r]) : m[r];
            }
            if (__any_sync(~0u, top[0] != m[0] || top[1] != m[1])) {
                const float c0 = ex2(m[0] - (top[0] == -INFINITY ? 0.0f : top[0])),
                            c1 = ex2(m[1] - (top[1] == -INFINITY ? 0.0f : top[1]));
                l[0] *= c0;
                l[1] *= c1;
#pragma unroll
                for (int i = 0; i < NT / 2; ++i) {
                    o[i][0] *= c0;
                    o[i][1] *= c1;
                    o[i][2] *= c0;
                    o[i][3] *= c1;
                }
                m[0] = top[0];
                m[1] = top[1];
            }
            const float n0 = m[0] == -INFINITY ? 0.0f : -m[0], n1 = m[1] == -INFINITY ? 0.0f : -m[1];
            // weights, turned so that a thread has those of row g and keys 2 j, 2 j + 1 (of
            // each eight)
            uint32_t pw[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float e0 = ex2(fmaf(sc[t >> 1][2 * (t & 1)], f[0], n0)),
                            e1 = ex2(fmaf(sc[t >> 1][2 * (t & 1) + 1], f[1], n1));
                l[0] += e0;
                l[1] += e1;
                asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(pw[t]) : "r"(pack_f16(e0 * kUp, e1 * kUp)));
            }
            // values: keys 16 u + {2j, 2j + 1, 2j + 8, 2j + 9}, channels as the products' rows
#pragma unroll
            for (int u = 0; u < 2; ++u) {
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
                        const int n = hv * 8 + c * 2;
                        mma16816(o[n], codes_f16(l0), codes_f16_hi(l0), codes_f16(h0), codes_f16_hi(h0),
                                 pw[2 * u], pw[2 * u + 1]);
                        mma16816(o[n + 1], codes_f16(l1), codes_f16_hi(l1), codes_f16(h1), codes_f16_hi(h1),
                                 pw[2 * u], pw[2 * u + 1]);
                    }
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        const bool full = kt1 - kt0 == ktiles, direct = full && a.Ng == 0;
        constexpr int W = D == 64 ? 8 : 16;  // channels of a thread (of each 128)
        float *const po = full ? a.whole : a.part, *const pml = full ? a.whole_ml : a.part_ml;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(~0u, l[r], 4);
            l[r] += __shfl_xor_sync(~0u, l[r], 8);
            l[r] += __shfl_xor_sync(~0u, l[r], 16);
            const uint32_t rr = row0 + 2 * j + r;
            if (rr >= nrows) continue;
            const uint32_t tok = rr / a.G;
            const int64_t t = sg.t0 + tok;
            const int hq = h * a.G + (int)(rr - tok * a.G);
            const int64_t slot = full ? ((s < a.B ? a.T : 0) + t) * a.Hq + hq
                                      : ((int64_t)(2 * me + (begins ? 0 : 1)) * a.heads + hw) * kRows + 2 * j + r;
            const float inv = row_factor(a.vs[h], l[r], a.ks[h]);
#pragma unroll
            for (int n = 0; n < NT / 2; n += 4) {
                const int d = (n / 8) * 128 + W * g + 2 * (n % 8);
                float v[8] = {o[n][r], o[n][2 + r], o[n + 1][r], o[n + 1][2 + r],
                              o[n + 2][r], o[n + 2][2 + r], o[n + 3][r], o[n + 3][2 + r]};
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] *= 1.0f / kUp;
                if (direct) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k] * inv, v[2 * k + 1] * inv);
                        w[k] = *reinterpret_cast<const uint32_t *>(&b);
                    }
                    *reinterpret_cast<uint4 *>(a.out + t * a.ldo + (int64_t)hq * D + d) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(po + slot * D + d);
                    dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                    dst[1] = make_float4(v[4], v[5], v[6], v[7]);
                }
            }
            if (g == 0) {
                if (!direct) {
                    pml[slot * 2] = m[r];
                    pml[slot * 2 + 1] = l[r];
                } else if (a.lse) {
                    a.lse[t * a.Hq + hq] = row_lse(m[r], l[r], a.ks[h]);
                }
            }
        }
        __syncwarp();
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
            bool bad = false;  // a sum below 0: the row saw a value that is NaN
            if (b + lane < n) {
                const float2 v = *reinterpret_cast<const float2 *>(ml + 2 * piece(b + lane));
                mi = v.x, li = fabsf(v.y);
                bad = v.y < 0.0f;
            }
            if (__any_sync(~0u, bad))
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = __uint_as_float(0x7FFFFFFFu);
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
        const float ks = a.ks[hq / a.G], inv = row_factor(a.vs[hq / a.G], l, ks);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const __nv_bfloat16 v = __float2bfloat16_rn(o[e] * inv);
            a.out[t * a.ldo + (int64_t)hq * D + lane + 32 * e] = *reinterpret_cast<const uint16_t *>(&v);
        }
        if (a.lse && lane == 0) a.lse[t * a.Hq + hq] = row_lse(m, l, ks);
    }
};

// Without groups: the rows of the units that more than one worker had.  A warp takes a
// row; a row of many pieces is shared by a CTA's eight.
template <int D>
__global__ void __launch_bounds__(256, 4) attention_join_split_kernel(const Args a) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float sh_o[8][D];
    __shared__ float2 sh_ml[8];
    const bool wide = a.wide_own;
    const int heads = wide ? 1 : a.heads, rows = wide ? kWideRows : kRows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int splits = a.plan->splits, many = a.plan->many;
    const float *po = wide ? a.wpart : a.part, *ml = wide ? a.wpart_ml : a.part_ml;
    for (int pass = 0; pass <= many; ++pass) {
        const int chunks = pass == 0 ? rows / 8 : rows;  // of a unit and head: 8 rows, or one
        for (int i = blockIdx.x; i < splits * heads * chunks; i += gridDim.x) {
            const int unit = i / chunks, chunk = i - unit * chunks, hw = unit % heads;
            const Split sp = a.splits[unit / heads];
            const int h = sp.head + hw, r = pass == 0 ? chunk * 8 + warp : chunk;
            if ((sp.n > kManyPieces) != (pass == 1) || h >= a.Hk || r >= sp.rows) continue;
            auto slot = [&](int k) -> int64_t {
                return ((k == 0 ? sp.first : 2 * (sp.c0 + k)) * (int64_t)heads + hw) * rows + r;
            };
            const uint32_t rr = sp.sub + r, tok = rr / (uint32_t)a.G;
            const int64_t t = sp.token + tok;
            const int hq = h * a.G + (int)(rr - tok * a.G);
            Row<D> row;
            if (pass == 0) {
                row.add(po, ml, sp.n, slot);
                row.write(a, t, hq);
                continue;
            }
            const int k0 = sp.n * warp / 8, k1 = sp.n * (warp + 1) / 8;
            row.add(po, ml, k1 - k0, [&](int k) { return slot(k0 + k); });
#pragma unroll
            for (int e = 0; e < D / 32; ++e) sh_o[warp][lane + 32 * e] = row.o[e];
            if (lane == 0) sh_ml[warp] = make_float2(row.m, row.l);
            __syncthreads();
            if (warp == 0) {
                Row<D> all;
                all.add(&sh_o[0][0], reinterpret_cast<const float *>(sh_ml), 8, [](int k) { return (int64_t)k; });
                all.write(a, t, hq);
            }
            __syncthreads();
        }
    }
}

// With groups: every row, from its prefix and its request's own part.  A CTA takes
// rows of request blockIdx.x, a warp one at a time.
template <int D>
__global__ void __launch_bounds__(256, 4) attention_join_kernel(const Args a) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const Segment own = a.segs[blockIdx.x];
    Segment pre;
    pre.k0 = pre.k1 = 0;
    if (own.group >= 0) pre = a.segs[a.B + own.group];
    const Plan plan = *a.plan;
    const int64_t rows = (int64_t)own.ntok * a.Hq;
    for (int64_t i = blockIdx.y * 8ll + (threadIdx.x >> 5); i < rows; i += gridDim.y * 8ll) {
        const uint32_t tok = (uint32_t)(i / a.Hq);
        const int64_t t = own.t0 + tok;
        const int hq = (int)(i - (int64_t)tok * a.Hq), h = hq / a.G, gi = hq - h * a.G;
        Row<D> row;
        for (int k = 0; k < 2; ++k) {  // the prefix, then the own part
            const Segment &g = k == 0 ? pre : own;
            if (g.k1 <= g.k0 || t < g.t0 || t >= g.t0 + g.ntok) continue;
            const bool wide = k == 0 ? a.wide_prefix : a.wide_own;
            int64_t u0 = g.before;
            int n, r;
            if (wide) {
                const Wide w(a, g);
                const int rt = (int)((uint32_t)(t - g.t0) / (uint32_t)w.tokens);
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
                r = (int)((t - g.t0) - (int64_t)rt * w.tokens) * a.G + gi;
            } else {
                const Narrow w(a, g);
                const uint32_t rr = (uint32_t)(t - g.t0) * a.G + gi;
                n = w.ktiles;
                u0 += ((int64_t)(rr / kRows) * w.groups + h / a.heads) * n;
                r = (int)(rr % kRows);
            }
            const Pieces p(u0, n, plan.total[wide], plan.workers[wide]);
            if (p.n == 1) {
                const int64_t at = ((k == 1 ? a.T : 0) + t) * a.Hq + hq;
                row.add(a.whole, a.whole_ml, 1, [&](int) { return at; });
            } else if (wide) {
                row.add(a.wpart, a.wpart_ml, p.n, [&](int j) { return p.slot(j) * kWideRows + r; });
            } else {
                row.add(a.part, a.part_ml, p.n,
                        [&](int j) { return (p.slot(j) * a.heads + h % a.heads) * kRows + r; });
            }
        }
        row.write(a, t, hq);
    }
}

// Which segments go to the wide kernel, by the rows that a unit has on average:
// requests' own parts and prefixes.  16 requests of 8192 keys, 8 KV heads: at 32 rows a
// unit the narrow kernel took 101 us and the wide one 119, at 64 rows 181 and 121.
constexpr int64_t kWideFrom = 48;

struct Layout {
    bool wide_own, wide_prefix;
    size_t part, part_ml, wpart, wpart_ml, whole, whole_ml, segs, order, starts, splits, plan, bytes;
};

Layout layout(int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t B, int64_t Ng) {
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    const int64_t G = Hq / Hk;
    Layout w;
    const bool can = D <= 128 && G <= 128;
    w.wide_own = can && T * G >= kWideFrom * B;
    w.wide_prefix = can && Ng > 0 && T * G >= kWideFrom * Ng;
    const size_t slots = !w.wide_own || (Ng > 0 && !w.wide_prefix) ? 2 * kNarrowWorkers * kRows : 0,
                 wslots = w.wide_own || w.wide_prefix ? 2 * kMaxCtas * kWideRows : 0,
                 rows = Ng > 0 ? (size_t)(2 * T * Hq) : 0;
    size_t at = 256;  // (room to begin at a multiple of 256)
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
    w.segs = take((size_t)(B + Ng) * sizeof(Segment));
    w.order = take((size_t)(B + Ng) * 2 * sizeof(int));
    w.starts = take((kNarrowWorkers + kMaxCtas) * sizeof(Start));
    w.splits = take((kNarrowWorkers + kMaxCtas) * sizeof(Split));
    w.plan = take(sizeof(Plan));
    w.bytes = at;
    return w;
}

bool shape_ok(int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t B, int64_t Ng) {
    if (T < 0 || Hq < 0 || Hk < 0 || B < 0 || Ng < 0) return false;
    if (Hq > 1024 || T >= (int64_t)1 << 24 || T * Hq >= (int64_t)1 << 31 || B > 8192 || Ng > B) return false;
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
    jet_status st = launch_pdl(attention_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a);
    if (st == JET_OK && (!a.wide_own || (a.Ng > 0 && !a.wide_prefix)))
        st = launch_pdl(attention_kernel<D>, dim3((unsigned)a.ctas), dim3(32 * C::kWarps), C::kSmem, stream, a);
    if (st == JET_OK && (a.wide_own || a.wide_prefix)) st = launch_attention_wide(dev, a, D, stream);
    if (st != JET_OK) return st;
    if (a.Ng > 0) {
        // rows of a request on average, eight warps a CTA
        const int64_t want = (a.T * a.Hq / a.B + 7) / 8;
        return launch_pdl(attention_join_kernel<D>, dim3((unsigned)a.B, (unsigned)(want < 1 ? 1 : want > 1024 ? 1024 : want)),
                          dim3(256), 0, stream, a);
    }
    return launch_pdl(attention_join_split_kernel<D>, dim3((unsigned)(4 * dev.num_sms)), dim3(256), 0, stream, a);
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
    a.bs_shift = -1;
    for (int i = 0; i < 30; ++i)
        if (block_size == (int64_t)1 << i) a.bs_shift = i;
    a.B = (int)B, a.po = prefix_offsets, a.pl = prefix_lengths, a.Ng = (int)n_prefix;
    a.scale = scale, a.out = out, a.ldo = ldo, a.lse = lse;
    // arrays begin at multiples of 256
    uint8_t *base = static_cast<uint8_t *>(ws) - (reinterpret_cast<uintptr_t>(ws) & 255);
    a.part = reinterpret_cast<float *>(base + w.part);
    a.part_ml = reinterpret_cast<float *>(base + w.part_ml);
    a.whole = reinterpret_cast<float *>(base + w.whole);
    a.whole_ml = reinterpret_cast<float *>(base + w.whole_ml);
    a.wpart = reinterpret_cast<float *>(base + w.wpart);
    a.wpart_ml = reinterpret_cast<float *>(base + w.wpart_ml);
    a.segs = reinterpret_cast<Segment *>(base + w.segs);
    a.order = reinterpret_cast<int *>(base + w.order);
    a.starts = reinterpret_cast<Start *>(base + w.starts);
    a.splits = reinterpret_cast<Split *>(base + w.splits);
    a.plan = reinterpret_cast<Plan *>(base + w.plan);
    a.wide_own = w.wide_own, a.wide_prefix = w.wide_prefix;
    a.ctas = dev.num_sms < kMaxCtas ? dev.num_sms : kMaxCtas;
    const int warps = D > 128 ? Cfg<256>::kWarps : kNarrowWarps;
    a.heads = a.Hk < warps ? a.Hk : warps;
    a.phases = warps / a.heads;
    const cudaStream_t s = as_stream(stream);
    return D == 64 ? launch<64>(dev, a, s) : D == 128 ? launch<128>(dev, a, s) : launch<256>(dev, a, s);
}
