// Log-probabilities of given tokens under the head, and their gradient, without
// the logits of the whole vocabulary in memory.
//
// With z_tv = scale x_t . w_v, lse_t = ln sum_v e^z_tv, logp_t = z_t,target - lse_t;
// backward, with g_t the gradient of logp_t (0 where the target is no token):
//   d_tv = scale g_t ([v = target] - e^(z_tv - lse_t)),  dx = d w,  dw = d^T x.
// All four products (z twice, dx, dw) are BF16 products on the 5th-generation
// tensor core with binary32 accumulators, one kernel template:
//   kLse   z tiles; the epilogue keeps each row's maximum and sum of a tile's half,
//          joined over the tiles by head_join_kernel.  The tensor core cuts
//          off its sums (2^-24 of the sum a step): over 4096 products that is 2e-5 of
//          a logit, so after every 1024 the sum is taken over into registers and
//          added up there, rounded to nearest;
//   kGrad  z tiles of a piece of the vocabulary again, with the same sums, so that
//          e^(z - lse) is of the forward's own logits; the epilogue writes d in
//          BF16 (the type that the next two products read: up to 2^-8 of each
//          value, whose errors mostly cancel in the sums of many tokens; up to 128
//          tokens have a second array with what the first left over, 2^-16, and
//          both products go over the two);
//   kDx    d w over the piece (w read MN-major as it lies), binary32 results of
//          one or more ranges of the contraction, added up by head_sum_kernel;
//   kDw    d^T x (both read MN-major as they lie), BF16.
// Forward: bound by the tensor core for many tokens (2 T K V operations), by the
// read of w for few.  Backward: 8 T K V operations, a quarter of them the logits
// again; d passes through memory once per piece.  4096 tokens, K = 4096, V = 128256:
// forward 2.76 ms (1562 TFLOP/s; 2.58 ms before its sums were taken over every 1024
// products), backward 8.45 ms (2040 TFLOP/s of the 8 T K V, above the library
// product's rate: what is left there is the logits' second product).  1537 tokens, K =
// 5120, V = 50257: backward 1.74 ms.  48 tokens, K = 512, V = 2048: forward 8.5 us, two
// launches of dependent loads.
//
// The kernel is persistent: warp 0 loads operand slices of 64 along the
// contraction by TMA into a ring of stages (128-byte swizzle), warp 1 issues the
// MMAs into one of two TMEM accumulators, warps 4-7 (kLse, kGrad: 4-11) drain the other one.  Large
// products run as CTA pairs on 256 x 256 tiles, few rows on single CTAs with 128 x
// 128.  Every mbarrier wait is bounded (jet_common.cuh); a role that gives up sets
// the CTA's abort flag, copies and MMAs in flight are awaited, TMEM is freed.  (A pair's
// other CTA learns of it through its own waits; the two then meet at the last cluster
// barrier.)
#include <cuda_bf16.h>

#include <mutex>

#include "jet_common.cuh"
#include "tcgen05_f16.cuh"
#include "tensor_map.cuh"

namespace {

using namespace jet;
using namespace jet::ptx;

enum Product { kLse = 0, kGrad = 1, kDx = 2, kDw = 3 };

// Wait sites in the status word (after those of jet_common.cuh).
constexpr unsigned kSiteProducer = 16, kSiteMma = 17, kSiteMmaTmem = 18, kSiteEpilogue = 19,
                   kSiteDrain = 20;

constexpr int BM = 128, BK = 64;
constexpr int kChunk = 16;  // kLse, kGrad: slices that the tensor core adds up by itself
__host__ __device__ constexpr bool sums_chunks(int product) { return product == kLse || product == kGrad; }
__host__ __device__ constexpr int threads_of(int product) { return sums_chunks(product) ? 384 : 256; }
// Their registers a thread after setmaxnreg: 128 x 72 + 256 x 216 = 384 x 168.
constexpr uint32_t kRegsControl = 72, kRegsEpilogue = 216;
static_assert(128 * kRegsControl + 256 * kRegsEpilogue <= 384 * 168, "registers");
constexpr int kStages = 6;
constexpr int kABytes = BM * BK * 2;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int CL>
struct Cfg {
    static constexpr int BN = CL == 2 ? 256 : 128;        // tile width
    static constexpr int kBRows = BN / CL;                 // of them in one CTA's memory
    static constexpr int kStageBytes = kABytes + kBRows * BK * 2;
    static constexpr int kSmem = kStages * kStageBytes + 1024;
    static constexpr int kTmemCols = 2 * BN;
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct Epilogue {
    const int64_t *target;
    const float *lse, *dlogp;
    float scale;
    int V, v0;               // vocabulary, and the first entry of the piece
    float2 *part;            // kLse: [2 column tiles][T] (maximum, sum) in powers of two
    float *zt;               // kLse: [T] the target's logit, in powers of two
    uint16_t *d;             // kGrad: [T][ldd]
    int64_t ldd;
    int second;              // kGrad, kDw: the first row of d's second part, or 0
    float *acc;              // kDx: [splits][rows of d][K]
    uint16_t *dw;            // kDw: [V][K]
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// rows R, columns C, contraction D in elements; `splits` ranges of the contraction.
template <int P, int CL>
__global__ void __launch_bounds__(threads_of(P), 1)
head_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb, int R,
            int C, int D, int splits, const Epilogue ep, unsigned *status) {
    using CF = Cfg<CL>;
    constexpr int S = kStages, BN = CF::BN;
    constexpr bool kPair = CL == 2, kAMn = P == kDw, kBMn = P == kDx || P == kDw, kChunks = sums_chunks(P);
    extern __shared__ uint8_t dyn[];
    __shared__ uint64_t full_bar[S], empty_bar[S], tfull_bar[2], tempty_bar[2], drain_bar;
    __shared__ uint32_t tmem_sh;
    __shared__ int abort_sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = (smem_u32(dyn) + 1023u) & ~1023u;
    const uint32_t rank = kPair ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    volatile int *abort = &abort_sh;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull_bar[b], 1);
            mbar_init(&tempty_bar[b], (kChunks ? 8 : 4) * CL);
        }
        mbar_init(&drain_bar, 1);
        abort_sh = 0;
        fence_mbar_init();
        prefetch_tmap(&ta);
        prefetch_tmap(&tb);
    }
    if (warp == 1) {
        if (kPair) {
            tmem_alloc_pair(&tmem_sh, CF::kTmemCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(&tmem_sh, CF::kTmemCols);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    if (kPair) cluster_sync(); else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_sh;
    griddep_launch_dependents();
    griddep_wait();

    const int tm = (R + BM * CL - 1) / (BM * CL), tn = (C + BN - 1) / BN;
    const int nk = (D + BK - 1) / BK;
    const int total = tm * tn * splits;
    const int unit0 = blockIdx.x / CL, step = gridDim.x / CL;
    // Unit t: the operand of fewer tiles is walked fastest, so that it stays in
    // L2 while the other streams.
    auto coords = [&](int t, int &m0, int &n0, int &k0, int &k1, int &sp) {
        sp = t % splits;
        const int u = t / splits;
        int mt, nt;
        if (P == kDw) {
            nt = u % tn;
            mt = u / tn;
        } else {
            mt = u % tm;
            nt = u / tm;
        }
        m0 = (mt * CL + (int)rank) * BM;
        n0 = nt * BN;
        k0 = (int)((int64_t)sp * nk / splits);
        k1 = (int)((int64_t)(sp + 1) * nk / splits);
    };

    // A wait of a whole warp; all lanes leave alike.
    auto wait = [&](uint64_t *bar, uint32_t parity, unsigned site) -> bool {
        return __all_sync(~0u, mbar_wait(bar, parity, abort, status, site));
    };
    if constexpr (kChunks)
        if (warp < 4) reg_dealloc<kRegsControl>();
    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int t = unit0; ok && t < total; t += step) {
                int m0, n0, k0, k1, sp;
                coords(t, m0, n0, k0, k1, sp);
                const int b0 = n0 + CF::kBRows * (int)rank;
                for (int kb = k0; kb < k1; ++kb, ++it) {
                    const int s = it % S;
                    if (!mbar_wait(&empty_bar[s], ((it / S) & 1u) ^ 1u, abort, status, kSiteProducer)) {
                        ok = false;
                        break;
                    }
                    const uint32_t as = base + s * CF::kStageBytes, bs = as + kABytes;
                    const uint32_t fb = kPair ? map_to_cta(&full_bar[s], 0) : 0u;
                    if (leader) mbar_arrive_expect_tx(&full_bar[s], CL * CF::kStageBytes);
                    auto load = [&](uint32_t dst, const CUtensorMap *m, int x, int y) {
                        if (kPair) tma_load_pair(dst, m, fb, x, y);
                        else tma_load(dst, m, &full_bar[s], x, y);
                    };
                    if (kAMn) {
#pragma unroll
                        for (int i = 0; i < BM / 64; ++i)
                            load(as + i * 8192, &ta, m0 + 64 * i, kb * BK);
                    } else {
                        load(as, &ta, kb * BK, m0);
                    }
                    if (kBMn) {
#pragma unroll
                        for (int i = 0; i < CF::kBRows / 64; ++i)
                            load(bs + i * 8192, &tb, b0 + 64 * i,
                                 P == kDw && kb * BK >= ep.second ? kb * BK - ep.second : kb * BK);
                    } else {
                        load(bs, &tb, kb * BK, b0);
                    }
                }
            }
            // every load has landed before the CTA may exit (a pair's are the leader's)
            // and, in a pair's other CTA, what the leader's commits still have to say to its
            // barriers: its memory may be another CTA's when they arrive, and the leader's own
            // drain does not say that they have (where one stays out the leader has given up,
            // and so do the others)
            for (uint32_t i = it > (uint32_t)S ? it - S : 0u; i < it; ++i)
                if (!mbar_wait(leader ? &full_bar[i % S] : &empty_bar[i % S], (i / S) & 1u, nullptr, status,
                               kSiteDrain) &&
                    !leader)
                    break;
        }
        __syncwarp();
    } else if (warp == 1 && leader) {
        constexpr uint32_t kIdesc = idesc_16bit(BM * CL, BN, true, kAMn, kBMn);
        // MN-major: atoms of 64 x 8 (1024 bytes apart along the contraction),
        // 8192 bytes between neighbouring blocks of 64
        auto desc = [](uint32_t a, bool mn, int ks) {
            return mn ? smem_desc(a + ks * 2048, 8192, 1024, kSwizzle128B)
                      : smem_desc(a + ks * 32, 16, 1024, kSwizzle128B);
        };
        uint32_t it = 0, sums = 0;  // slices, and sums (a tile's, or a chunk's of it) so far
        bool ok = true;
        for (int t = unit0; ok && t < total; t += step) {
            int m0, n0, k0, k1, sp;
            coords(t, m0, n0, k0, k1, sp);
            for (int kb = k0; kb < k1; ++kb, ++it) {
                const bool begins = kChunks ? (kb - k0) % kChunk == 0 : kb == k0;
                const bool ends = kb + 1 == k1 || (kChunks && (kb + 1 - k0) % kChunk == 0);
                const uint32_t buf = sums & 1u;
                const int s = it % S;
                if ((begins && !wait(&tempty_bar[buf], ((sums >> 1) & 1u) ^ 1u, kSiteMmaTmem)) ||
                    !wait(&full_bar[s], (it / S) & 1u, kSiteMma)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t as = base + s * CF::kStageBytes, bs = as + kABytes;
#pragma unroll
                    for (int ks = 0; ks < BK / 16; ++ks) {
                        const uint64_t da = desc(as, kAMn, ks), db = desc(bs, kBMn, ks);
                        const uint32_t more = !begins || ks > 0;
                        if (kPair) mma_16bit_pair(tmem + buf * BN, da, db, kIdesc, more);
                        else mma_16bit(tmem + buf * BN, da, db, kIdesc, more);
                    }
                    if (kPair) mma_commit_pair_mc(&empty_bar[s], 0x3);
                    else mma_commit(&empty_bar[s]);
                    if (ends) {
                        if (kPair) mma_commit_pair_mc(&tfull_bar[buf], 0x3);
                        else mma_commit(&tfull_bar[buf]);
                    }
                }
                sums += ends;
                __syncwarp();
            }
        }
        if (lane == 0) {
            if (kPair) mma_commit_pair_mc(&drain_bar, 0x1);
            else mma_commit(&drain_bar);
        }
        __syncwarp();
        mbar_wait(&drain_bar, 0, nullptr, status, kSiteDrain);
    } else if (kChunks && warp >= 4) {
        if constexpr (kChunks) {
            reg_alloc<kRegsEpilogue>();
            constexpr int H = BN / 2;  // columns of a thread
            const int quad = warp & 3, half = (warp - 4) >> 2;
            uint32_t release[2] = {0u, 0u};
            if (kPair) {
                release[0] = map_to_cta(&tempty_bar[0], 0);
                release[1] = map_to_cta(&tempty_bar[1], 0);
            }
            const float c = ep.scale * kLog2e;
            uint32_t sums = 0;
            bool ok = true;
            for (int t = unit0; ok && t < total; t += step) {
                int m0, n0, k0, k1, sp;
                coords(t, m0, n0, k0, k1, sp);
                const int row = m0 + quad * 32 + lane, col0 = n0 + half * H;
                float2 acc[H / 2];
#pragma unroll
                for (int i = 0; i < H / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
                for (int kb = k0; kb < k1; kb += kChunk, ++sums) {
                    const uint32_t buf = sums & 1u;
                    if (!wait(&tfull_bar[buf], (sums >> 1) & 1u, kSiteEpilogue)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t from = tmem + ((uint32_t)(quad * 32) << 16) + buf * BN + half * H;
#pragma unroll
                    for (int ch = 0; ch < H / 16; ++ch) {
                        uint32_t r[16];
                        tmem_ld16(from + ch * 16, r);
                        tmem_ld_wait(r);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            acc[ch * 8 + i] = __fadd2_rn(
                                acc[ch * 8 + i],
                                make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])));
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (kPair) mbar_arrive_cluster_relaxed(release[buf]);
                        else mbar_arrive(&tempty_bar[buf]);
                    }
                }
                if (!ok) break;
                if (row >= (P == kGrad ? max(R, ep.second) : R)) continue;
                // the target's column, if it is one of these (kGrad: rows from R on are zeros)
                const int64_t token = P == kLse || row < R ? ep.target[row] : -1;
                const bool real = token >= 0 && token < ep.V;
                const int want = real ? (int)token - (P == kGrad ? ep.v0 : 0) - col0 : -1;
                if constexpr (P == kLse) {
                    float top = -INFINITY, zt = 0.0f;
#pragma unroll
                    for (int i = 0; i < H / 2; ++i) {
                        float2 x = __fmul2_rn(acc[i], make_float2(c, c));
                        if (col0 + 2 * i >= C) x.x = -INFINITY;
                        if (col0 + 2 * i + 1 >= C) x.y = -INFINITY;
                        if (want == 2 * i) zt = x.x;
                        if (want == 2 * i + 1) zt = x.y;
                        acc[i] = x;
                        top = fmaxf(top, fmaxf(x.x, x.y));
                    }
                    if (want >= 0 && want < H) ep.zt[row] = zt;
                    const float2 use = make_float2(top == -INFINITY ? 0.0f : -top, top == -INFINITY ? 0.0f : -top);
                    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int i = 0; i < H / 2; ++i) {
                        const float2 d = __fadd2_rn(acc[i], use);
                        sum = __fadd2_rn(sum, make_float2(ex2(d.x), ex2(d.y)));
                    }
                    ep.part[(int64_t)(2 * (n0 / BN) + half) * R + row] = make_float2(top, sum.x + sum.y);
                } else {
                    const float g = real ? ep.dlogp[row] * ep.scale : 0.0f, neg = real ? -ep.lse[row] * kLog2e : 0.0f;
                    uint16_t *dst = ep.d + (int64_t)row * ep.ldd + col0;
#pragma unroll
                    for (int i = 0; i < H / 2; i += 4) {
                        if (col0 + 2 * i >= C) break;  // (up to the padded row end past the piece's last)
#pragma unroll
                        for (int k = i; k < i + 4; ++k) {
                            const float2 x = __ffma2_rn(acc[k], make_float2(c, c), make_float2(neg, neg));
                            acc[k].x = g * ((want == 2 * k ? 1.0f : 0.0f) - ex2(x.x));
                            acc[k].y = g * ((want == 2 * k + 1 ? 1.0f : 0.0f) - ex2(x.y));
                            if (g == 0.0f) acc[k] = make_float2(0.0f, 0.0f);  // whatever lse is there
                        }
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) w[k] = pack2(acc[i + k].x, acc[i + k].y);
                        *reinterpret_cast<uint4 *>(dst + 2 * i) = make_uint4(w[0], w[1], w[2], w[3]);
                        if (ep.second > 0) {  // what is left over
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                w[k] = pack2(acc[i + k].x - __uint_as_float(w[k] << 16),
                                             acc[i + k].y - __uint_as_float(w[k] & 0xFFFF0000u));
                            *reinterpret_cast<uint4 *>(dst + ep.second * ep.ldd + 2 * i) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
            }
        }
    } else if (!kChunks && warp >= 4) {
        const int quad = warp & 3;
        uint32_t release[2] = {0u, 0u};
        if (kPair) {
            release[0] = map_to_cta(&tempty_bar[0], 0);
            release[1] = map_to_cta(&tempty_bar[1], 0);
        }
        uint32_t tiles = 0;
        for (int t = unit0; t < total; t += step, ++tiles) {
            int m0, n0, k0, k1, sp;
            coords(t, m0, n0, k0, k1, sp);
            const int row = m0 + quad * 32 + lane;
            const bool row_ok = row < R;
            const uint32_t buf = tiles & 1u;
            if (!wait(&tfull_bar[buf], (tiles >> 1) & 1u, kSiteEpilogue)) break;
            tc_fence_after();
            const uint32_t acc0 = tmem + ((uint32_t)(quad * 32) << 16) + buf * BN;
#pragma unroll 1
            for (int ch = 0; ch < BN / 32; ++ch) {
                uint32_t r[32];
                __syncwarp();
                tmem_ld32(acc0 + ch * 32, r);
                tmem_wait32(r);
                const int col = n0 + ch * 32;
                if constexpr (P == kDx) {
                    float *dst = ep.acc + ((int64_t)sp * R + row) * C + col;
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        if (row_ok && col + i < C)
                            *reinterpret_cast<uint4 *>(dst + i) =
                                make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
                } else {
                    uint16_t *dst = ep.dw + ((int64_t)ep.v0 + row) * C + col;
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        auto two = [&](int k) {
                            return pack2(__uint_as_float(r[i + k]), __uint_as_float(r[i + k + 1]));
                        };
                        if (row_ok && col + i < C)
                            *reinterpret_cast<uint4 *>(dst + i) = make_uint4(two(0), two(2), two(4), two(6));
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (kPair) mbar_arrive_cluster_relaxed(release[buf]);
                else mbar_arrive(&tempty_bar[buf]);
            }
        }
    }
    tc_fence_before();
    // neither CTA of a pair leaves while the other can still use its barriers,
    // memory or TMEM
    if (kPair) cluster_sync(); else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        if (kPair) tmem_dealloc_pair(tmem, CF::kTmemCols);
        else tmem_dealloc(tmem, CF::kTmemCols);
    }
}

// lse and logp of every row from the tiles' maxima and sums, in a fixed order:
// 32 rows a CTA, 32 slices of the tiles.
__global__ void __launch_bounds__(1024)
head_join_kernel(const float2 *__restrict__ part, const float *__restrict__ zt,
                 const int64_t *__restrict__ target, int64_t T, int V, int tiles,
                 float *__restrict__ logp, float *__restrict__ lse) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float2 sh[32][33];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int64_t row = blockIdx.x * 32ll + lane;
    float m = -INFINITY, s = 0.0f;
    auto add = [&](float2 v) {
        const float top = fmaxf(m, v.x), use = top == -INFINITY ? 0.0f : top;
        s = s * ex2(m - use) + v.y * ex2(v.x - use);
        m = top;
    };
    if (row < T)
        for (int i = slice; i < tiles; i += 32) add(part[(int64_t)i * T + row]);
    sh[slice][lane] = make_float2(m, s);
    __syncthreads();
    if (slice != 0 || row >= T) return;
    m = -INFINITY, s = 0.0f;
#pragma unroll 8
    for (int i = 0; i < 32; ++i) add(sh[i][lane]);
    const float l = log2f(s);
    lse[row] = kLn2 * (m + l);
    const int64_t token = target[row];
    logp[row] = token >= 0 && token < V ? kLn2 * ((zt[row] - m) - l) : 0.0f;
}

// dx = BF16(sum of the ranges' results, in order, after the pieces before); a range has
// `each` values, the second part of d's from `second` on (or 0: none).
__global__ void __launch_bounds__(256)
head_sum_kernel(const float4 *__restrict__ acc, int splits, int64_t n4, int64_t each, int64_t second,
                const float4 *__restrict__ before,
                float4 *__restrict__ run, uint2 *__restrict__ dx) {
    griddep_launch_dependents();
    griddep_wait();
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n4; i += gridDim.x * 256ll) {
        float4 a = before ? before[i] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int s = 0; s < splits; ++s) {
            float4 b = acc[s * each + i];
            if (second > 0) {
                const float4 c = acc[s * each + second + i];
                b.x += c.x, b.y += c.y, b.z += c.z, b.w += c.w;
            }
            a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
        }
        if (dx) dx[i] = make_uint2(pack2(a.x, a.y), pack2(a.z, a.w));
        else run[i] = a;
    }
}

// ------------------------------------------------------------------- host --

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// How a call is cut; by the sizes alone, so that the workspace and the order of
// the sums do not depend on the device.
struct Plan {
    int cl_z, cl_dx;          // CTAs a tile (dw: by the piece)
    int64_t piece;            // vocabulary entries of a piece (backward)
    int splits;               // ranges of dx's contraction in a piece
    int64_t tiles_z;          // column tiles of the forward
    int64_t second, rows;     // where d's second part begins (0: none); rows of d
    size_t fwd_bytes, d_bytes, acc_bytes, run_bytes;
};

constexpr int64_t kClusters = 76;        // what the plan counts with: pairs of 152 SMs
constexpr int64_t kPieceBytes = 512ll << 20;

Plan plan(int64_t T, int64_t V, int64_t K) {
    Plan p;
    // up to 128 rows a pair would have half a tile idle; above, single CTAs read w once for
    // each 128 rows (forward, K = 4096, V = 32000: 128 rows 59.3 us on single CTAs and 61.1 on
    // pairs, 256 rows 106.6 and 61.9)
    p.cl_z = p.cl_dx = T <= BM ? 1 : 2;
    p.tiles_z = 2 * ceil_div(V, p.cl_z == 2 ? 256 : 128);  // halves of tiles
    p.fwd_bytes = up256((size_t)(p.tiles_z * T) * sizeof(float2)) + up256((size_t)T * 4);
    // d in two parts for the few rows of one tile: one gradient's rounding can be all of an
    // output's error there (0.0031 of its norm against 0.0017), and the products are bound by
    // w (K = 4096, V = 32000, cold caches: 64 tokens 220 us, 128 tokens 270; 129 in one part
    // on pairs 230)
    p.second = T <= BM ? ceil_div(T, BK) * BK : 0;
    p.rows = p.second > 0 ? 2 * p.second : T;
    // pieces of equal size whose d takes at most kPieceBytes, 4096 entries at least
    int64_t most = kPieceBytes / (2 * (p.rows > 0 ? p.rows : 1)) / 256 * 256;
    if (most < 4096) most = 4096;
    const int64_t pieces = ceil_div(V, most);
    p.piece = ceil_div(ceil_div(V, pieces), 256) * 256;
    // dx has few tiles and a long contraction: the ranges that make the shortest
    // time of whole waves (a slice of 64 takes about 540 cycles on a pair, 270 on
    // one CTA; a range 12 slices of start-up) and of its results' way through
    // memory (about 3500 bytes a cycle, written and read)
    const int64_t tiles = ceil_div(p.rows, BM * p.cl_dx) * ceil_div(K, p.cl_dx == 2 ? 256 : 128);
    const int64_t at_once = p.cl_dx == 2 ? kClusters : 2 * kClusters, nk = ceil_div(p.piece, BK);
    const int64_t cycles = p.cl_dx == 2 ? 540 : 270;
    int64_t best = -1;
    p.splits = 1;
    for (int64_t s = 1; s <= 16 && s <= nk; ++s) {
        if (s > 1 && s * p.rows * K * 4 > (512ll << 20)) break;
        const int64_t cost = ceil_div(tiles * s, at_once) * (ceil_div(nk, s) + 12) * cycles + s * p.rows * K * 8 / 3500;
        if (best < 0 || cost < best) best = cost, p.splits = (int)s;
    }
    p.d_bytes = up256((size_t)(p.rows * p.piece) * 2);
    p.acc_bytes = up256((size_t)(p.splits * p.rows * K) * 4);
    p.run_bytes = p.piece < V ? up256((size_t)(T * K) * 4) : 0;
    return p;
}

bool shape_ok(int64_t T, int64_t K, int64_t V) {
    return T >= 0 && T < (int64_t)1 << 22 && K >= 8 && K <= 65536 && K % 8 == 0 && V >= 1 &&
           V < (int64_t)1 << 24;
}

// One product: A's rows R, B's C, contraction D.
template <int P, int CL>
jet_status product(const DeviceInfo &dev, const CUtensorMap &ta, const CUtensorMap &tb, int64_t R,
                   int64_t C, int64_t D, int splits, const Epilogue &ep, cudaStream_t stream) {
    using CF = Cfg<CL>;
    auto kernel = head_kernel<P, CL>;
    static std::mutex mu;
    static void *done[64] = {};
    static int at_once[64] = {};
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.blockDim = dim3(threads_of(P));
    cfg.dynamicSmemBytes = CF::kSmem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CL;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int units;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev.context == nullptr || done[dev.ordinal] != dev.context) {
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, CF::kSmem) !=
                cudaSuccess) {
                cudaGetLastError();
                return JET_ERR_CUDA;
            }
            int n = dev.num_sms / CL;
            if (CL > 1) {
                cfg.gridDim = dim3((unsigned)(dev.num_sms - dev.num_sms % CL));
                int clusters = 0;
                if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) == cudaSuccess && clusters > 0)
                    n = clusters;
                cudaGetLastError();
            }
            at_once[dev.ordinal] = n;
            done[dev.ordinal] = dev.context;
        }
        units = at_once[dev.ordinal];
    }
    const int64_t total = ceil_div(R, BM * CL) * ceil_div(C, CF::BN) * splits;
    cfg.gridDim = dim3((unsigned)((total < units ? total : units) * CL));
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, ta, tb, (int)R, (int)C, (int)D, splits, ep,
                           dev.status_word) != cudaSuccess) {
        cudaGetLastError();
        return JET_ERR_CUDA;
    }
    return launch_status();
}

template <int P>
jet_status product(int cl, const DeviceInfo &dev, const CUtensorMap &ta, const CUtensorMap &tb,
                   int64_t R, int64_t C, int64_t D, int splits, const Epilogue &ep, cudaStream_t s) {
    return cl == 2 ? product<P, 2>(dev, ta, tb, R, C, D, splits, ep, s)
                   : product<P, 1>(dev, ta, tb, R, C, D, splits, ep, s);
}

inline bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

size_t jet_head_workspace(int op, int64_t T, int64_t V, int64_t K) {
    if (!shape_ok(T, K, V) || T == 0) return 0;
    const Plan p = plan(T, V, K);
    return op == JET_OP_HEAD_LOGP ? p.fwd_bytes : p.d_bytes + p.acc_bytes + p.run_bytes;
}

jet_status jet_head_logp(const uint16_t *x, const uint16_t *w, int64_t T, int64_t K, int64_t V,
                         const int64_t *target, float scale, float *logp, float *lse, void *ws,
                         size_t ws_bytes, jet_stream_t stream) {
    JET_REQUIRE(shape_ok(T, K, V) && scale > 0.0f && scale < INFINITY, JET_ERR_SHAPE);
    JET_REQUIRE(T == 0 || (x && w && target && logp && lse), JET_ERR_NULL);
    JET_REQUIRE(aligned16(x) && aligned16(w) && aligned16(ws) && aligned_to(target, 8) &&
                    aligned_to(logp, 4) && aligned_to(lse, 4),
                JET_ERR_ALIGN);
    const Plan p = plan(T, V, K);
    JET_REQUIRE(T == 0 || (ws && ws_bytes >= p.fwd_bytes), JET_ERR_WORKSPACE);
    DeviceInfo dev;
    jet_status st = current_device(&dev);
    if (st != JET_OK) return st;
    if (T == 0) return JET_OK;
    const cudaStream_t s = as_stream(stream);
    Epilogue ep = {};
    ep.target = target, ep.scale = scale, ep.V = (int)V;
    ep.part = static_cast<float2 *>(ws);
    ep.zt = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) +
                                      up256((size_t)(p.tiles_z * T) * sizeof(float2)));
    CUtensorMap ta, tb;
    if (!map_rows16(&ta, x, (uint64_t)K, (uint64_t)T, (uint64_t)K, BM) ||
        !map_rows16(&tb, w, (uint64_t)K, (uint64_t)V, (uint64_t)K, BM))
        return JET_ERR_CUDA;
    st = product<kLse>(p.cl_z, dev, ta, tb, T, V, K, 1, ep, s);
    if (st != JET_OK) return st;
    return launch_pdl(head_join_kernel, dim3((unsigned)ceil_div(T, 32)), dim3(1024), 0, s,
                      (const float2 *)ep.part, (const float *)ep.zt, target, T, (int)V,
                      (int)p.tiles_z, logp, lse);
}

jet_status jet_head_logp_bwd(const uint16_t *x, const uint16_t *w, int64_t T, int64_t K, int64_t V,
                             const int64_t *target, const float *lse, const float *dlogp,
                             float scale, uint16_t *dx, uint16_t *dw, void *ws, size_t ws_bytes,
                             jet_stream_t stream) {
    JET_REQUIRE(shape_ok(T, K, V) && scale > 0.0f && scale < INFINITY, JET_ERR_SHAPE);
    JET_REQUIRE(T == 0 || (x && w && target && lse && dlogp && (dx || dw)), JET_ERR_NULL);
    JET_REQUIRE(aligned16(x) && aligned16(w) && aligned16(dx) && aligned16(dw) && aligned16(ws) &&
                    aligned_to(target, 8) && aligned_to(lse, 4) && aligned_to(dlogp, 4),
                JET_ERR_ALIGN);
    const Plan p = plan(T, V, K);
    JET_REQUIRE(T == 0 || (ws && ws_bytes >= p.d_bytes + p.acc_bytes + p.run_bytes), JET_ERR_WORKSPACE);
    DeviceInfo dev;
    jet_status st = current_device(&dev);
    if (st != JET_OK) return st;
    const cudaStream_t s = as_stream(stream);
    if (T == 0) {
        if (dw && cudaMemsetAsync(dw, 0, (size_t)(V * K) * 2, s) != cudaSuccess) {
            cudaGetLastError();
            return JET_ERR_CUDA;
        }
        return JET_OK;
    }
    uint8_t *base = static_cast<uint8_t *>(ws);
    Epilogue ep = {};
    ep.target = target, ep.lse = lse, ep.dlogp = dlogp, ep.scale = scale, ep.V = (int)V;
    ep.d = reinterpret_cast<uint16_t *>(base), ep.ldd = p.piece, ep.second = (int)p.second;
    ep.acc = reinterpret_cast<float *>(base + p.d_bytes);
    ep.dw = dw;
    float *run = reinterpret_cast<float *>(base + p.d_bytes + p.acc_bytes);
    CUtensorMap tx, tx64;
    if (!map_rows16(&tx, x, (uint64_t)K, (uint64_t)T, (uint64_t)K, BM) ||
        !map_rows16(&tx64, x, (uint64_t)K, (uint64_t)T, (uint64_t)K, BK))
        return JET_ERR_CUDA;
    for (int64_t v0 = 0; v0 < V; v0 += p.piece) {
        const int64_t nv = V - v0 < p.piece ? V - v0 : p.piece;
        CUtensorMap tw, tw64, td, td64;
        if (!map_rows16(&tw, w + v0 * K, (uint64_t)K, (uint64_t)nv, (uint64_t)K, BM) ||
            !map_rows16(&tw64, w + v0 * K, (uint64_t)K, (uint64_t)nv, (uint64_t)K, BK) ||
            !map_rows16(&td, ep.d, (uint64_t)nv, (uint64_t)p.rows, (uint64_t)p.piece, BM) ||
            !map_rows16(&td64, ep.d, (uint64_t)nv, (uint64_t)p.rows, (uint64_t)p.piece, BK))
            return JET_ERR_CUDA;
        ep.v0 = (int)v0;
        st = product<kGrad>(p.cl_z, dev, tx, tw, T, nv, K, 1, ep, s);
        if (st != JET_OK) return st;
        if (dx) {
            const int64_t nk = ceil_div(nv, BK);
            const int splits = (int)(p.splits < nk ? p.splits : nk);
            st = product<kDx>(p.cl_dx, dev, td, tw64, p.rows, K, nv, splits, ep, s);
            if (st != JET_OK) return st;
            const bool last = v0 + nv == V;
            const int64_t n4 = T * K / 4, want = ceil_div(n4, 256), cap = (int64_t)dev.num_sms * 8;
            st = launch_pdl(head_sum_kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(256), 0,
                            s, reinterpret_cast<const float4 *>(ep.acc), splits, n4, p.rows * K / 4, p.second * K / 4,
                            v0 > 0 ? reinterpret_cast<const float4 *>(run) : (const float4 *)nullptr,
                            reinterpret_cast<float4 *>(run),
                            last ? reinterpret_cast<uint2 *>(dx) : (uint2 *)nullptr);
            if (st != JET_OK) return st;
        }
        if (dw) {
            // (a last piece of up to 128 entries has no rows for a pair's second CTA)
            st = product<kDw>(nv <= BM ? 1 : 2, dev, td64, tx64, nv, K, p.rows, 1, ep, s);
            if (st != JET_OK) return st;
        }
    }
    return JET_OK;
}
