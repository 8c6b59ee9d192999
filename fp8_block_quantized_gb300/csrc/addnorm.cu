// The residual addition, RMSNorm and the 1x128 quantization of its output in
// one pass (jet_add_rmsnorm_quant_1x128), and the backward of the addition
// and the norm (jet_add_rmsnorm_bwd).
//
// Forward: h = BF16(x + d) (one rounding: what the residual stream holds),
// then exactly the arithmetic of jet_rmsnorm_quant_1x128 on h: lane l of a
// warp adds the squares of the elements 8 (32 j + l) + t in order, a five-level
// butterfly, ms = ss / K, r = 1 / sqrt(ms + eps), y = (h r) g in binary32 and
// the 1x128 group rule.  So the codes and scales equal those of the separate
// addition and jet_rmsnorm_quant_1x128 bit for bit, for any number of rows.
//
// Both directions are bound by HBM at many rows, each input read and each output
// written once (forward 16384 x 5120: 87.5 us, 6742 GB/s, 99% of a copy's rate;
// backward of 8192 x 4096 with three gradients and the residual's: 60.8 us, 6618
// GB/s), and by latency at few (forward 16 x 4096: 2.3 us).
#include <cuda_bf16.h>

#include "jet_common.cuh"
#include "quant_rule.cuh"

namespace {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two binary32 values rounded to BF16 (nearest, ties to even), a in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
    return pack_bf16(__fadd_rn(bf16_lo(a), bf16_lo(b)), __fadd_rn(bf16_hi(a), bf16_hi(b)));
}

__device__ __forceinline__ uint4 add_chunk(const uint4 &a, const uint4 &b) {
    return make_uint4(add_bf16x2(a.x, b.x), add_bf16x2(a.y, b.y), add_bf16x2(a.z, b.z),
                      add_bf16x2(a.w, b.w));
}

// acc += square of each of the 8 BF16 values of a chunk, in order.
__device__ __forceinline__ float add_squares(float acc, const uint4 &c) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = bf16_lo(w[i]), b = bf16_hi(w[i]);
        acc = __fmaf_rn(a, a, acc);
        acc = __fmaf_rn(b, b, acc);
    }
    return acc;
}

__device__ __forceinline__ float rms_factor(float acc, int64_t K, float eps) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) acc = __fadd_rn(acc, __shfl_xor_sync(0xffffffffu, acc, d));
    const float v = __fadd_rn(__fdiv_rn(acc, (float)K), eps);
    return v == 0.0f ? 0.0f : __fdiv_rn(1.0f, __fsqrt_rn(v));
}

// Quantize this lane's chunk of row m (group grp, the 16 lanes of one
// half-warp); all lanes call it (shuffles), those past the row's end with
// `valid` false.  The products run on -r, which gives -y bit for bit, the
// form the division of quant_rule.cuh wants.
__device__ __forceinline__ void quant_chunk(const uint4 &hc, const uint4 &gc, float nr, bool valid,
                                            int64_t grp, int64_t m, int64_t M, int64_t K, int lane,
                                            uint8_t *q, float *s) {
    const uint32_t hw[4] = {hc.x, hc.y, hc.z, hc.w}, gw[4] = {gc.x, gc.y, gc.z, gc.w};
    const float2 nr2 = make_float2(nr, nr);
    float ny[8];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __fmul2_rn(make_float2(bf16_lo(hw[i]), bf16_hi(hw[i])), nr2);
        const float2 v = __fmul2_rn(t, make_float2(bf16_lo(gw[i]), bf16_hi(gw[i])));
        ny[2 * i] = v.x;
        ny[2 * i + 1] = v.y;
        amax = max_abs2(amax, v.x, v.y);
    }
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    if (valid) {
        const float sc = group_scale(amax);
        const Divisor dv = make_divisor(sc);
        uint2 out;
        out.x = encode4(ny, dv);
        out.y = encode4(ny + 4, dv);
        *reinterpret_cast<uint2 *>(q + m * K + grp * 128 + 8 * (lane & 15)) = out;
        if ((lane & 15) == 0) s[grp * M + m] = sc;
    }
}

// One CTA of T threads per row, NI chunks a thread (K <= 8 T NI).  All of a
// thread's loads go out at once; h stays in its registers for the
// quantization, and a copy in shared memory lets warp 0 sum the squares in the
// fixed order (its 32 lanes' chains of K / 32 additions are the only serial part).
// h may be x or d (in place): a thread reads its chunks before it writes them.
template <int T, int NI>
__global__ void __launch_bounds__(T)
add_rmsnorm_row_kernel(const uint16_t *x, const uint16_t *d, const uint16_t *__restrict__ g,
                       int64_t M, int64_t K, float eps, uint16_t *h, uint8_t *q, float *s,
                       float *rstd) {
    extern __shared__ uint4 rowbuf[];  // the row's K / 8 chunks of h
    __shared__ float r_sh;
    jet::griddep_launch_dependents();
    jet::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int nchunks = (int)(K / 8), nj = (nchunks + 31) / 32;
    const int64_t m = blockIdx.x;
    const uint4 *xr = reinterpret_cast<const uint4 *>(x + m * K);
    const uint4 *dr = reinterpret_cast<const uint4 *>(d + m * K);
    uint4 *hr = reinterpret_cast<uint4 *>(h + m * K);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 c[NI], b[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int ci = threadIdx.x + i * T;
        c[i] = ci < nchunks ? xr[ci] : zero;
        b[i] = ci < nchunks ? dr[ci] : zero;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int ci = threadIdx.x + i * T;
        c[i] = add_chunk(c[i], b[i]);
        if (ci < nchunks) {
            rowbuf[ci] = c[i];
            hr[ci] = c[i];
        }
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        float acc = 0.0f;
#pragma unroll 4
        for (int j = 0; j < nj; ++j) {
            const int ci = 32 * j + lane;
            acc = add_squares(acc, ci < nchunks ? rowbuf[ci] : zero);
        }
        const float r = rms_factor(acc, K, eps);
        if (lane == 0) {
            r_sh = r;
            if (rstd) rstd[m] = r;
        }
    }
    const uint4 *gain = reinterpret_cast<const uint4 *>(g);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int ci = threadIdx.x + i * T;
        b[i] = ci < nchunks ? gain[ci] : zero;
    }
    __syncthreads();
    const float nr = -r_sh;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int ci = threadIdx.x + i * T;
        quant_chunk(c[i], b[i], nr, ci < nchunks, ci >> 4, m, M, K, lane, q, s);
    }
}

// Rows too long for that: one warp per row at a time.  The first pass adds, writes h and sums the
// squares; the second reads back this lane's own chunks of h.  h may be x or
// d (in place), so none of the three is read-only to the compiler.
constexpr int kAnThreads = 256;
constexpr int kAnBatch = 4;

__global__ void __launch_bounds__(kAnThreads)
add_rmsnorm_quant_kernel(const uint16_t *x, const uint16_t *d, const uint16_t *__restrict__ g,
                         int64_t M, int64_t K, float eps, uint16_t *h, uint8_t *q, float *s,
                         float *rstd) {
    jet::griddep_launch_dependents();
    jet::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t nchunks = K / 8, nj = (nchunks + 31) / 32;
    const int64_t warps = (int64_t)gridDim.x * (kAnThreads / 32);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint4 *gain = reinterpret_cast<const uint4 *>(g);
    for (int64_t m = (int64_t)blockIdx.x * (kAnThreads / 32) + (threadIdx.x >> 5); m < M;
         m += warps) {
        const uint4 *xr = reinterpret_cast<const uint4 *>(x + m * K);
        const uint4 *dr = reinterpret_cast<const uint4 *>(d + m * K);
        uint4 *hr = reinterpret_cast<uint4 *>(h + m * K);
        float acc = 0.0f;
        for (int64_t j = 0; j < nj; j += kAnBatch) {
            uint4 a[kAnBatch], b[kAnBatch];
#pragma unroll
            for (int u = 0; u < kAnBatch; ++u) {
                const int64_t ci = 32 * (j + u) + lane;
                a[u] = ci < nchunks ? xr[ci] : zero;
                b[u] = ci < nchunks ? dr[ci] : zero;
            }
#pragma unroll
            for (int u = 0; u < kAnBatch; ++u) {
                const int64_t ci = 32 * (j + u) + lane;
                const uint4 c = add_chunk(a[u], b[u]);
                if (ci < nchunks) hr[ci] = c;
                acc = add_squares(acc, c);
            }
        }
        const float r = rms_factor(acc, K, eps);
        if (rstd && lane == 0) rstd[m] = r;
        for (int64_t j = 0; j < nj; ++j) {
            const int64_t ci = 32 * j + lane;
            const bool ok = ci < nchunks;
            quant_chunk(ok ? hr[ci] : zero, ok ? gain[ci] : zero, -r, ok, 2 * j + (lane >> 4), m,
                        M, K, lane, q, s);
        }
    }
}

// ---------------------------------------------------------------------------
// Backward.  With xh = h r (r the saved 1 / rms of the row), dy the sum of
// the given output gradients and u = g dy:
//   dx = dres + r (u - xh a),  a = (sum_k u xh) / K,   dg = sum_m dy xh,
// all in binary32, dx rounded once to BF16.  One CTA per row at a time; a
// thread owns the same NC chunks of 8 columns in every row, so its share of
// dg stays in registers and is written once, as one of at most kBwdParts
// partial rows that a second kernel adds in order (deterministic).
// ---------------------------------------------------------------------------
constexpr int kBwdParts = 304;
constexpr int64_t kBwdMaxK = 32768;

__device__ __forceinline__ void unpack8(const uint4 &c, float (&f)[8]) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

// The CTA's next row is copied into shared memory (cp.async, every thread its
// own chunks, so no barrier is needed for it) while this one is reduced and
// written; three or four rows in flight were slower (8192 x 4096, three
// gradients: 69 and 70 us against 61), as fewer CTAs fit.
__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     (unsigned)__cvta_generic_to_shared(dst)),
                 "l"(src)
                 : "memory");
}

struct BwdArgs {
    int stages;  // rows in shared memory
    const uint16_t *in[5];  // h, then the gradients: dy0 .. , and dres last if it is there
    int ny, nt;             // output gradients; tensors in all
    const uint16_t *g;
    const float *rstd;
    int64_t M, K;
    uint16_t *dx;
    float *part;
};

// dot over the CTA, the same in every thread; `red` alternates between rows, so
// that one barrier a row is enough.
__device__ __forceinline__ float block_sum(float v, float *red) {
    const int lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < nwarps ? red[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                      pack_bf16(f[6], f[7]));
}

__device__ __forceinline__ void store_part(float *p, const float (&dg)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(dg[0], dg[1], dg[2], dg[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(dg[4], dg[5], dg[6], dg[7]);
}

// K <= 8192: one chunk a thread, at most kMax of them; two CTAs an SM where the
// registers allow it.
template <int kMax>
__global__ void __launch_bounds__(kMax, kMax <= 640 ? 2 : 1)
add_rmsnorm_bwd_kernel(const BwdArgs a) {
    extern __shared__ uint4 stage[];  // [2][nt][threads]
    __shared__ float red[2][32];
    jet::griddep_launch_dependents();
    jet::griddep_wait();
    const int64_t M = a.M;
    const int nchunks = (int)(a.K / 8), T = blockDim.x, ci = threadIdx.x;
    const bool ok = ci < nchunks, has_res = a.nt > a.ny + 1;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint4 gain = ok ? reinterpret_cast<const uint4 *>(a.g)[ci] : zero;
    float dg[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    auto fetch = [&](int64_t m, int ph) {
        if (m < M && ok) {
#pragma unroll
            for (int k = 0; k < 5; ++k)
                if (k < a.nt)
                    cp_async16(stage + (ph * a.nt + k) * T + ci,
                               reinterpret_cast<const uint4 *>(a.in[k]) + m * nchunks + ci);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(blockIdx.x, 0);
    float r_next = (int64_t)blockIdx.x < M ? a.rstd[blockIdx.x] : 0.0f;
    int phase = 0;
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x, phase ^= 1) {
        const float r = r_next;
        if (m + gridDim.x < M) r_next = a.rstd[m + gridDim.x];
        fetch(m + gridDim.x, phase ^ 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        const uint4 *in = stage + phase * a.nt * T + ci;
        float xh[8], u[8], f[8], dot = 0.0f;
        unpack8(ok ? in[0] : zero, xh);
        unpack8(ok ? in[T] : zero, u);
#pragma unroll
        for (int k = 2; k < 4; ++k) {
            if (k > a.ny) break;
            unpack8(ok ? in[k * T] : zero, f);
#pragma unroll
            for (int t = 0; t < 8; ++t) u[t] += f[t];
        }
        unpack8(gain, f);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            xh[t] *= r;
            dg[t] = fmaf(u[t], xh[t], dg[t]);
            u[t] *= f[t];
            dot = fmaf(u[t], xh[t], dot);
        }
        const float mean = block_sum(dot, red[phase]) / (float)a.K;
        if (!ok) continue;
        unpack8(has_res ? in[(a.nt - 1) * T] : zero, f);
#pragma unroll
        for (int t = 0; t < 8; ++t) f[t] = fmaf(r, fmaf(-xh[t], mean, u[t]), f[t]);
        reinterpret_cast<uint4 *>(a.dx)[m * nchunks + ci] = pack8(f);
    }
    if (ok) store_part(a.part + blockIdx.x * a.K + 8 * (int64_t)ci, dg);
}

// Longer rows, NC chunks a thread: no registers to keep a row, which is read again
// for its second pass, from shared memory where a.stages (1 or 2) rows fit, else
// from L2 (4096 x 10240 with two gradients and the residual's: 97 us with two rows,
// 102 with one, 147 from L2; 1024 x 20480: 64 with one, 98 from L2).
template <int NC, bool kStaged>
__global__ void __launch_bounds__(1024)
add_rmsnorm_bwd_wide_kernel(const BwdArgs a) {
    extern __shared__ uint4 stage[];  // [stages][nt][NC][threads]
    __shared__ float red[2][32];
    jet::griddep_launch_dependents();
    jet::griddep_wait();
    const int nchunks = (int)(a.K / 8), T = blockDim.x;
    const bool has_res = a.nt > a.ny + 1;
    float dg[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int t = 0; t < 8; ++t) dg[i][t] = 0.0f;
    auto fetch = [&](int64_t m, int ph) {
        if (m < a.M) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int ci = threadIdx.x + i * T;
                for (int k = 0; ci < nchunks && k < a.nt; ++k)
                    cp_async16(stage + ((ph * a.nt + k) * NC + i) * T + threadIdx.x,
                               reinterpret_cast<const uint4 *>(a.in[k]) + m * nchunks + ci);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (kStaged) fetch(blockIdx.x, 0);
    int phase = 0;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, phase ^= 1) {
        const float r = a.rstd[m];
        const int ph = a.stages == 2 ? phase : 0;
        if (kStaged && a.stages == 2) {
            fetch(m + gridDim.x, phase ^ 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else if (kStaged) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        // a thread reads what it fetched itself
        auto chunk = [&](int k, int i) {
            return kStaged ? stage[((ph * a.nt + k) * NC + i) * T + threadIdx.x]
                           : reinterpret_cast<const uint4 *>(a.in[k])[m * nchunks + threadIdx.x + i * T];
        };
        auto terms = [&](int i, float (&xh)[8], float (&dy)[8]) {
            float f[8];
            unpack8(chunk(0, i), xh);
            unpack8(chunk(1, i), dy);
#pragma unroll 1
            for (int k = 2; k <= a.ny; ++k) {
                unpack8(chunk(k, i), f);
#pragma unroll
                for (int t = 0; t < 8; ++t) dy[t] += f[t];
            }
#pragma unroll
            for (int t = 0; t < 8; ++t) xh[t] *= r;
        };
        float xh[8], u[8], f[8], dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int ci = threadIdx.x + i * T;
            if (ci >= nchunks) continue;
            terms(i, xh, u);
            unpack8(reinterpret_cast<const uint4 *>(a.g)[ci], f);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                dg[i][t] = fmaf(u[t], xh[t], dg[i][t]);
                dot = fmaf(u[t] * f[t], xh[t], dot);
            }
        }
        const float mean = block_sum(dot, red[phase]) / (float)a.K;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int ci = threadIdx.x + i * T;
            if (ci >= nchunks) continue;
            float gf[8];
            terms(i, xh, u);
            unpack8(reinterpret_cast<const uint4 *>(a.g)[ci], gf);
            unpack8(has_res ? chunk(a.nt - 1, i) : make_uint4(0, 0, 0, 0), f);
#pragma unroll
            for (int t = 0; t < 8; ++t) f[t] = fmaf(r, fmaf(-xh[t], mean, u[t] * gf[t]), f[t]);
            reinterpret_cast<uint4 *>(a.dx)[m * nchunks + ci] = pack8(f);
        }
        if (kStaged && a.stages == 1) fetch(m + gridDim.x, 0);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int ci = threadIdx.x + i * T;
        if (ci < nchunks) store_part(a.part + blockIdx.x * a.K + 8 * (int64_t)ci, dg[i]);
    }
}

// dg[k] = the partial rows' sum in a fixed order: a CTA takes 32 columns, eight
// threads of four columns a row, 128 rows at a time (304 rows of 5120: 2.0 us;
// 2.6 with one column a thread); then the lanes of a warp, then the warps.
__global__ void __launch_bounds__(1024)
dgain_reduce_kernel(const float *__restrict__ part, int parts, int64_t K, float *__restrict__ dg) {
    __shared__ float4 sum[32][9];
    jet::griddep_launch_dependents();
    jet::griddep_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = lane & 7;
    const float *col = part + blockIdx.x * (int64_t)32 + 4 * c;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](const float4 &v) {
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
    };
    for (int p0 = threadIdx.x >> 3; p0 < parts; p0 += 128 * 3) {
        float4 v[3];
#pragma unroll
        for (int i = 0; i < 3; ++i)
            v[i] = p0 + 128 * i < parts ? *reinterpret_cast<const float4 *>(col + (p0 + 128 * i) * K)
                                        : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 3; ++i) add(v[i]);
    }
#pragma unroll
    for (int o = 8; o < 32; o *= 2)
        add(make_float4(__shfl_xor_sync(0xffffffffu, acc.x, o), __shfl_xor_sync(0xffffffffu, acc.y, o),
                        __shfl_xor_sync(0xffffffffu, acc.z, o), __shfl_xor_sync(0xffffffffu, acc.w, o)));
    if (lane < 8) sum[w][c] = acc;
    __syncthreads();
    if (w == 0) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += reinterpret_cast<const float *>(sum[i])[lane];
        dg[blockIdx.x * (int64_t)32 + lane] = s;
    }
}

// CTAs of the backward at most: short rows leave room for more of them
// (16384 x 2048: 53 us with 608, 81 with 304; x 1024: 38 with 1216, 54 with 608).
int64_t bwd_parts(int64_t M, int64_t K) {
    const int64_t cap = K <= 1024 ? 4 * kBwdParts : K <= 2048 ? 2 * kBwdParts : kBwdParts;
    return M < cap ? M : cap;
}

// Allows a kernel more than the 48 KB of shared memory, its static part among
// them, that every launch may have.  The limit is the kernel's, whatever a call
// needs: another thread may be about to launch it with other sizes.
constexpr size_t kMostSmem = 225 * 1024;

template <typename K>
bool allow_smem(K *kernel) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostSmem) ==
        cudaSuccess)
        return true;
    cudaGetLastError();
    return false;
}

template <int kBytes>
bool aligned_to(const void *p) { return (reinterpret_cast<uintptr_t>(p) & (kBytes - 1)) == 0; }

}  // namespace

// Partial rows of dg.
size_t jet_add_rmsnorm_bwd_workspace(int64_t M, int64_t K) {
    return (size_t)bwd_parts(M, K) * (size_t)K * sizeof(float);
}

jet_status jet_add_rmsnorm_quant_1x128(const uint16_t *x, const uint16_t *d, const uint16_t *g,
                                       int64_t M, int64_t K, float eps, uint16_t *h, uint8_t *q,
                                       float *s, float *rstd, jet_stream_t stream) {
    JET_REQUIRE(M >= 0 && K >= 0, JET_ERR_SHAPE);
    const bool empty = (M == 0 || K == 0);
    JET_REQUIRE(empty || (x && d && g && h && q && s), JET_ERR_NULL);
    JET_REQUIRE(K % 128 == 0 && M < ((int64_t)1 << 31) && K < ((int64_t)1 << 24) &&
                    eps >= 0.0f && eps <= 3.0e38f,
                JET_ERR_SHAPE);
    JET_REQUIRE(jet::aligned16(x) && jet::aligned16(d) && jet::aligned16(g) && jet::aligned16(h) &&
                    jet::aligned16(q) && jet::aligned16(s) && aligned_to<4>(rstd),
                JET_ERR_ALIGN);
    jet::DeviceInfo dev;
    jet_status st = jet::current_device(&dev);
    if (st != JET_OK) return st;
    if (empty) return JET_OK;
    cudaStream_t cs = jet::as_stream(stream);
    const int64_t nchunks = K / 8;
    if (nchunks <= 8 * 512) {
        // Threads of a row, by what keeps enough loads in flight (us, measured):
        // up to four rows an SM 512 (600 x 4096: 5.0, 7.4 with 128); then 128 for
        // K <= 5120 (16384 x 5120: 87, 99 with 256) and 256 for longer rows (4096 x
        // 8192: 40, 45 with 128).
        const int T = M <= 4 * (int64_t)dev.num_sms || nchunks > 8 * 256 ? 512
                      : nchunks > 640                                    ? 256
                                                                         : 128;
        const int ni = (int)((nchunks + T - 1) / T);
        void (*kernel)(const uint16_t *, const uint16_t *, const uint16_t *, int64_t, int64_t, float,
                       uint16_t *, uint8_t *, float *, float *) =
            T == 128 ? (ni == 1 ? add_rmsnorm_row_kernel<128, 1>
                        : ni == 2 ? add_rmsnorm_row_kernel<128, 2>
                        : ni <= 4 ? add_rmsnorm_row_kernel<128, 4> : add_rmsnorm_row_kernel<128, 5>)
            : T == 256 ? (ni <= 4 ? add_rmsnorm_row_kernel<256, 4> : add_rmsnorm_row_kernel<256, 8>)
                       : (ni == 1 ? add_rmsnorm_row_kernel<512, 1>
                          : ni == 2 ? add_rmsnorm_row_kernel<512, 2>
                          : ni <= 4 ? add_rmsnorm_row_kernel<512, 4> : add_rmsnorm_row_kernel<512, 8>);
        const size_t smem = (size_t)K * 2;
        if (smem > 40 * 1024 && !allow_smem(kernel)) return JET_ERR_CUDA;
        return jet::launch_pdl(kernel, dim3((unsigned)M), dim3((unsigned)T), smem, cs, x, d, g, M, K,
                               eps, h, q, s, rstd);
    }
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, add_rmsnorm_quant_kernel,
                                                      kAnThreads, 0) != cudaSuccess ||
        per_sm < 1) {
        cudaGetLastError();
        per_sm = 1;
    }
    const int64_t want = (M + kAnThreads / 32 - 1) / (kAnThreads / 32);
    const int64_t cap = (int64_t)dev.num_sms * per_sm;
    return jet::launch_pdl(add_rmsnorm_quant_kernel, dim3((unsigned)(want < cap ? want : cap)),
                           dim3(kAnThreads), 0, cs, x, d, g, M, K, eps, h, q, s, rstd);
}

jet_status jet_add_rmsnorm_bwd(const uint16_t *h, const uint16_t *g, const float *rstd,
                               const uint16_t *dy0, const uint16_t *dy1, const uint16_t *dy2,
                               const uint16_t *dres, int64_t M, int64_t K, uint16_t *dx, float *dg,
                               void *ws, size_t ws_bytes, jet_stream_t stream) {
    JET_REQUIRE(M >= 0 && K >= 0, JET_ERR_SHAPE);
    JET_REQUIRE(K == 0 || dg, JET_ERR_NULL);
    JET_REQUIRE(M == 0 || K == 0 || (h && g && rstd && dy0 && dx), JET_ERR_NULL);
    JET_REQUIRE(K % 128 == 0 && M < ((int64_t)1 << 31) && K <= kBwdMaxK, JET_ERR_SHAPE);
    JET_REQUIRE(jet::aligned16(h) && jet::aligned16(g) && aligned_to<4>(rstd) &&
                    jet::aligned16(dy0) && jet::aligned16(dy1) && jet::aligned16(dy2) &&
                    jet::aligned16(dres) && jet::aligned16(dx) && jet::aligned16(dg) &&
                    jet::aligned16(ws),
                JET_ERR_ALIGN);
    const size_t need = jet_add_rmsnorm_bwd_workspace(M, K);
    JET_REQUIRE(need == 0 || (ws && ws_bytes >= need), JET_ERR_WORKSPACE);
    jet::DeviceInfo dev;
    jet_status st = jet::current_device(&dev);
    if (st != JET_OK) return st;
    if (K == 0) return JET_OK;
    cudaStream_t cs = jet::as_stream(stream);
    if (M == 0) {  // no row: the gain's gradient is zero
        if (cudaMemsetAsync(dg, 0, (size_t)K * sizeof(float), cs) == cudaSuccess) return JET_OK;
        cudaGetLastError();
        return JET_ERR_CUDA;
    }
    const int64_t nchunks = K / 8;
    const int nc = nchunks <= 1024 ? 1 : nchunks <= 2048 ? 2 : 4;
    const int threads = (int)(((nchunks + nc - 1) / nc + 31) / 32 * 32);
    BwdArgs a = {};
    a.in[a.nt++] = h;
    for (const uint16_t *dy : {dy0, dy1, dy2})
        if (dy) a.in[a.nt++] = dy;
    a.ny = a.nt - 1;
    if (dres) a.in[a.nt++] = dres;
    a.g = g;
    a.rstd = rstd;
    a.M = M;
    a.K = K;
    a.dx = dx;
    a.part = static_cast<float *>(ws);
    const size_t row = (size_t)a.nt * nc * threads * 16;  // in shared memory
    a.stages = nc == 1 || 2 * row <= kMostSmem ? 2 : row <= kMostSmem ? 1 : 0;
    auto *kernel = nc == 1       ? (threads <= 512   ? add_rmsnorm_bwd_kernel<512>
                                    : threads <= 640 ? add_rmsnorm_bwd_kernel<640>
                                                     : add_rmsnorm_bwd_kernel<1024>)
                   : a.stages > 0 ? (nc == 2 ? add_rmsnorm_bwd_wide_kernel<2, true>
                                             : add_rmsnorm_bwd_wide_kernel<4, true>)
                                  : add_rmsnorm_bwd_wide_kernel<4, false>;
    const size_t smem = a.stages * row;
    if (smem > 40 * 1024 && !allow_smem(kernel)) return JET_ERR_CUDA;
    // persistent CTAs, as many as fit (registers, shared memory with 1 KB
    // of the system's) and as there are partial rows
    const int64_t by_threads = threads > 512 && threads <= 640 ? 2 : 1024 / threads;
    const int64_t by_smem = 228 * 1024 / (smem + 1024 + 256);
    const int64_t per_sm = by_threads < by_smem ? by_threads : by_smem;
    const int64_t resident = (int64_t)dev.num_sms * (per_sm > 0 ? per_sm : 1);
    const int64_t most = bwd_parts(M, K);
    const int parts = (int)(most < resident ? most : resident);
    st = jet::launch_pdl(kernel, dim3((unsigned)parts), dim3((unsigned)threads), smem, cs, a);
    if (st != JET_OK) return st;
    return jet::launch_pdl(dgain_reduce_kernel, dim3((unsigned)(K / 32)), dim3(1024), 0, cs,
                           (const float *)a.part, parts, K, dg);
}
