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

// One warp per row at a time.  The first pass adds, writes h and sums the
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

template <int NC>
__global__ void __launch_bounds__(1024)
add_rmsnorm_bwd_kernel(const uint16_t *__restrict__ h, const uint16_t *__restrict__ g,
                       const float *__restrict__ rstd, const uint16_t *__restrict__ dy0,
                       const uint16_t *__restrict__ dy1, const uint16_t *__restrict__ dy2,
                       const uint16_t *dres, int64_t M, int64_t K, uint16_t *dx, float *part) {
    __shared__ float red[2][32];
    jet::griddep_launch_dependents();
    jet::griddep_wait();
    const int64_t nchunks = K / 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    float dg[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int t = 0; t < 8; ++t) dg[i][t] = 0.0f;
    int phase = 0;
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x, phase ^= 1) {
        const float r = rstd[m];
        float xh[NC][8], u[NC][8];
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t ci = threadIdx.x + (int64_t)i * blockDim.x;
            const bool ok = ci < nchunks;
            const int64_t at = m * nchunks + ci;
            auto get = [&](const uint16_t *p, int64_t k) {
                return ok ? reinterpret_cast<const uint4 *>(p)[k] : zero;
            };
            const uint4 hc = get(h, at), a = get(dy0, at), gc = get(g, ci);
            const uint4 b = dy1 ? get(dy1, at) : zero, c = dy2 ? get(dy2, at) : zero;
            float gf[8], t1[8], t2[8];
            unpack8(hc, xh[i]);
            unpack8(a, u[i]);
            unpack8(b, t1);
            unpack8(c, t2);
            unpack8(gc, gf);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                xh[i][t] *= r;
                const float dy = u[i][t] + t1[t] + t2[t];
                dg[i][t] = fmaf(dy, xh[i][t], dg[i][t]);
                u[i][t] = dy * gf[t];
                dot = fmaf(u[i][t], xh[i][t], dot);
            }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0) red[phase][warp] = dot;
        __syncthreads();
        float sum = lane < nwarps ? red[phase][lane] : 0.0f;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float a = sum / (float)K;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t ci = threadIdx.x + (int64_t)i * blockDim.x;
            if (ci >= nchunks) continue;
            const int64_t at = m * nchunks + ci;
            float f[8];
            unpack8(dres ? reinterpret_cast<const uint4 *>(dres)[at] : zero, f);
#pragma unroll
            for (int t = 0; t < 8; ++t) f[t] = fmaf(r, fmaf(-xh[i][t], a, u[i][t]), f[t]);
            reinterpret_cast<uint4 *>(dx)[at] =
                make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                           pack_bf16(f[6], f[7]));
        }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t ci = threadIdx.x + (int64_t)i * blockDim.x;
        if (ci >= nchunks) continue;
        float4 *p = reinterpret_cast<float4 *>(part + blockIdx.x * K + 8 * ci);
        p[0] = make_float4(dg[i][0], dg[i][1], dg[i][2], dg[i][3]);
        p[1] = make_float4(dg[i][4], dg[i][5], dg[i][6], dg[i][7]);
    }
}

// dg[k] = the partial rows' sum in a fixed order: 8 row groups per CTA of 32
// columns, each adding every eighth partial row, then the groups in order.
__global__ void __launch_bounds__(256)
dgain_reduce_kernel(const float *__restrict__ part, int parts, int64_t K, float *__restrict__ dg) {
    __shared__ float sum[8][32];
    jet::griddep_launch_dependents();
    jet::griddep_wait();
    const int c = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t k = blockIdx.x * (int64_t)32 + c;
    float acc = 0.0f;
#pragma unroll 8
    for (int p = w; p < parts; p += 8) acc += part[p * K + k];
    sum[w][c] = acc;
    __syncthreads();
    if (w == 0) {
#pragma unroll
        for (int i = 1; i < 8; ++i) acc += sum[i][c];
        dg[k] = acc;
    }
}

int64_t bwd_parts(int64_t M) { return M < kBwdParts ? M : kBwdParts; }

template <int kBytes>
bool aligned_to(const void *p) { return (reinterpret_cast<uintptr_t>(p) & (kBytes - 1)) == 0; }

}  // namespace

// Partial rows of dg.
size_t jet_add_rmsnorm_bwd_workspace(int64_t M, int64_t K) {
    return (size_t)bwd_parts(M) * (size_t)K * sizeof(float);
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
                           dim3(kAnThreads), 0, jet::as_stream(stream), x, d, g, M, K, eps, h, q,
                           s, rstd);
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
    const int parts = (int)bwd_parts(M);
    const int64_t nchunks = K / 8;
    const int nc = nchunks <= 1024 ? 1 : nchunks <= 2048 ? 2 : 4;
    const int threads = (int)(((nchunks + nc - 1) / nc + 31) / 32 * 32);
    auto *kernel = nc == 1 ? add_rmsnorm_bwd_kernel<1>
                           : nc == 2 ? add_rmsnorm_bwd_kernel<2> : add_rmsnorm_bwd_kernel<4>;
    float *part = static_cast<float *>(ws);
    st = jet::launch_pdl(kernel, dim3((unsigned)parts), dim3((unsigned)threads), 0, cs, h, g, rstd,
                         dy0, dy1, dy2, dres, M, K, dx, part);
    if (st != JET_OK) return st;
    return jet::launch_pdl(dgain_reduce_kernel, dim3((unsigned)(K / 32)), dim3(256), 0, cs, part,
                           parts, K, dg);
}
