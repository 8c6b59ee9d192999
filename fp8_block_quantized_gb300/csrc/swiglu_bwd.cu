// Backward of the gated activation h = silu(gate) up, with the 1x128
// quantization of both gradients fused: the inputs of the gate and up
// projections' DGrads, without BF16 gradients in between.  With s = 1 / (1 +
// e^-g):
//   dup = dh g s,   dgate = dh up s (1 + g (1 - s)).
// With t = e^-g, s = 1 / (1 + t) and 1 - s = t s, so neither cancels; t is one exp2 of
// a binary32 product (relative error 2^-22 + |g| 2^-24) held below 2^127, the
// reciprocal approximation's error 2^-23; where s would be below 2^-126 it is 0.  Then
// the 1x128 group rule of quant_rule.cuh on the binary32 values.
//
// Work is split as in the forward's quantizer: half a warp takes a group of 128
// (8 elements a lane, one 16-byte load of each tensor), a warp two neighbouring
// groups of a row, consecutive warps consecutive rows; the next item's loads go
// out before an item's arithmetic.
//
// What bounds it: 8.06 bytes an element; 8192 x 14336 takes 168 us, 5.6 TB/s of the 6.8 of a
// copy, with 39 warp instructions for 32 elements in 69% of the issue slots.  Five CTAs an SM spill
// (178 us).  128 x 1024 is a launch and one round of loads, 2.2 us in a graph.
#include <cuda_bf16.h>

#include "jet_common.cuh"
#include "stream_ld.cuh"
#include "quant_rule.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kCtasPerSm = 4;

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 unpack(uint32_t w) { return make_float2(lo(w), hi(w)); }

// -dgate and -dup of two elements, for the division routine, in packed arithmetic
__device__ __forceinline__ void neg_gradients(uint32_t g, uint32_t u, uint32_t d, float *ng, float *nu) {
    const float2 m = unpack(g ^ 0x80008000u), dh = unpack(d);  // m = -g
    const float2 x = __fmul2_rn(m, both(1.4426950408889634f));
    float2 t, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t.x) : "f"(fminf(x.x, 127.0f)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t.y) : "f"(fminf(x.y, 127.0f)));
    const float2 q = __fadd2_rn(t, both(1.0f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(q.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(q.y));
    const float2 ds = __fmul2_rn(dh, s);
    const float2 a = __fmul2_rn(ds, m);
    const float2 f = __ffma2_rn(m, __fmul2_rn(t, s), both(-1.0f));  // -(1 + g (1 - s))
    const float2 b = __fmul2_rn(__fmul2_rn(ds, unpack(u)), f);
    nu[0] = a.x, nu[1] = a.y, ng[0] = b.x, ng[1] = b.y;
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm)
swiglu_bwd_kernel(const uint16_t *__restrict__ gate, const uint16_t *__restrict__ up, int64_t ld,
                  const uint16_t *__restrict__ dh, int64_t M, int64_t F, uint8_t *__restrict__ qg,
                  float *__restrict__ sg, uint8_t *__restrict__ qu, float *__restrict__ su) {
    jet::griddep_launch_dependents();
    jet::griddep_wait();
    const int lane = threadIdx.x & 31, half = lane >> 4, j = lane & 15;
    const int64_t nfb = F / 128, npairs = (nfb + 1) / 2;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    // item t = (pair p, row m), t = p M + m, walked without a division
    const int64_t t0 = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t dp = warps / M, dm = warps % M;
    int64_t p = t0 / M, m = t0 % M;
    auto load = [&](int64_t p_, int64_t m_, uint4 (&v)[3]) {
        const int64_t fb = 2 * p_ + half;
        if (p_ < npairs && fb < nfb) {
            const int64_t col = fb * 128 + 8 * j;
            v[0] = ld_stream16(gate + m_ * ld + col);
            v[1] = ld_stream16(up + m_ * ld + col);
            v[2] = ld_stream16(dh + m_ * F + col);
        }
    };
    uint4 cur[3] = {};
    load(p, m, cur);
    while (p < npairs) {
        const int64_t fb = 2 * p + half;
        int64_t p2 = p + dp, m2 = m + dm;
        if (m2 >= M) {
            m2 -= M;
            ++p2;
        }
        uint4 nxt[3] = {};
        load(p2, m2, nxt);
        const uint32_t g[4] = {cur[0].x, cur[0].y, cur[0].z, cur[0].w},
                       u[4] = {cur[1].x, cur[1].y, cur[1].z, cur[1].w},
                       d[4] = {cur[2].x, cur[2].y, cur[2].z, cur[2].w};
        float ng[8], nu[8], ag = 0.0f, au = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            neg_gradients(g[i], u[i], d[i], ng + 2 * i, nu + 2 * i);
            ag = max_abs2(ag, ng[2 * i], ng[2 * i + 1]);
            au = max_abs2(au, nu[2 * i], nu[2 * i + 1]);
        }
        // the first eight lanes of a group take dgate's maximum, scale and reciprocal, the
        // others dup's
        const bool second = j >= 8;
        float amax = fmaxf(second ? au : ag, __shfl_xor_sync(~0u, second ? ag : au, 8));
#pragma unroll
        for (int off = 4; off >= 1; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, off));
        const Divisor mine = make_divisor(group_scale(amax));
        Divisor d0, d1;
        d0.s = __shfl_sync(~0u, mine.s, 0, 16), d1.s = __shfl_sync(~0u, mine.s, 8, 16);
        d0.ny = __shfl_sync(~0u, mine.ny, 0, 16), d1.ny = __shfl_sync(~0u, mine.ny, 8, 16);
        d0.fast = d0.ny != 0.0f, d1.fast = d1.ny != 0.0f;
        if (fb < nfb) {
            const int64_t at = m * F + fb * 128 + 8 * j;
            *reinterpret_cast<uint2 *>(qg + at) = make_uint2(encode4(ng, d0), encode4(ng + 4, d0));
            *reinterpret_cast<uint2 *>(qu + at) = make_uint2(encode4(nu, d1), encode4(nu + 4, d1));
            if ((j & 7) == 0) (second ? su : sg)[fb * M + m] = mine.s;
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) cur[i] = nxt[i];
        p = p2;
        m = m2;
    }
}

}  // namespace

jet_status jet_swiglu_bwd_quant_1x128(const uint16_t *gate, const uint16_t *up, int64_t ld,
                                      const uint16_t *dh, int64_t M, int64_t F, uint8_t *qg,
                                      float *sg, uint8_t *qu, float *su, jet_stream_t stream) {
    JET_REQUIRE(M >= 0 && F >= 0 && ld >= F, JET_ERR_SHAPE);
    const bool empty = M == 0 || F == 0;
    JET_REQUIRE(empty || (gate && up && dh && qg && sg && qu && su), JET_ERR_NULL);
    JET_REQUIRE(F % 128 == 0 && M < (int64_t)1 << 31 && ld < (int64_t)1 << 40, JET_ERR_SHAPE);
    JET_REQUIRE(ld % 8 == 0 && jet::aligned16(gate) && jet::aligned16(up) && jet::aligned16(dh) &&
                    jet::aligned16(qg) && jet::aligned16(sg) && jet::aligned16(qu) &&
                    jet::aligned16(su),
                JET_ERR_ALIGN);
    jet::DeviceInfo dev;
    const jet_status st = jet::current_device(&dev);
    if (st != JET_OK) return st;
    if (empty) return JET_OK;
    const int64_t items = M * ((F / 128 + 1) / 2);
    const int64_t want = (items + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t cap = (int64_t)dev.num_sms * kCtasPerSm;
    return jet::launch_pdl(swiglu_bwd_kernel, dim3((unsigned)(want < cap ? want : cap)),
                           dim3(kThreads), 0, jet::as_stream(stream), gate, up, ld, dh, M, F, qg,
                           sg, qu, su);
}
