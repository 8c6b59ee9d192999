// Rotary positions of q and k (jet_rope, forward and backward), and the same
// rotation fused with the FP8 KV-cache write (jet_rope_kv_cache_write).
//
// Channel pair i of a head (the first R of its D channels; pairs (i, i + R/2)
// in the half layout, (2 i, 2 i + 1) in the interleaved one) is turned by the
// angle pos * f_i and scaled by mscale:
//   y_a = a cos - b sin,  y_b = b cos + a sin;
// channels R .. D-1 pass through.  The backward turns by the negative angle.
//
// Angles: pos * f_i reaches 10^6 radians and more in long contexts, where a
// binary32 product keeps no fraction.  Here f_i / (2 pi) is held as a 64-bit
// binary fraction of a turn, so pos * fraction modulo 2^64 is the angle modulo
// a whole turn, in integer arithmetic with an error below |pos| 2^-54 turns (the
// binary64 product) at any position; its top 32 bits, as a signed half-turn count,
// go to sincospi in binary32.
//
// Bound by HBM: every input is read once and every output written once, 16 bytes
// at a time (8192 tokens of 32 + 8 heads of 128: 26.9 us, 6229 GB/s, 92% of a
// copy's rate; with the cache write, 16384 tokens of 64 + 8 + 8 heads: 98.8 us,
// 6453 GB/s, 95%).  Few tokens: latency (64 tokens of 32 + 8 + 8 heads 3.6 us).
#include <algorithm>
#include <cmath>

#include "jet_common.cuh"
#include "quant_rule.cuh"

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxD = 1024;
constexpr int kRopeBatch = 4;  // heads per thread at most (one set of angles)

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two binary32 values rounded to BF16 (nearest, ties to even), a in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// The fraction of a turn per position, times 2^64.
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
    double t = f * 0.15915494309189533577;  // 1 / (2 pi)
    t -= floor(t);
    return __double2ull_rn(t * 18446744073709551616.0);
}

__device__ __forceinline__ void angle(unsigned long long frac, int64_t pos, float mscale,
                                      bool backward, float &c, float &s) {
    const unsigned long long p = frac * (unsigned long long)pos;
    const float half_turns = __int2float_rn((int)(p >> 32)) * 0x1p-31f;
    sincospif(half_turns, &s, &c);
    c *= mscale;
    s *= backward ? -mscale : mscale;
}

struct RopeArgs {
    const uint16_t *q, *k, *v;
    int64_t ldq, ldk, ldv;
    int Hq, Hk, Hv, D, R;
    int64_t T;
    const double *freq;
    const int64_t *pos;
    float mscale;
    int backward;
    uint16_t *qo, *ko;
    int64_t ldqo, ldko;
    // KV-cache form
    const float *ks, *vs;
    const int64_t *slots;
    uint8_t *kc, *vc;
    int64_t S;
    // split of the work: T * groups * items threads, or T * groups tiles, of hpt heads
    int groups, items, hpt;
    int by[4];  // rope_any_kernel's divisions
};

// One head's place: where it is read and where its result goes.
struct Head {
    const uint16_t *in;
    uint16_t *out;   // BF16 output, or null
    uint8_t *code;   // cache entry, or null
    float scale;
    bool rotate;
};

template <bool kCache>
__device__ __forceinline__ Head head_of(const RopeArgs &a, int64_t t, int h, int64_t slot) {
    Head r;
    r.out = nullptr;
    r.code = nullptr;
    r.scale = 1.0f;
    r.rotate = true;
    if (h < a.Hq) {
        r.in = a.q + t * a.ldq + (int64_t)h * a.D;
        r.out = a.qo + t * a.ldqo + (int64_t)h * a.D;
        return r;
    }
    h -= a.Hq;
    const bool is_v = kCache && h >= a.Hk;
    if (is_v) h -= a.Hk;
    r.rotate = !is_v;
    r.in = (is_v ? a.v + t * a.ldv : a.k + t * a.ldk) + (int64_t)h * a.D;
    if (kCache) {
        if (slot >= 0 && slot < a.S) {
            r.code = (is_v ? a.vc : a.kc) + (slot * a.Hk + h) * a.D;
            r.scale = (is_v ? a.vs : a.ks)[h];
        }
    } else {
        r.out = a.ko + t * a.ldko + (int64_t)h * a.D;
    }
    return r;
}

// Eight BF16 values (packed) to where a head's chunk at channel d goes.
template <bool kCache>
__device__ __forceinline__ void store8(const Head &hd, int d, const uint4 &y) {
    if (!kCache || hd.out) {
        *reinterpret_cast<uint4 *>(hd.out + d) = y;
    } else if (hd.code) {
        const Divisor dv = make_divisor(hd.scale);
        const uint32_t w[4] = {y.x, y.y, y.z, y.w};
        float nf[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            nf[2 * i] = __uint_as_float((w[i] << 16) ^ 0x80000000u);
            nf[2 * i + 1] = __uint_as_float((w[i] & 0xFFFF0000u) ^ 0x80000000u);
        }
        *reinterpret_cast<uint2 *>(hd.code + d) = make_uint2(encode4(nf, dv), encode4(nf + 4, dv));
    }
}

// Half layout, one pair of words: x holds channels i, i+1 of the first half,
// y those of the second.
__device__ __forceinline__ void turn_half(uint32_t &x, uint32_t &y, const float *c, const float *s) {
    const float a0 = bf16_lo(x), a1 = bf16_hi(x), b0 = bf16_lo(y), b1 = bf16_hi(y);
    x = pack_bf16(__fmaf_rn(a0, c[0], -__fmul_rn(b0, s[0])), __fmaf_rn(a1, c[1], -__fmul_rn(b1, s[1])));
    y = pack_bf16(__fmaf_rn(b0, c[0], __fmul_rn(a0, s[0])), __fmaf_rn(b1, c[1], __fmul_rn(a1, s[1])));
}

__device__ __forceinline__ uint32_t turn_pair(uint32_t x, float c, float s) {
    const float a = bf16_lo(x), b = bf16_hi(x);
    return pack_bf16(__fmaf_rn(a, c, -__fmul_rn(b, s)), __fmaf_rn(b, c, __fmul_rn(a, s)));
}

// Interleaved layout, the first `pairs` pairs of a chunk.
__device__ __forceinline__ void turn_chunk(uint4 &x, const float *c, const float *s, int pairs) {
    if (pairs > 0) x.x = turn_pair(x.x, c[0], s[0]);
    if (pairs > 1) x.y = turn_pair(x.y, c[1], s[1]);
    if (pairs > 2) x.z = turn_pair(x.z, c[2], s[2]);
    if (pairs > 3) x.w = turn_pair(x.w, c[3], s[3]);
}

// A thread takes one item of up to kRopeBatch heads of one token, so that their
// loads are in flight together and share one set of angles.  Items of a head:
// kHalf (R % 16 == 0): R/16 pairs of 8-channel chunks (c, c + R/16), then the
// chunks past R in twos; interleaved (any R): chunks (c, c + n) of 2n or 2n - 1,
// so that a warp's lanes turn alike where half of the channels turn.
// kBatch heads at a time: all of them, or two with the registers of four CTAs an
// SM (the cache form of many tokens, whose encoding keeps the SMs busy: 16384
// tokens of 64 + 8 + 8 heads 98 us, 110 with four; without a cache 8192 tokens
// of 32 + 8 heads 28.4 with two, 27.3 with four).
template <bool kHalf, bool kCache, int kBatch>
__global__ void __launch_bounds__(kRopeThreads, kBatch < kRopeBatch ? 4 : 0)
rope_kernel(const RopeArgs a) {
    extern __shared__ unsigned long long frac[];  // [R/2]
    jet::griddep_launch_dependents();
    jet::griddep_wait();
    for (int i = threadIdx.x; i < a.R / 2; i += kRopeThreads) frac[i] = turn_fraction(a.freq[i]);
    __syncthreads();
    const int nrot = a.R / 16;  // half layout
    const int heads = a.Hq + a.Hk + a.Hv;
    const uint32_t per_token = (uint32_t)a.groups * a.items;
    const uint32_t total = (uint32_t)a.T * per_token;
    const bool inplace = !kCache && a.q == a.qo && a.k == a.ko;
    for (uint64_t idx = blockIdx.x * (uint64_t)kRopeThreads + threadIdx.x; idx < total;
         idx += (uint64_t)gridDim.x * kRopeThreads) {
        const uint32_t t = (uint32_t)idx / per_token, rest = (uint32_t)idx - t * per_token;
        const uint32_t grp = rest / a.items;
        const int item = (int)(rest - grp * a.items);
        // the item's chunks, at channels d0 and d1, and the pairs of each that turn
        // (half layout: the pairs between the two)
        const int d0 = !kHalf ? 8 * item : item < nrot ? 8 * item : a.R + 16 * (item - nrot);
        const int d1 = !kHalf ? 8 * (item + a.items) : item < nrot ? a.R / 2 + 8 * item : d0 + 8;
        const bool both = d1 < a.D;
        const int rot0 = kHalf ? (item < nrot ? 8 : 0) : min(max((a.R - d0) / 2, 0), 4);
        const int rot1 = kHalf ? 0 : min(max((a.R - d1) / 2, 0), 4);
        if (rot0 == 0 && inplace) continue;
        const int h0 = (int)grp * a.hpt, h1 = min(h0 + a.hpt, heads);
        const int64_t slot = kCache ? a.slots[t] : 0;
        float c[8], s[8];
#pragma unroll 1
        for (int hb = h0; hb < h1; hb += kBatch) {
            uint4 x[kBatch], y[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (hb + b >= h1) break;
                const Head hd = head_of<kCache>(a, t, hb + b, -1);
                x[b] = *reinterpret_cast<const uint4 *>(hd.in + d0);
                if (both) y[b] = *reinterpret_cast<const uint4 *>(hd.in + d1);
            }
            if (rot0 > 0 && hb == h0) {
                const int64_t pos = a.pos[t];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (kHalf || i < rot0 || (i >= 4 && i - 4 < rot1))
                        angle(frac[kHalf ? 8 * item + i : i < 4 ? d0 / 2 + i : d1 / 2 + i - 4], pos, a.mscale,
                              a.backward, c[i], s[i]);
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (hb + b >= h1) break;
                const Head hd = head_of<kCache>(a, t, hb + b, slot);
                if (rot0 > 0 && hd.rotate) {
                    if constexpr (kHalf) {
                        turn_half(x[b].x, y[b].x, c, s);
                        turn_half(x[b].y, y[b].y, c + 2, s + 2);
                        turn_half(x[b].z, y[b].z, c + 4, s + 4);
                        turn_half(x[b].w, y[b].w, c + 6, s + 6);
                    } else {
                        turn_chunk(x[b], c, s, rot0);
                        turn_chunk(y[b], c + 4, s + 4, rot1);
                    }
                }
                store8<kCache>(hd, d0, x[b]);
                if (both) store8<kCache>(hd, d1, y[b]);
            }
            if (kBatch == kRopeBatch) break;  // all of them
        }
    }
}

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     (unsigned)__cvta_generic_to_shared(dst)),
                 "l"(src)
                 : "memory");
}

// The half layout where the second half starts inside a 16-byte chunk.  A CTA
// takes whole heads of one token, about kAnyChunks chunks of them: those that hold
// turned channels go to shared memory while the CTA computes the token's angles
// once and copies the others, a thread then turns single pairs there, and chunks
// go out (8192 tokens of 32 + 8 heads of 128, 34 turned: 34 us, 63 channel by
// channel; with the cache write 44 and 102).
constexpr int kAnyChunks = 1024;

// The CTA's threads over `per` items of each head: this thread's first (head,
// item) and the step to its next, without divisions (by is 2^16 / per, rounded
// up: exact for the quotients of 0 .. 255, and of 256 up to per = 256).
struct Walk {
    int per, h0, i0, dh, di;
    __device__ Walk(int n, int by) : per(n) {
        h0 = n > 0 ? ((int)threadIdx.x * by) >> 16 : 1 << 30;
        i0 = (int)threadIdx.x - h0 * n;
        dh = n > kRopeThreads ? 0 : (kRopeThreads * by) >> 16;
        di = kRopeThreads - dh * n;
    }
    template <typename F>
    __device__ __forceinline__ void over(int heads, F f) const {
        int h = h0, i = i0;
#pragma unroll 1
        while (h < heads) {
            f(h, i);
            h += dh;
            i += di;
            if (i >= per) {
                i -= per;
                ++h;
            }
        }
    }
};

template <bool kCache>
__global__ void __launch_bounds__(kRopeThreads, 8)
rope_any_kernel(const RopeArgs a) {
    extern __shared__ uint4 tile[];  // [hpt][R8], then the fractions and angles [R / 2]
    const int R2 = a.R / 2, R8 = (a.R + 7) / 8, rest = a.D / 8 - R8, heads = a.Hq + a.Hk + a.Hv;
    unsigned long long *frac = reinterpret_cast<unsigned long long *>(tile + a.hpt * R8);
    float2 *cs = reinterpret_cast<float2 *>(frac + R2);
    jet::griddep_launch_dependents();
    jet::griddep_wait();
    for (int i = threadIdx.x; i < R2; i += kRopeThreads) frac[i] = turn_fraction(a.freq[i]);
    const bool inplace = !kCache && a.q == a.qo && a.k == a.ko;
    const Walk chunks(R8, a.by[0]), pairs(R2, a.by[1]), others(inplace ? 0 : rest, a.by[2]),
        whole(R8 + rest, a.by[3]);
    for (int64_t unit = blockIdx.x; unit < a.T * a.groups; unit += gridDim.x) {
        const int64_t t = unit / a.groups;
        const int h0 = (int)(unit - t * a.groups) * a.hpt;
        const int n = min(a.hpt, heads - h0), turned = min(n, max(a.Hq + a.Hk - h0, 0));
        const int64_t pos = a.pos[t], slot = kCache ? a.slots[t] : 0;
        __syncthreads();  // the last unit's tile and angles have been read
        chunks.over(turned, [&](int h, int i) {
            cp_async16(tile + h * R8 + i, head_of<kCache>(a, t, h0 + h, -1).in + 8 * i);
        });
        asm volatile("cp.async.commit_group;" ::: "memory");
        auto copy = [&](int h, int i) {
            const Head hd = head_of<kCache>(a, t, h0 + h, slot);
            store8<kCache>(hd, 8 * i, *reinterpret_cast<const uint4 *>(hd.in + 8 * i));
        };
        others.over(turned, [&](int h, int i) { copy(h, R8 + i); });
        if (kCache) whole.over(n - turned, [&](int h, int i) { copy(turned + h, i); });
        for (int i = threadIdx.x; i < R2; i += kRopeThreads) {
            float c, s;
            angle(frac[i], pos, a.mscale, a.backward, c, s);
            cs[i] = make_float2(c, s);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        pairs.over(turned, [&](int h, int i) {
            uint16_t *row = reinterpret_cast<uint16_t *>(tile + h * R8);
            const float2 f = cs[i];
            const uint32_t w = turn_pair(row[i] | ((uint32_t)row[i + R2] << 16), f.x, f.y);
            row[i] = (uint16_t)w;
            row[i + R2] = (uint16_t)(w >> 16);
        });
        __syncthreads();
        chunks.over(turned, [&](int h, int i) {
            store8<kCache>(head_of<kCache>(a, t, h0 + h, slot), 8 * i, tile[h * R8 + i]);
        });
    }
}

jet_status rope_launch(RopeArgs a, int layout, bool cache, const jet::DeviceInfo &dev,
                       jet_stream_t stream) {
    const bool half = layout == JET_ROPE_HALF;
    const int64_t sms = dev.num_sms;
    const int heads = a.Hq + a.Hk + a.Hv;
    if (half && a.R % 16 != 0) {
        // heads of kAnyChunks chunks a CTA, fewer while there are not two CTAs an SM
        // (of 64 chunks at least; 300 tokens of 32 + 8 heads 3.2 us, 3.5 with four)
        a.hpt = std::max(1, std::min(heads, kAnyChunks / (a.D / 8)));
        while (a.hpt > 1 && a.hpt * a.D > 8 * 64 && a.T * ((heads + a.hpt - 1) / a.hpt) < 2 * sms)
            a.hpt = (a.hpt + 1) / 2;
        a.groups = (heads + a.hpt - 1) / a.hpt;
        const int per[4] = {(a.R + 7) / 8, a.R / 2, a.D / 8 - (a.R + 7) / 8, a.D / 8};
        for (int i = 0; i < 4; ++i) a.by[i] = per[i] ? (65536 + per[i] - 1) / per[i] : 0;
        const int64_t want = a.T * a.groups, cap = 24 * sms;
        return jet::launch_pdl(cache ? rope_any_kernel<true> : rope_any_kernel<false>,
                               dim3((unsigned)(want < cap ? want : cap)), dim3(kRopeThreads),
                               (size_t)a.hpt * ((a.R + 7) / 8) * 16 + (size_t)a.R / 2 * 16,
                               jet::as_stream(stream), a);
    }
    a.items = half ? a.R / 16 + (a.D - a.R + 15) / 16 : (a.D + 15) / 16;
    // More heads per thread share one set of angles; fewer keep the SMs busy
    // when there are few tokens (with less than 512 items an SM: 1000 tokens of
    // 32 + 8 heads 6.4 us with four heads, 8.8 with one; 256 tokens 3.5 with one).
    a.hpt = kRopeBatch;
    while (a.hpt > 1 && a.T * ((heads + a.hpt - 1) / a.hpt) * a.items < sms * 512)
        a.hpt /= 2;
    a.groups = (heads + a.hpt - 1) / a.hpt;
    // Twice the resident CTAs (3 per SM; 8192 tokens of 32 + 8 heads 27 us with 6
    // per SM, 29 with 3).  With a cache, items that 3 CTAs an SM cannot hold at
    // once go to the kernel of pairs, with the 4 that are resident (1000 tokens of
    // 32 + 8 + 8 heads 8.3 us, 9.4 in pairs; 1500 tokens 9.7 in pairs, 12.4 without).
    const bool pairs = cache && a.hpt == kRopeBatch &&
                       a.T * a.groups * a.items > 3 * kRopeThreads * sms;
    const int64_t cap = sms * (pairs ? 4 : 6);
    void (*kernel)(RopeArgs) =
        pairs ? (half ? rope_kernel<true, true, 2> : rope_kernel<false, true, 2>)
        : half ? (cache ? rope_kernel<true, true, kRopeBatch> : rope_kernel<true, false, kRopeBatch>)
               : (cache ? rope_kernel<false, true, kRopeBatch> : rope_kernel<false, false, kRopeBatch>);
    // The kernels count a launch's items in 32 bits: more tokens take several launches.
    const int64_t all = a.T, most = (((int64_t)1 << 32) - 1) / ((int64_t)a.groups * a.items);
    for (int64_t t0 = 0; t0 < all; t0 += most) {
        a.T = all - t0 < most ? all - t0 : most;
        const int64_t want = (a.T * a.groups * a.items + kRopeThreads - 1) / kRopeThreads;
        const jet_status st = jet::launch_pdl(
            kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(kRopeThreads),
            (size_t)a.R / 2 * sizeof(unsigned long long), jet::as_stream(stream), a);
        if (st != JET_OK) return st;
        auto step = [&](const uint16_t *&p, int64_t ld) { p = p ? p + most * ld : p; };
        step(a.q, a.ldq);
        step(a.k, a.ldk);
        step(a.v, a.ldv);
        a.qo = a.qo ? a.qo + most * a.ldqo : a.qo;
        a.ko = a.ko ? a.ko + most * a.ldko : a.ko;
        a.pos += most;
        a.slots = a.slots ? a.slots + most : a.slots;
    }
    return JET_OK;
}

// Sizes both entry points share.
bool rope_sizes_ok(int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t R, int layout) {
    return T < ((int64_t)1 << 31) && Hq <= 1024 && Hk <= 1024 && D <= kRopeMaxD && D % 8 == 0 &&
           R >= 0 && R <= D && R % 2 == 0 &&
           (layout == JET_ROPE_HALF || layout == JET_ROPE_INTERLEAVED);
}

bool ld_ok(int64_t ld, int64_t H, int64_t D) { return ld >= H * D && ld < ((int64_t)1 << 40); }

// In place with another stride, a token would be written before it is read.
bool in_place_ok(const uint16_t *in, int64_t ld, const uint16_t *out, int64_t ldo, int64_t T) {
    return in != out || ld == ldo || T <= 1;
}

template <int kBytes>
bool aligned_to(const void *p) { return (reinterpret_cast<uintptr_t>(p) & (kBytes - 1)) == 0; }

}  // namespace

jet_status jet_rope(const uint16_t *q, int64_t ldq, int64_t Hq, const uint16_t *k, int64_t ldk,
                    int64_t Hk, int64_t T, int64_t D, int64_t R, const double *inv_freq,
                    const int64_t *pos, int layout, float mscale, int backward, uint16_t *qo,
                    int64_t ldqo, uint16_t *ko, int64_t ldko, jet_stream_t stream) {
    JET_REQUIRE(T >= 0 && Hq >= 0 && Hk >= 0 && D >= 0, JET_ERR_SHAPE);
    const bool hasq = T > 0 && D > 0 && Hq > 0, hask = T > 0 && D > 0 && Hk > 0;
    JET_REQUIRE((!hasq || (q && qo)) && (!hask || (k && ko)), JET_ERR_NULL);
    JET_REQUIRE((!hasq && !hask) || (pos && (R <= 0 || inv_freq)), JET_ERR_NULL);
    JET_REQUIRE(rope_sizes_ok(T, Hq, Hk, D, R, layout), JET_ERR_SHAPE);
    JET_REQUIRE(!hasq || (ld_ok(ldq, Hq, D) && ld_ok(ldqo, Hq, D) && in_place_ok(q, ldq, qo, ldqo, T)),
                JET_ERR_SHAPE);
    JET_REQUIRE(!hask || (ld_ok(ldk, Hk, D) && ld_ok(ldko, Hk, D) && in_place_ok(k, ldk, ko, ldko, T)),
                JET_ERR_SHAPE);
    JET_REQUIRE(!hasq || (ldq % 8 == 0 && ldqo % 8 == 0 && jet::aligned16(q) && jet::aligned16(qo)),
                JET_ERR_ALIGN);
    JET_REQUIRE(!hask || (ldk % 8 == 0 && ldko % 8 == 0 && jet::aligned16(k) && jet::aligned16(ko)),
                JET_ERR_ALIGN);
    JET_REQUIRE(aligned_to<8>(pos) && aligned_to<8>(inv_freq), JET_ERR_ALIGN);
    jet::DeviceInfo dev;
    jet_status st = jet::current_device(&dev);
    if (st != JET_OK) return st;
    if (!hasq && !hask) return JET_OK;
    RopeArgs a = {};
    a.q = q;
    a.k = k;
    a.ldq = ldq;
    a.ldk = ldk;
    a.Hq = (int)Hq;
    a.Hk = (int)Hk;
    a.D = (int)D;
    a.R = (int)R;
    a.T = T;
    a.freq = inv_freq;
    a.pos = pos;
    a.mscale = mscale;
    a.backward = backward != 0;
    a.qo = qo;
    a.ko = ko;
    a.ldqo = ldqo;
    a.ldko = ldko;
    return rope_launch(a, layout, false, dev, stream);
}

jet_status jet_rope_kv_cache_write(const uint16_t *q, int64_t ldq, int64_t Hq, const uint16_t *k,
                                   int64_t ldk, const uint16_t *v, int64_t ldv, int64_t Hk,
                                   int64_t T, int64_t D, int64_t R, const double *inv_freq,
                                   const int64_t *pos, int layout, float mscale,
                                   const float *k_scale, const float *v_scale,
                                   const int64_t *slots, uint16_t *qo, int64_t ldqo,
                                   uint8_t *k_cache, uint8_t *v_cache, int64_t S,
                                   jet_stream_t stream) {
    JET_REQUIRE(T >= 0 && Hq >= 0 && Hk >= 0 && D >= 0 && S >= 0, JET_ERR_SHAPE);
    const bool hasq = T > 0 && D > 0 && Hq > 0, hask = T > 0 && D > 0 && Hk > 0;
    JET_REQUIRE(!hasq || (q && qo), JET_ERR_NULL);
    JET_REQUIRE(!hask || (k && v && k_scale && v_scale && slots && (S == 0 || (k_cache && v_cache))),
                JET_ERR_NULL);
    JET_REQUIRE((!hasq && !hask) || (pos && (R <= 0 || inv_freq)), JET_ERR_NULL);
    JET_REQUIRE(rope_sizes_ok(T, Hq, Hk, D, R, layout) && D % 16 == 0 && S < ((int64_t)1 << 40),
                JET_ERR_SHAPE);
    JET_REQUIRE(!hasq || (ld_ok(ldq, Hq, D) && ld_ok(ldqo, Hq, D) && in_place_ok(q, ldq, qo, ldqo, T)),
                JET_ERR_SHAPE);
    JET_REQUIRE(!hask || (ld_ok(ldk, Hk, D) && ld_ok(ldv, Hk, D)), JET_ERR_SHAPE);
    JET_REQUIRE(!hasq || (ldq % 8 == 0 && ldqo % 8 == 0 && jet::aligned16(q) && jet::aligned16(qo)),
                JET_ERR_ALIGN);
    JET_REQUIRE(!hask || (ldk % 8 == 0 && ldv % 8 == 0 && jet::aligned16(k) && jet::aligned16(v) &&
                          aligned_to<4>(k_scale) && aligned_to<4>(v_scale) &&
                          aligned_to<8>(slots) && jet::aligned16(k_cache) &&
                          jet::aligned16(v_cache)),
                JET_ERR_ALIGN);
    JET_REQUIRE(aligned_to<8>(pos) && aligned_to<8>(inv_freq), JET_ERR_ALIGN);
    jet::DeviceInfo dev;
    jet_status st = jet::current_device(&dev);
    if (st != JET_OK) return st;
    if (!hasq && !hask) return JET_OK;
    RopeArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.ldq = ldq;
    a.ldk = ldk;
    a.ldv = ldv;
    a.Hq = (int)Hq;
    a.Hk = (int)Hk;
    a.Hv = (int)Hk;
    a.D = (int)D;
    a.R = (int)R;
    a.T = T;
    a.freq = inv_freq;
    a.pos = pos;
    a.mscale = mscale;
    a.qo = qo;
    a.ldqo = ldqo;
    a.ks = k_scale;
    a.vs = v_scale;
    a.slots = slots;
    a.kc = k_cache;
    a.vc = v_cache;
    a.S = S;
    return rope_launch(a, layout, hask, dev, stream);  // no heads to cache: slots may be null
}

jet_status jet_rope_inv_freq(int64_t R, double base, int scaling, double factor, double context,
                             double low, double high, double *inv_freq, float *mscale) {
    JET_REQUIRE(inv_freq && mscale, JET_ERR_NULL);
    JET_REQUIRE(R >= 2 && R <= kRopeMaxD && R % 2 == 0 && base > 1.0 && base <= 1e300,
                JET_ERR_SHAPE);
    const bool blend = scaling == JET_ROPE_SCALE_WAVELENGTH || scaling == JET_ROPE_SCALE_RAMP;
    JET_REQUIRE(blend || scaling == JET_ROPE_SCALE_NONE || scaling == JET_ROPE_SCALE_LINEAR,
                JET_ERR_SHAPE);
    JET_REQUIRE(scaling == JET_ROPE_SCALE_NONE || (factor > 0.0 && factor <= 1e300), JET_ERR_SHAPE);
    JET_REQUIRE(!blend || (context > 0.0 && context <= 1e300 && low > 0.0 && high > low &&
                           high <= 1e300),
                JET_ERR_SHAPE);
    constexpr double kTwoPi = 6.28318530717958647693;
    double from = 0.0, to = 0.0;
    if (scaling == JET_ROPE_SCALE_RAMP) {
        const double last = (double)(R - 1);
        from = std::floor((double)R * std::log(context / (kTwoPi * high)) / (2.0 * std::log(base)));
        to = std::ceil((double)R * std::log(context / (kTwoPi * low)) / (2.0 * std::log(base)));
        from = std::fmin(std::fmax(from, 0.0), last);
        to = std::fmin(std::fmax(to, 0.0), last);
        if (to <= from) to = from + 0.001;  // a step
    }
    for (int64_t i = 0; i < R / 2; ++i) {
        double f = std::pow(base, -2.0 * (double)i / (double)R);
        if (scaling == JET_ROPE_SCALE_LINEAR) {
            f /= factor;
        } else if (blend) {
            const double s = scaling == JET_ROPE_SCALE_WAVELENGTH
                                 ? (high - context * f / kTwoPi) / (high - low)
                                 : ((double)i - from) / (to - from);
            const double c = std::fmin(std::fmax(s, 0.0), 1.0);
            f *= 1.0 - c + c / factor;
        }
        inv_freq[i] = f;
    }
    *mscale = scaling == JET_ROPE_SCALE_RAMP && factor > 1.0
                  ? (float)(1.0 + 0.1 * std::log(factor)) : 1.0f;
    return JET_OK;
}
