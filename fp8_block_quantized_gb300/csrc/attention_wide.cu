// Attention over the paged FP8 cache for many rows a KV head: chunks of a prompt,
// and prefixes that a group of requests shares.  The mathematics, the segments
// and the deal of the key tiles are those of attention.cu; here a tile is two
// 128 x 128 score products on the 5th-generation tensor core.
//
// One CTA an SM, 20 warps:
//   warps 0-3, 4-7  two halves (A, B), one thread a row: the row's query to FP16 in
//                   shared memory, then for every tile its scores from TMEM, their
//                   maximum, weights e^(x - max) as FP16 back to TMEM over the
//                   scores (handed on 64 keys at a time), and at a piece's end its
//                   output;
//   warps 8-15      the tiles' codes, four warps a stage: read through the block table
//                   into registers two tiles ahead (64 KB in flight), turned to FP16
//                   (exact) and laid out in shared memory, K and V alike as rows of
//                   keys with the 128-byte swizzle: K-major for the scores, MN-major
//                   for the values;
//   warps 16, 17    issue the MMAs of A and of B: scores S = Q K^T (both operands in
//                   shared memory) and O += P V (P in TMEM);
//   warp 18         walks the CTA's range and tells the others its pieces.
// In a wide unit A and B are the two halves of 256 rows at the same keys; a unit
// of at most 128 rows has them at alternate tiles of the same rows, whose results
// are added at the end.  While one half's weights are computed the tensor core
// works for the other.  A row's output is rescaled in TMEM only when its maximum
// has grown by more than 2^8 since the last time.  The weights' reference lies 2^7 below
// the maximum at that time: weights reach 2^15 at most, within FP16, those below 2^-21
// of the row's largest are off by 2^-32 of it (the others by 2^-11 of themselves), and
// they are summed in binary32.
//
// What bounds it: a 256 x 128 tile is 2048 cycles of MMAs and takes about 4300, a half's
// chain of scores (1950 cycles from its last weights on, behind the other half's
// products) and of two times 64 keys' weights (1200 each).  A unit's start (queries, first
// keys) and end (output) add 10000 to 25000.  Eight requests of up to 1024 new tokens
// behind 1024 to 4096 keys, 32 query and 8 KV heads of 128: 215 us of 238 with the plan and the
// join, 566 TFLOP/s; a prefix of 32768 keys with 128 responses of 64 query heads: 120 us.
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

constexpr int kThreads = 640;
constexpr int kLoaders = 8;
// Registers a thread of each warpgroup after setmaxnreg: 2 x 128 x 112 + 2 x 128 x 96 +
// 128 x 64 = 640 x 96, what the block is launched with.
constexpr uint32_t kRegsRows = 112, kRegsLoad = 96, kRegsControl = 64;
static_assert(256 * kRegsRows + 256 * kRegsLoad + 128 * kRegsControl <= kThreads * 96, "registers");
constexpr int kStages = 2;
// Wait sites in the status word (after those of head.cu).
constexpr unsigned kSiteLoad = 24, kSiteQuery = 25, kSiteTile = 26, kSiteWeights = 27, kSiteScores = 28,
                   kSiteOutput = 29, kSiteDrain = 30, kSitePiece = 31;

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

// One stretch of a unit in a CTA's range, as warp 18 tells it the others.
struct Piece {
    int64_t token;     // the unit's first
    int s, r0, r1;     // segment; its requests
    int k0, k1, row;   // keys, table row
    int base;          // the first token's position, or -1
    int h;
    int kt0, n;        // first tile (or pair of tiles) and their number; n = 0: no more
    int ktiles;        // of the unit
    int rows;
    int pairs, both;   // A and B at alternate tiles; B takes part
    int first;         // of this CTA
};

// How often the stages were used before a piece; its tiles take them in turn from the
// first one on (where A and B have alternate tiles, each half has its own stage).  The
// same for all roles.
struct Ring {
    uint32_t used[kStages] = {0, 0};
    __device__ static int stage(int tile) { return tile & 1; }
    __device__ uint32_t use(int tile) const { return (tile & 1 ? used[1] : used[0]) + (tile >> 1); }
    __device__ void end(int tiles) { used[0] += (tiles + 1) >> 1, used[1] += tiles >> 1; }
};

__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}

// Place of 16-byte chunk c (8 FP16 channels) of row r in a [D / 64][128][128 bytes]
// operand with the 128-byte swizzle.
__device__ __forceinline__ uint32_t place(int r, int c) {
    return (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// The weights' reference at a maximum, and how far maxima may be before it is set again.
// Where a score's own rounding comes near a power of two (2^20 and above: 2^-4), neither
// has slack.
__device__ __forceinline__ float reference(float top) { return fabsf(top) < 0x1p20f ? top - 7.0f : top; }
__device__ __forceinline__ float limit(float ref) { return fabsf(ref) < 0x1p20f ? ref + 15.0f : ref; }

// max(a, b, c) in one instruction.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 32 bytes to a 32-byte boundary.
__device__ __forceinline__ void stg32(void *p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e,
                                      uint32_t f, uint32_t g, uint32_t h) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a), "r"(b),
                 "r"(c), "r"(d), "r"(e), "r"(f), "r"(g), "r"(h)
                 : "memory");
}

// Tensor core instructions under a predicate, for a warp whose lanes all run the loop
// around them: `lead` is 1 in the lane that issues them.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
__device__ __forceinline__ void mma_16bit_if(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
// A in TMEM: its rows are lanes, two 16-bit values a column.
__device__ __forceinline__ void mma_16bit_ta_if(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                                uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t lead, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(lead)
        : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attention_wide_kernel(const Args a, unsigned *status) {
    using C = Cfg<D>;
    extern __shared__ uint8_t dyn[];
    __shared__ uint64_t q_full, kv_full[kStages], kv_empty[kStages], s_full[2], p_full[2][2], pv_done[2],
        o_full[2], ml_full, drain_bar, piece_full[2], piece_empty[2];
    __shared__ Piece pieces[2];
    // of a stage's keys: those that are there; those with a NaN among their values (and
    // then not in the first), where some row does not see all keys
    __shared__ __align__(16) uint32_t sh_mask[kStages][4], sh_nan[kStages][4];
    __shared__ float sh_m[128], sh_l[128];
    // Whether the row sees a value that is NaN, by the piece's parity: B clears its flags for
    // the next piece while A may still have to read the last one's.
    __shared__ bool sh_bad[2][2][128];
    __shared__ uint32_t tmem_sh;
    __shared__ int abort_sh;
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
    const uint32_t smem = (smem_u32(dyn) + 1023u) & ~1023u;
    volatile int *abort = &abort_sh;

    if (tid == 0) {
        mbar_init(&q_full, 8);
        mbar_init(&ml_full, 4);
        mbar_init(&drain_bar, 2);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&kv_full[i], kLoaders / 2);
            mbar_init(&kv_empty[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i][0], 4);
            mbar_init(&p_full[i][1], 4);
            mbar_init(&o_full[i], 1);
            mbar_init(&pv_done[i], 1);
            mbar_init(&piece_full[i], 1);
            mbar_init(&piece_empty[i], 8 + kLoaders + 2);
        }
        abort_sh = 0;
        fence_mbar_init();
    }
    if (warp == 16) {
        tmem_alloc(&tmem_sh, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_sh;
    griddep_launch_dependents();
    griddep_wait();
    if (a.Ng == 0 && a.starts[kNarrowWorkers + blockIdx.x].empty > 0) clear_rows<D>(a, tid, kThreads);

    // A warp's wait for the n-th phase of a barrier (every lane asks: one lane's answer
    // passed on by a shuffle took a fifth longer), and its arrival, by one lane.
    auto wait = [&](uint64_t *bar, uint32_t n, unsigned site) -> bool {
        return __all_sync(~0u, mbar_wait(bar, n & 1u, abort, status, site));
    };
    auto arrive = [&](uint64_t *bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    const uint32_t q_s = smem;
    auto keys_at = [&](int st) -> uint32_t { return smem + 2 * C::kQBytes + st * C::kStageBytes; };
    auto values_at = [&](int st) -> uint32_t { return keys_at(st) + C::kKBytes; };
    uint32_t np = 0;  // pieces so far
    Ring ring;
    // The next piece (a warp's calls): waited for, and given back when done with.  It
    // stays in shared memory: registers are short.
    auto next = [&]() -> bool {
        return wait(&piece_full[np & 1], np >> 1, kSitePiece) && pieces[np & 1].n > 0;
    };
    auto done = [&]() {
        arrive(&piece_empty[np & 1]);
        ++np;
    };

    if (warp >= 16) {
        reg_dealloc<kRegsControl>();
        if (warp == 18) {
            // ------------------------------------------------------ the walk
            const Start &start = a.starts[kNarrowWorkers + blockIdx.x];
            int64_t left = start.left, from = start.from;  // tiles of the range; the next, in its segment
            int at = start.at, s = start.s;
            Segment g = start.g;
            const int *order = a.order + a.B + a.Ng;
            bool more = true, first = true;
            for (uint32_t i = 0; more; ++i) {
                Piece p;
                p.n = 0;
                if (left > 0) {
                    if (from < 0) {  // the next segment
                        s = order[++at];
                        g = a.segs[s];
                        from = 0;
                    }
                    const Wide w(a, g);
                    // the row tile that holds tile `from`
                    int64_t u = from;
                    int rt = 0;
                    if (g.base < 0) {
                        const int64_t each = (int64_t)w.ktiles(g, 0) * a.Hk;
                        rt = (int)(u / each);
                        u -= rt * each;
                    } else {
                        while (u >= (int64_t)w.ktiles(g, rt) * a.Hk) u -= (int64_t)w.ktiles(g, rt++) * a.Hk;
                    }
                    p.token = g.t0 + (int64_t)rt * w.tokens;
                    p.s = s;
                    p.r0 = g.r0, p.r1 = g.r1;
                    p.k0 = g.k0, p.k1 = g.k1, p.row = g.row;
                    p.base = g.base >= 0 ? g.base + rt * w.tokens : -1;
                    p.ktiles = w.ktiles(g, rt);
                    p.h = (int)((uint32_t)u / (uint32_t)p.ktiles);
                    p.kt0 = (int)((uint32_t)u - (uint32_t)p.h * p.ktiles);
                    p.n = (int)min((int64_t)(p.ktiles - p.kt0), left);
                    p.pairs = w.keys != kTile;
                    p.rows = min(w.tokens, g.ntok - rt * w.tokens) * a.G;
                    p.both = p.pairs || p.rows > 128;
                    if (lane == 0 && first && a.Ng == 0)
                        tell_split(a, true, blockIdx.x, g, from, p.kt0, p.ktiles, p.token, 0, p.h, p.rows);
                    p.first = first;
                    first = false;
                    left -= p.n;
                    from += p.n;
                    if (rt == w.rtiles - 1 && p.h == a.Hk - 1 && p.kt0 + p.n == p.ktiles) from = -1;
                }
                more = p.n > 0;
                if (!wait(&piece_empty[i & 1], (i >> 1) + 1, kSitePiece)) break;
                if (lane == 0) {
                    pieces[i & 1] = p;
                    mbar_arrive(&piece_full[i & 1]);
                }
                __syncwarp();
            }
        } else if (warp < 18) {
            // ---------------------------------------------------------- MMAs
            constexpr uint32_t kS = idesc_16bit(128, 128, false, false, false);
            constexpr uint32_t kO = idesc_16bit(128, D, false, false, true);
            // descriptors: their upper words are constant, the lower ones an address / 16
            constexpr uint64_t kKMajor = (uint64_t)1 << 16 | (uint64_t)64 << 32 | (uint64_t)1 << 46 |
                                         (uint64_t)kSwizzle128B << 61;  // offsets 16, 1024
            constexpr uint64_t kMnMajor = (uint64_t)1024 << 16 | (uint64_t)64 << 32 | (uint64_t)1 << 46 |
                                          (uint64_t)kSwizzle128B << 61;  // offsets 16384, 1024
            const int hf = warp - 16;
            const uint32_t s_t = tmem + hf * 128, o_t = tmem + 256 + hf * D;
            const uint32_t lead = elect_one();
            uint32_t nt = 0;  // the half's tiles so far
            bool ok = true;
            while (ok && wait(&piece_full[np & 1], np >> 1, kSitePiece)) {
                const Piece &p = pieces[np & 1];
                const bool pairs = __shfl_sync(~0u, p.pairs, 0), both = __shfl_sync(~0u, p.both, 0);
                const int all = __shfl_sync(~0u, p.n, 0), n = hf == 0 || both ? all : 0, each = pairs ? 2 : 1;
                if (all == 0) break;
                const bool alone = pairs || !both;  // nobody else reads this half's tiles
                if (!wait(&q_full, np, kSiteQuery)) break;
                done();
                const uint64_t qa = kKMajor + ((q_s + (pairs ? 0 : hf) * C::kQBytes) >> 4);
                auto scores = [&](int i) -> bool {
                    const int tile = i * each + (pairs ? hf : 0), st = Ring::stage(tile);
                    if (!wait(&kv_full[st], ring.use(tile), kSiteTile)) return false;
                    tc_fence_after();
                    const uint64_t kb = kKMajor + (keys_at(st) >> 4);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t o = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
                        mma_16bit_if(lead, s_t, qa + o, kb + o, kS, ks > 0);
                    }
                    commit_if(lead, &s_full[hf]);
                    return true;
                };
                if (n > 0) ok = scores(0);
                for (int i = 0; ok && i < n; ++i, ++nt) {
                    const int st = Ring::stage(i * each + (pairs ? hf : 0));
                    const uint64_t vb = kMnMajor + (values_at(st) >> 4);
                    // values, 64 keys at a time, the later ones first
#pragma unroll
                    for (int b = 1; b >= 0; --b) {
                        ok = ok && wait(&p_full[hf][b], nt, kSiteWeights);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_16bit_ta_if(lead, o_t, s_t + 64 + b * 32 + ks * 8, vb + (b * 8192 + ks * 2048) / 16, kO,
                                            i > 0 || b == 0 || ks > 0);
                        if (b == 1) commit_if(lead, &pv_done[hf]);
                    }
                    if (!ok) break;
                    commit_if(lead, &kv_empty[st]);
                    if (alone) commit_if(lead, &kv_empty[st]);
                    if (i + 1 == n) commit_if(lead, &o_full[hf]);
                    else ok = scores(i + 1);
                }
                ring.end(all * each);
            }
            commit_if(lead, &drain_bar);
            __syncwarp();
            mbar_wait(&drain_bar, 0, nullptr, status, kSiteDrain);
        }
    } else if (warp >= 8) {
        // ------------------------------------------------------------- codes
        reg_dealloc<kRegsLoad>();
        constexpr int CH = D / 16;          // 16-byte chunks of a key's codes
        constexpr int RW = 32 / CH;         // rows a warp reads at once
        constexpr int KW = 2 * kTile / kLoaders;  // rows of a warp
        constexpr int NI = KW / RW;
        const int w = warp & 3, set = (warp - 8) >> 2;  // the two sets have a stage each
        bool ok = true;
        while (ok && next()) {
            const Piece &p = pieces[np & 1];
            const bool pairs = p.pairs;
            const int64_t key0 = (int64_t)p.k0 + (int64_t)p.kt0 * (pairs ? 2 : 1) * kTile + KW * w + lane;
            const int k1 = p.k1, tiles = p.n * (pairs ? 2 : 1);
            const int64_t head = (int64_t)p.h * D;
            const int32_t *tab = a.table + (int64_t)p.row * a.width;
            // the block of key KW w + lane of tile i (the table's entry, or -1) and the
            // key's place in it
            struct Entry {
                int id;
                uint32_t at;
            };
            auto entry_of = [&](int i) -> Entry {
                const int64_t key = key0 + (int64_t)i * kTile;
                Entry e = {-1, 0u};
                if (i < tiles && key < k1) {
                    e.id = tab[block_of(a, (uint32_t)key, e.at)];
                }
                return e;
            };
            auto slot_of = [&](Entry e) -> int {
                const int64_t slot = (int64_t)e.id * a.bs + e.at;
                return e.id >= 0 && slot < a.S ? (int)slot : -1;
            };
            // the first key from which on a tile may begin that not all rows see whole
            const int whole = (int)max(p.base - (key0 - lane - KW * w) - (kTile - 2), (int64_t)-1);
            uint4 kr[NI] = {}, vr[NI] = {};
            const int c = lane % CH, rq = lane / CH;
            // (a missing key reads slot 0: its score is left out, its value zeroed)
            auto load = [&](int slot) {
                if (a.S == 0) return;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int sl = __shfl_sync(~0u, slot, RW * i + rq);
                    const int64_t from = (int64_t)max(sl, 0) * a.Hk * D + head + c * 16;
                    kr[i] = __ldg(reinterpret_cast<const uint4 *>(a.kc + from));
                    vr[i] = __ldg(reinterpret_cast<const uint4 *>(a.vc + from));
                }
            };
            auto store = [&](uint32_t dst, const uint4 (&v)[NI]) {
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int r = KW * w + RW * i + rq;
                    // chunks 2 c and 2 c + 1; the lanes of the upper half of a row (and of odd
                    // rows where a row has four chunks) write the odd one first, so that
                    // eight lanes touch every bank once
                    const bool swap = D == 128 ? c >= 4 : (rq & 1);
                    const uint32_t f = swap ? v[i].z : v[i].x, g = swap ? v[i].w : v[i].y,
                                   y = swap ? v[i].x : v[i].z, z = swap ? v[i].y : v[i].w;
                    sts16(dst + place(r, 2 * c + swap), codes_f16(f), codes_f16_hi(f), codes_f16(g),
                          codes_f16_hi(g));
                    sts16(dst + place(r, 2 * c + !swap), codes_f16(y), codes_f16_hi(y), codes_f16(z),
                          codes_f16_hi(z));
                }
            };
            // Loads come back in order: the entry of a tile is asked for before the
            // codes of the tile before it, and used behind them.
            Entry nxt = entry_of(set + 2);
            int cur = slot_of(entry_of(set));
            if (set < tiles) load(cur);
            for (int i = set; i < tiles; i += 2) {
                const int st = set;
                // A NaN among the values of a key that some row does not see (weight 0) would
                // reach that row: taken out below, and given to the rows that see the key.
                bool some = false;
                if (i * kTile >= whole) {
#pragma unroll
                    for (int j = 0; j < NI; ++j) some = some || nan_bits(vr[j]) != 0;
                }
                if (!wait(&kv_empty[st], ring.use(i) + 1, kSiteLoad)) {
                    ok = false;
                    break;
                }
                const uint32_t mask = __ballot_sync(~0u, cur >= 0);
                if (lane == 0) sh_mask[st][w] = mask, sh_nan[st][w] = 0u;
                __syncwarp();
                if (mask != ~0u) {
#pragma unroll
                    for (int j = 0; j < NI; ++j)
                        if (!((mask >> (RW * j + rq)) & 1u)) vr[j] = make_uint4(0, 0, 0, 0);
                }
                store(keys_at(st), kr);
                if (some) {
#pragma unroll
                    for (int j = 0; j < NI; ++j) {
                        if (nan_bits(vr[j]) == 0) continue;
                        atomicOr(&sh_nan[st][w], 1u << (RW * j + rq));
                        atomicAnd(&sh_mask[st][w], ~(1u << (RW * j + rq)));
                        vr[j] = make_uint4(0, 0, 0, 0);
                    }
                }
                store(values_at(st), vr);
                fence_proxy_async();
                arrive(&kv_full[st]);
                cur = slot_of(nxt);
                nxt = entry_of(i + 4);
                if (i + 2 < tiles) load(cur);
            }
            ring.end(tiles);
            done();
        }
    } else {
        // ----------------------------------------------- weights and outputs
        reg_alloc<kRegsRows>();
        const int hf = warp >> 2, r = tid & 127;  // half, its row = TMEM lane
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_t = lanes + hf * 128, o_t = lanes + 256 + hf * D;
        const bool wide_out = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0 && a.ldo % 16 == 0;
        uint32_t nt = 0, no[2] = {0, 0}, nml = 0;  // the half's tiles, outputs, merges so far
        bool ok = true;
        while (ok && next()) {
            const Piece &p = pieces[np & 1];
            const bool pairs = p.pairs, active = hf == 0 || p.both;
            const int n = active ? p.n : 0;
            const int lr = r + (pairs ? 0 : 128 * hf);
            const bool row_ok = lr < p.rows, idle = !__any_sync(~0u, row_ok);
            // token and query head of the row
            auto place_of = [&](int64_t &t, int &hq) {
                const uint32_t row = row_ok ? lr : 0, tok = row / (uint32_t)a.G;
                t = p.token + tok;
                hq = p.h * a.G + (int)(row - tok * a.G);
            };
            // the query
            float f, ref = -INFINITY, l = 0.0f;  // factor of the scores; the weights' reference
                                                 // (an exponent of two) and sum
            int pos = 0x7FFFFFFF;                // a row past the unit's last hides no key
            {
                int64_t t;
                int hq;
                place_of(t, hq);
                const uint4 *src = reinterpret_cast<const uint4 *>(a.q + t * a.ldq + (int64_t)hq * D);
                // (half a row at a time: registers are short)
                constexpr int NH = 8, NQ = D / 8 / NH;
                uint4 v[NH];
                auto read = [&](int part) {
#pragma unroll
                    for (int i = 0; i < NH; ++i) v[i] = row_ok ? src[part * NH + i] : make_uint4(0, 0, 0, 0);
                };
                float top = 0.0f;
#pragma unroll 1
                for (int part = NQ - 1; part >= 0; --part) {
                    read(part);
#pragma unroll
                    for (int i = 0; i < NH; ++i) {
                        const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            top = max3(top, fabsf(__uint_as_float(u[k] << 16)),
                                       fabsf(__uint_as_float(u[k] & 0xFFFF0000u)));
                    }
                }
                if (row_ok) {
                    Segment g;
                    g.t0 = p.token, g.r0 = p.r0, g.r1 = p.r1, g.base = p.base;
                    pos = position(a, g, p.s, t);
                }
                float up = row_power(top);
                f = a.scale * a.ks[p.h] * kLog2e * inverse_power(up);
                if (f < 0.0f) f = -f, up = -up;  // maxima are of the raw scores
                f = fmaxf(f, 0x1p-126f);
                if (!pairs || hf == 0) {
                    const uint32_t dst = q_s + hf * C::kQBytes;
#pragma unroll 1
                    for (int part = 0; part < NQ; ++part) {
                        if (part > 0) read(part);
#pragma unroll
                        for (int i = 0; i < NH; ++i) {
                            const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                w[k] = pack_f16(__uint_as_float(u[k] << 16) * up,
                                                __uint_as_float(u[k] & 0xFFFF0000u) * up);
                            sts16(dst + place(r, part * NH + i), w[0], w[1], w[2], w[3]);
                        }
                    }
                    fence_proxy_async();
                }
            }
            sh_bad[np & 1][hf][r] = false;
            tc_fence_before();  // the last piece's reads of TMEM
            arrive(&q_full);
            const int each = pairs ? 2 : 1;
            const int64_t key0 = (int64_t)p.k0 + (int64_t)p.kt0 * each * kTile;
            if (!active && !wait(&q_full, no[0], kSiteQuery)) break;  // its next arrival is the next piece's
            for (int i = 0; i < n; ++i, ++nt) {
                const int tile = i * each + (pairs ? hf : 0), st = Ring::stage(tile);
                if (!wait(&s_full[hf], nt, kSiteScores) || !wait(&kv_full[st], ring.use(tile), kSiteScores)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (idle) {  // no row of the warp's is the unit's: nobody reads its weights' products
                    arrive(&p_full[hf][1]);
                    arrive(&p_full[hf][0]);
                    continue;
                }
                // the keys that the row sees, where some are hidden
                const int64_t left = pos - (key0 + (int64_t)tile * kTile);
                const uint4 there = *reinterpret_cast<const uint4 *>(&sh_mask[st][0]);
                const bool hidden = __any_sync(~0u, left < kTile - 1 || (there.x & there.y & there.z & there.w) != ~0u);
                // the scores of keys 64 h .. 64 h + 63, -inf for those the row does not see
                // (rolled loops below: more code than the instruction cache holds beside the
                // other warps' slows every role)
                uint32_t v0[32], v1[32];
                auto read = [&](int h) {
                    __syncwarp();
                    tmem_ld32(s_t + 64 * h, v0);
                    tmem_ld32(s_t + 64 * h + 32, v1);
                    tmem_wait32(v0);
                    tmem_wait32(v1);
                    if (hidden) {
                        const uint32_t nan[2] = {sh_nan[st][2 * h], sh_nan[st][2 * h + 1]};
                        uint32_t see[2] = {(h ? there.z : there.x) | nan[0], (h ? there.w : there.y) | nan[1]};
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int64_t l = left - 64 * h - 32 * c;
                            if (l < 31) see[c] &= l < 0 ? 0u : (2u << (int)l) - 1u;
                        }
                        if ((see[0] & nan[0]) | (see[1] & nan[1])) sh_bad[np & 1][hf][r] = true;
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            if (!((see[0] >> k) & 1u)) v0[k] = __float_as_uint(-INFINITY);
                            if (!((see[1] >> k) & 1u)) v1[k] = __float_as_uint(-INFINITY);
                        }
                    }
                };
                const float2 f2 = make_float2(f, f);
                // 64 keys at a time, the later ones first: their maximum, the reference raised
                // where it has grown too far, their weights (hidden keys' scores are -inf) to
                // 32 columns over the upper half of the scores
#pragma unroll
                for (int h = 1; h >= 0; --h) {
                    read(h);
                    float top = -INFINITY, top1 = -INFINITY;
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        top = max3(top, __uint_as_float(v0[k]), __uint_as_float(v0[k + 1]));
                        top1 = max3(top1, __uint_as_float(v1[k]), __uint_as_float(v1[k + 1]));
                    }
                    top = fmaxf(top, top1) * f;
                    const bool start = i == 0 && h == 1, grown = !start && top > limit(ref);
                    if (start) ref = reference(top);
                    if (__any_sync(~0u, grown)) {
                        // the output so far: the products of the last tile were issued before these
                        // scores, whose arrival was waited for; those of this tile's later keys
                        if (h == 0 && !wait(&pv_done[hf], nt, kSiteOutput)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const float now = grown ? reference(top) : ref, c = grown ? ex2(ref - now) : 1.0f;
                        ref = now;
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
                    const float nm = ref == -INFINITY ? 0.0f : -ref;
                    const float2 nm2 = make_float2(nm, nm);
                    float2 s0 = make_float2(0.0f, 0.0f), s1 = s0;
                    auto weigh = [&](const uint32_t (&v)[32], int col) {
                        uint32_t w[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float2 x = __ffma2_rn(
                                make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), f2, nm2);
                            const float2 e = make_float2(ex2(x.x), ex2(x.y));
                            if (k & 1) s1 = __fadd2_rn(s1, e); else s0 = __fadd2_rn(s0, e);
                            w[k] = pack_f16(e.x, e.y);
                        }
                        __syncwarp();
                        tmem_st16(s_t + 64 + col, w);
                    };
                    weigh(v0, 32 * h);
                    weigh(v1, 32 * h + 16);
                    l += (s0.x + s0.y) + (s1.x + s1.y);
                    tmem_st_wait();
                    tc_fence_before();
                    arrive(&p_full[hf][h]);
                }
                if (!ok) break;
            }
            ring.end(p.n * each);
            if (!ok) break;
            // the output
            if (active) {
                if (!wait(&o_full[hf], no[hf], kSiteOutput)) break;
                if (pairs && hf == 1) {
                    sh_m[r] = ref;
                    sh_l[r] = l;
                    arrive(&ml_full);
                } else {
                    float ca = 1.0f, cb = 0.0f;
                    if (pairs) {
                        if (!wait(&o_full[1], no[1], kSiteOutput) ||
                            !wait(&ml_full, nml, kSiteOutput))
                            break;
                        const float mb = sh_m[r], both = fmaxf(ref, mb), use = both == -INFINITY ? 0.0f : both;
                        ca = ex2(ref - use);
                        cb = ex2(mb - use);
                        l = l * ca + sh_l[r] * cb;
                        ref = both;
                    }
                    __syncwarp();
                    tc_fence_after();
                    int64_t t;
                    int hq;
                    place_of(t, hq);
                    const bool full = p.n == p.ktiles, direct = full && a.Ng == 0;
                    const int64_t slot = full ? ((p.s < a.B ? a.T : 0) + t) * a.Hq + hq
                                              : (int64_t)(2 * blockIdx.x + (p.first ? 0 : 1)) * kWideRows + lr;
                    float *po = (full ? a.whole : a.wpart) + slot * D;
                    const bool bad = sh_bad[np & 1][hf][r] || (pairs && sh_bad[np & 1][1][r]);
                    const float inv = bad ? __uint_as_float(0x7FFFFFFFu) : row_factor(a.vs[p.h], l, a.ks[p.h]);
                    uint16_t *out = a.out + t * a.ldo + (int64_t)hq * D;
#pragma unroll 1
                    for (int ch = 0; ch < D / 32; ++ch) {
                        uint32_t v[32];
                        __syncwarp();
                        tmem_ld32(o_t + ch * 32, v);
                        tmem_wait32(v);
                        if (pairs) {
                            uint32_t w[32];
                            tmem_ld32(o_t + D + ch * 32, w);
                            tmem_wait32(w);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                v[k] = __float_as_uint(ca * __uint_as_float(v[k]) + cb * __uint_as_float(w[k]));
                        }
                        if (!row_ok) continue;
                        if (direct) {
                            uint32_t w[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const __nv_bfloat162 b = __floats2bfloat162_rn(
                                    __uint_as_float(v[2 * k]) * inv, __uint_as_float(v[2 * k + 1]) * inv);
                                w[k] = *reinterpret_cast<const uint32_t *>(&b);
                            }
                            uint16_t *to = out + ch * 32;
#pragma unroll
                            for (int k = 0; k < 16; k += 8) {
                                if (wide_out) {
                                    stg32(to + 2 * k, w[k], w[k + 1], w[k + 2], w[k + 3], w[k + 4], w[k + 5],
                                          w[k + 6], w[k + 7]);
                                } else {
                                    *reinterpret_cast<uint4 *>(to + 2 * k) =
                                        make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
                                    *reinterpret_cast<uint4 *>(to + 2 * k + 8) =
                                        make_uint4(w[k + 4], w[k + 5], w[k + 6], w[k + 7]);
                                }
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < 32; k += 8)
                                stg32(po + ch * 32 + k, v[k], v[k + 1], v[k + 2], v[k + 3], v[k + 4], v[k + 5],
                                      v[k + 6], v[k + 7]);
                        }
                    }
                    if (row_ok) {
                        if (!direct) {
                            float *ml = (full ? a.whole_ml : a.wpart_ml) + slot * 2;
                            ml[0] = ref;
                            ml[1] = bad ? -l : l;
                        } else if (a.lse) {
                            a.lse[t * a.Hq + hq] = row_lse(ref, l, a.ks[p.h]);
                        }
                    }
                }
            }
            ++no[0];
            if (p.both) ++no[1];
            if (pairs) ++nml;
            done();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
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
    return launch_pdl(attention_wide_kernel<D>, dim3((unsigned)a.ctas), dim3(kThreads), Cfg<D>::kSmem,
                      stream, a, dev.status_word);
}

}  // namespace

namespace jet {
jet_status launch_attention_wide(const DeviceInfo &dev, const attn::Args &a, int D, cudaStream_t stream) {
    return D == 64 ? launch<64>(dev, a, stream) : launch<128>(dev, a, stream);
}
}  // namespace jet
