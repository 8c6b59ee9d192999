// Block tables and slot maps of a paged KV cache, built on the GPU from the
// requests' lengths (jet_kv_slot_map): the slots jet_kv_cache_write takes and
// the positions jet_rope takes, without a host round trip.
//
// Request b holds cached[b] tokens and adds added[b]; with bs the block size
//   old_b = ceil(cached/bs),  need_b = max(0, min(ceil((cached+added)/bs), width) - old_b),
// and its new blocks come from the free list in request order, at
// free_next + sum_{b' < b} need_b'.  Token t of the batch belongs to the
// request whose offset range holds it and sits at
//   pos = cached_b + t - offset_b,  slot = table[b][pos / bs] bs + pos % bs.
//
// All integers, and latency-bound at serving sizes: every CTA scans the
// requests itself (two prefix sums in one pass, at most 8192 requests, kept in
// shared memory), so one launch suffices and no CTA waits for another; a fresh
// block's id is computed from the scan, never read back from the table.  256
// requests of one token take 3.2 us, 65536 tokens 4.4, half of it the launch.
#include "jet_common.cuh"

namespace {

constexpr int kSmThreads = 512;
constexpr int64_t kSmMaxRequests = 8192;

__global__ void __launch_bounds__(kSmThreads)
kv_slot_map_kernel(const int *__restrict__ cached, const int *__restrict__ added, int B, int bs,
                   int *table, int64_t width, const int *__restrict__ free_blocks, int64_t n_free,
                   const int64_t *__restrict__ free_next, int64_t N, int64_t *__restrict__ offsets,
                   int64_t *__restrict__ positions, int64_t *__restrict__ slots,
                   int *__restrict__ rows, int64_t *__restrict__ counts) {
    extern __shared__ int64_t off[];  // [B + 1] token offsets, [B] first new block, [B] cached
    __shared__ int64_t warp_tok[kSmThreads / 32], warp_blk[kSmThreads / 32];
    int64_t *blk = off + B + 1;
    int *len = reinterpret_cast<int *>(blk + B);
    jet::griddep_launch_dependents();
    jet::griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t next = *free_next;
    next = next < 0 ? 0 : next > n_free ? n_free : next;
    int64_t base_tok = 0, base_blk = 0;
    for (int b0 = 0; b0 < B; b0 += kSmThreads) {
        const int b = b0 + threadIdx.x;
        const int64_t c = b < B ? max(cached[b], 0) : 0, n = b < B ? max(added[b], 0) : 0;
        const int64_t old = (c + bs - 1) / bs;
        int64_t need = min((c + n + bs - 1) / bs, width) - old;
        need = need > 0 ? need : 0;
        int64_t ti = n, bi = need;  // inclusive sums over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t a = __shfl_up_sync(0xffffffffu, ti, o), d = __shfl_up_sync(0xffffffffu, bi, o);
            if (lane >= o) {
                ti += a;
                bi += d;
            }
        }
        if (lane == 31) {
            warp_tok[warp] = ti;
            warp_blk[warp] = bi;
        }
        __syncthreads();
        int64_t pt = 0, pb = 0, tt = 0, tb = 0;
#pragma unroll
        for (int w = 0; w < kSmThreads / 32; ++w) {
            if (w == warp) {
                pt = tt;
                pb = tb;
            }
            tt += warp_tok[w];
            tb += warp_blk[w];
        }
        if (b < B) {
            off[b] = base_tok + pt + ti - n;
            blk[b] = base_blk + pb + bi - need;
            len[b] = (int)c;
        }
        base_tok += tt;
        base_blk += tb;
        __syncthreads();
    }
    if (threadIdx.x == 0) off[B] = base_tok;
    __syncthreads();
    if (blockIdx.x == 0) {
        for (int b = threadIdx.x; b <= B; b += kSmThreads) offsets[b] = off[b];
        if (threadIdx.x == 0) {
            const int64_t end = next + base_blk < n_free ? next + base_blk : n_free;
            counts[0] = end;
            counts[1] = next + base_blk - end;
        }
    }
    const int64_t last = base_tok > N ? base_tok : N;
    for (int64_t t = blockIdx.x * (int64_t)kSmThreads + threadIdx.x; t < last;
         t += (int64_t)gridDim.x * kSmThreads) {
        if (t >= base_tok) {  // padding of the outputs
            positions[t] = 0;
            slots[t] = -1;
            rows[t] = -1;
            continue;
        }
        int lo = 0, hi = B - 1;  // the first request whose range ends after t
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (off[mid + 1] > t) hi = mid;
            else lo = mid + 1;
        }
        const uint32_t c = (uint32_t)len[lo];
        const uint32_t pos = c + (uint32_t)(t - off[lo]);  // below 2^32: two int32 lengths
        const uint32_t j = pos / (uint32_t)bs, in_block = pos - j * (uint32_t)bs;
        const uint32_t old = c / (uint32_t)bs + (c % (uint32_t)bs != 0);
        int id = -1;
        if ((int64_t)j < width) {
            int *entry = table + lo * width + j;
            if (j < old) {
                id = *entry;
            } else {
                const int64_t at = next + blk[lo] + (j - old);
                if (at < n_free) id = free_blocks[at];
                if (in_block == 0) *entry = id;  // a new block's first token is a new token
            }
        }
        if (t < N) {
            positions[t] = pos;
            slots[t] = id < 0 ? -1 : (int64_t)id * bs + in_block;
            rows[t] = lo;
        }
    }
}

template <int kBytes>
bool aligned_to(const void *p) { return (reinterpret_cast<uintptr_t>(p) & (kBytes - 1)) == 0; }

}  // namespace

jet_status jet_kv_slot_map(const int32_t *cached, const int32_t *added, int64_t B,
                           int64_t block_size, int32_t *table, int64_t width,
                           const int32_t *free_blocks, int64_t n_free, const int64_t *free_next,
                           int64_t N, int64_t *offsets, int64_t *positions, int64_t *slots,
                           int32_t *rows, int64_t *counts, jet_stream_t stream) {
    JET_REQUIRE(B >= 0 && width >= 0 && n_free >= 0 && N >= 0, JET_ERR_SHAPE);
    JET_REQUIRE(free_next && offsets && counts && (B == 0 || (cached && added)), JET_ERR_NULL);
    JET_REQUIRE((B == 0 || width == 0 || table) && (n_free == 0 || free_blocks), JET_ERR_NULL);
    JET_REQUIRE(N == 0 || (positions && slots && rows), JET_ERR_NULL);
    JET_REQUIRE(B <= kSmMaxRequests && block_size >= 1 && block_size < ((int64_t)1 << 30) &&
                    width < ((int64_t)1 << 31) && N < ((int64_t)1 << 40) &&
                    n_free < ((int64_t)1 << 31) && free_next != counts && free_next != counts + 1,
                JET_ERR_SHAPE);
    // element-wise accesses: a free list may start inside an allocation
    JET_REQUIRE(aligned_to<4>(cached) && aligned_to<4>(added) && aligned_to<4>(table) &&
                    aligned_to<4>(free_blocks) && aligned_to<8>(free_next) &&
                    aligned_to<8>(offsets) && aligned_to<8>(positions) && aligned_to<8>(slots) &&
                    aligned_to<4>(rows) && aligned_to<8>(counts),
                JET_ERR_ALIGN);
    jet::DeviceInfo dev;
    jet_status st = jet::current_device(&dev);
    if (st != JET_OK) return st;
    constexpr size_t kMaxSmem = (kSmMaxRequests + 1) * 8 + kSmMaxRequests * 12;
    const size_t smem = (size_t)(B + 1) * 8 + (size_t)B * 12;
    if (smem > 40 * 1024 &&
        cudaFuncSetAttribute(kv_slot_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)kMaxSmem) != cudaSuccess) {
        cudaGetLastError();
        return JET_ERR_CUDA;
    }
    const int64_t want = (N + kSmThreads - 1) / kSmThreads;
    const int64_t g = want < 1 ? 1 : want < dev.num_sms ? want : dev.num_sms;
    return jet::launch_pdl(kv_slot_map_kernel, dim3((unsigned)g), dim3(kSmThreads), smem,
                           jet::as_stream(stream), cached, added, (int)B, (int)block_size, table,
                           width, free_blocks, n_free, free_next, N, offsets, positions, slots,
                           rows, counts);
}
