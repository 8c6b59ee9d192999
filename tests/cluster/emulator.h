// Runs a cluster kernel's source on the CPU: every CUDA thread is a fiber, and
// the schedule is chosen by the test, so that an order of execution that a GPU
// allows but seldom takes can be forced.  Holds what csrc/sample.cu uses, no more.
#pragma once
#include <setjmp.h>
#include <stdint.h>
#include <string.h>
#include <sys/mman.h>
#include <ucontext.h>

#include <algorithm>
#include <cmath>
#include <vector>

struct uint4 { unsigned x, y, z, w; };
struct float2 { float x, y; };
struct ulonglong2 { unsigned long long x, y; };
struct Dim { unsigned x, y = 1, z = 1; };

namespace emu {

constexpr size_t kStack = 128 << 10;

struct Fiber {
    jmp_buf at;
    ucontext_t first;
    bool begun = false, done = false;
    const unsigned *wait = nullptr;  // runs once *wait differs from value
    unsigned value = 0;
    unsigned arrived = 0;  // the cluster barrier's generation at this thread's arrival
    Dim tid, bid;
    unsigned cta, warp;
};

// A barrier of n threads; its generation changes when the last one arrives.
struct Barrier {
    unsigned n = 0, arrived = 0, gen = 0;
};

struct Warp {
    Barrier bar;
    uint64_t v[2][32];
};

struct Cta {
    Barrier bar;
    bool begun = false;
    unsigned live = 0;
    std::vector<unsigned char> smem;
};

struct Cluster {
    std::vector<Fiber> fibers;
    std::vector<Warp> warps;
    std::vector<Cta> ctas;
    Barrier bar;
    unsigned threads = 0, syncs = 0;
    int early = 0;  // accesses to a CTA that has not begun or has ended
    void (*kernel)(const void *) = nullptr;
    const void *args = nullptr;
};

static Cluster cluster;
static Fiber *cur;
static jmp_buf scheduler;

__attribute__((noinline)) static void yield() {
    asm volatile("" ::: "memory");
    if (!_setjmp(cur->at)) _longjmp(scheduler, 1);
    asm volatile("" ::: "memory");
}

static unsigned arrive(Barrier &b) {
    const unsigned gen = b.gen;
    if (++b.arrived == b.n) {
        b.arrived = 0;
        ++b.gen;
    }
    return gen;
}

static void await(const Barrier &b, unsigned gen) {
    cur->wait = &b.gen;
    cur->value = gen;
    yield();
}

// What every lane of the warp holds.
static const uint64_t *exchange(uint64_t v) {
    Warp &w = cluster.warps[cur->warp];
    uint64_t *to = w.v[w.bar.gen & 1];
    to[cur->tid.x & 31] = v;
    await(w.bar, arrive(w.bar));
    return to;
}

static Cta &cta() { return cluster.ctas[cur->cta]; }
static unsigned char *smem() { return cta().smem.data(); }

static void cluster_arrive() {
    cur->arrived = arrive(cluster.bar);
    if (cur->arrived != cluster.bar.gen) ++cluster.syncs;
}
static void cluster_wait() { await(cluster.bar, cur->arrived); }

static void enter() {
    Cta &c = cta();
    if (!c.begun) {
        c.begun = true;
        std::fill(c.smem.begin(), c.smem.end(), (unsigned char)0xA5);  // what a CTA before left
    }
    cluster.kernel(cluster.args);
    --cta().live;
    cur->done = true;
    _longjmp(scheduler, 1);
}

static void run(Fiber &f) {
    cur = &f;
    f.wait = nullptr;
    if (_setjmp(scheduler)) return;
    if (f.begun) _longjmp(f.at, 1);
    f.begun = true;
    setcontext(&f.first);
}

// Who falls behind: nobody, a CTA, all CTAs but one, or a warp of the cluster.
enum Lag { kNobody, kCta, kOthers, kWarp };

// One launch of a cluster of C CTAs.  From the cluster barrier number `from` on
// (0: from the start), those who fall behind run only while no other thread can.
// 0, or 1 when threads wait for one another for ever.
static int launch(void (*kernel)(const void *), const void *args, unsigned C, unsigned threads,
                  size_t smem_bytes, Lag lag, unsigned who, unsigned from) {
    Cluster &k = cluster;
    k = Cluster();
    k.kernel = kernel;
    k.args = args;
    k.threads = threads;
    k.fibers.resize(C * threads);
    k.warps.resize(C * threads / 32);
    k.ctas.resize(C);
    k.bar.n = C * threads;
    for (Warp &w : k.warps) w.bar.n = 32;
    for (Cta &c : k.ctas) {
        c.bar.n = c.live = threads;
        c.smem.resize(smem_bytes);
    }
    const size_t all = kStack * k.fibers.size();
    char *stacks = (char *)mmap(nullptr, all, PROT_READ | PROT_WRITE,
                                MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0);
    if (stacks == MAP_FAILED) return 2;
    for (unsigned i = 0; i < k.fibers.size(); ++i) {
        Fiber &f = k.fibers[i];
        f.tid.x = i % threads;
        f.bid.x = f.cta = i / threads;
        f.warp = i / 32;
        getcontext(&f.first);
        f.first.uc_stack.ss_sp = stacks + kStack * i;
        f.first.uc_stack.ss_size = kStack;
        f.first.uc_link = nullptr;
        makecontext(&f.first, enter, 0);
    }
    int status = 0;
    for (size_t left = k.fibers.size(); left;) {
        bool ran = false;
        for (int lagging = 0; lagging < 2 && !ran; ++lagging)
            for (Fiber &f : k.fibers) {
                const bool late = k.syncs >= from && (lag == kCta      ? f.cta == who
                                                      : lag == kOthers ? f.cta != who
                                                                       : lag == kWarp && f.warp == who);
                if (f.done || late != (bool)lagging || (f.wait && *f.wait == f.value)) continue;
                run(f);
                ran = true;
                left -= f.done;
            }
        if (!ran) {
            status = 1;
            break;
        }
    }
    munmap(stacks, all);
    return status;
}

}  // namespace emu

#define __device__
#define __global__
#define __forceinline__ inline
#define __noinline__ __attribute__((noinline))
#define __launch_bounds__(...)
#define threadIdx (emu::cur->tid)
#define blockIdx (emu::cur->bid)
#define blockDim (Dim{emu::cluster.threads})

using std::max;
using std::min;

inline void __cluster_barrier_arrive_relaxed() { emu::cluster_arrive(); }

namespace cooperative_groups {
struct cluster_group {
    void barrier_arrive() const { emu::cluster_arrive(); }
    void barrier_wait() const { emu::cluster_wait(); }
    void sync() const {
        barrier_arrive();
        barrier_wait();
    }
    unsigned num_blocks() const { return (unsigned)emu::cluster.ctas.size(); }
    unsigned block_rank() const { return emu::cur->cta; }
    template <typename T>
    T *map_shared_rank(T *p, unsigned rank) const {
        emu::Cta &c = emu::cluster.ctas[rank];
        if (!c.begun || !c.live) ++emu::cluster.early;
        return reinterpret_cast<T *>(c.smem.data() + (reinterpret_cast<unsigned char *>(p) - emu::smem()));
    }
};
inline cluster_group this_cluster() { return {}; }
}  // namespace cooperative_groups

namespace jet {
inline void griddep_launch_dependents() {}
inline void griddep_wait() {}
}  // namespace jet

inline void __syncthreads() { emu::await(emu::cta().bar, emu::arrive(emu::cta().bar)); }

template <typename A, typename B>
inline B bits_as(A a) {
    static_assert(sizeof(A) == sizeof(B), "same size");
    B b;
    memcpy(&b, &a, sizeof(b));
    return b;
}
inline unsigned __float_as_uint(float f) { return bits_as<float, unsigned>(f); }
inline float __uint_as_float(unsigned u) { return bits_as<unsigned, float>(u); }
inline float __int_as_float(int i) { return bits_as<int, float>(i); }
inline uint4 make_uint4(unsigned x, unsigned y, unsigned z, unsigned w) { return {x, y, z, w}; }
inline float2 make_float2(float x, float y) { return {x, y}; }
inline ulonglong2 make_ulonglong2(unsigned long long x, unsigned long long y) { return {x, y}; }
inline float __fadd_rn(float a, float b) { return a + b; }
inline float __fmul_rn(float a, float b) { return a * b; }
inline float __fdiv_rn(float a, float b) { return a / b; }
inline float2 __fadd2_rn(float2 a, float2 b) { return {a.x + b.x, a.y + b.y}; }
inline float2 __fmul2_rn(float2 a, float2 b) { return {a.x * b.x, a.y * b.y}; }
inline float2 __ffma2_rn(float2 a, float2 b, float2 c) { return {fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)}; }
inline unsigned long long __float2ull_rn(float f) { return (unsigned long long)nearbyintf(f); }
inline float __ull2float_rn(unsigned long long u) { return (float)u; }
inline unsigned long long __umul64hi(unsigned long long a, unsigned long long b) {
    return (unsigned long long)(((unsigned __int128)a * b) >> 64);
}
inline int __popc(unsigned v) { return __builtin_popcount(v); }
inline int __popcll(unsigned long long v) { return __builtin_popcountll(v); }
inline int __ffsll(long long v) { return __builtin_ffsll(v); }
inline int __clz(int v) { return v ? __builtin_clz((unsigned)v) : 32; }
inline int __clzll(long long v) { return v ? __builtin_clzll((unsigned long long)v) : 64; }

template <typename T>
inline T from_lane(T v, int lane) {
    uint64_t b = 0;
    memcpy(&b, &v, sizeof(v));
    b = emu::exchange(b)[lane & 31];
    memcpy(&v, &b, sizeof(v));
    return v;
}
template <typename T>
inline T __shfl_sync(unsigned, T v, int lane) { return from_lane(v, lane); }
template <typename T>
inline T __shfl_xor_sync(unsigned, T v, int mask) { return from_lane(v, (int)(emu::cur->tid.x & 31) ^ mask); }
template <typename T>
inline T __shfl_up_sync(unsigned, T v, int by) {
    const int lane = emu::cur->tid.x & 31;
    return from_lane(v, lane < by ? lane : lane - by);
}
template <typename F>
inline unsigned over_lanes(unsigned v, F f) {
    const uint64_t *all = emu::exchange(v);
    unsigned r = (unsigned)all[0];
    for (int i = 1; i < 32; ++i) r = f(r, (unsigned)all[i]);
    return r;
}
inline unsigned __reduce_add_sync(unsigned, unsigned v) {
    return over_lanes(v, [](unsigned a, unsigned b) { return a + b; });
}
inline unsigned __reduce_min_sync(unsigned, unsigned v) {
    return over_lanes(v, [](unsigned a, unsigned b) { return a < b ? a : b; });
}
inline int __reduce_min_sync(unsigned, int v) {
    return (int)(__reduce_min_sync(0, (unsigned)v ^ 0x80000000u) ^ 0x80000000u);
}
inline unsigned __reduce_max_sync(unsigned, unsigned v) {
    return over_lanes(v, [](unsigned a, unsigned b) { return a > b ? a : b; });
}
inline unsigned __ballot_sync(unsigned, bool p) {
    const uint64_t *all = emu::exchange(p);
    unsigned r = 0;
    for (int i = 0; i < 32; ++i) r |= (unsigned)all[i] << i;
    return r;
}
inline unsigned atomicAdd(unsigned *p, unsigned v) {
    const unsigned old = *p;
    *p += v;
    return old;
}
inline unsigned atomicMin(unsigned *p, unsigned v) {
    const unsigned old = *p;
    *p = std::min(old, v);
    return old;
}
inline unsigned atomicMax(unsigned *p, unsigned v) {
    const unsigned old = *p;
    *p = std::max(old, v);
    return old;
}
