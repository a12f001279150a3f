// Stands in for the library's mla_device.cuh when a kernel's source is compiled for the CPU: the same names, as far as the
// kernels tested here use them. A CTA's threads are contexts of one thread, switched where they wait for each other: a warp
// runs until all its lanes are at a barrier of the CTA, in an order of warps that the caller chooses, so that what a
// kernel leaves to chance between two barriers comes out at its worst. Shared variables are static: each starts with what
// the CTA before left.
#pragma once

#include <ucontext.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <functional>
#include <vector>

#include "mlasparse.h"

#define __global__ static
#define __device__
#define __host__
#define __forceinline__ inline
#define __launch_bounds__(...)
#define __shared__ static
#define __align__(n) __attribute__((aligned(n)))

struct int2 { int x, y; };
struct float2 { float x, y; };
struct float4 { float x, y, z, w; };
struct uint4 { uint32_t x, y, z, w; };
struct dim3 { unsigned x = 1, y = 1, z = 1; dim3() = default; explicit dim3(unsigned n) : x(n) {} };
inline int2 make_int2(int x, int y) { return {x, y}; }
inline float2 make_float2(float x, float y) { return {x, y}; }
inline float4 make_float4(float x, float y, float z, float w) { return {x, y, z, w}; }
inline uint4 make_uint4(uint32_t x, uint32_t y, uint32_t z, uint32_t w) { return {x, y, z, w}; }
using std::max;
using std::min;

// ---- the CTA ----

namespace simt {

constexpr size_t kStack = 96 << 10;

struct Lane { ucontext_t context; std::vector<char> stack; bool done; int line; };    // line: of the barrier it waits at, or 0
struct Warp { uint32_t value[2][32]; int here; unsigned phase; int kind; };

inline std::vector<Lane> lanes;
inline std::vector<Warp> warps;
inline ucontext_t scheduler;
inline int current, threads, at_barrier, barrier_line;
inline unsigned barriers;
inline bool failed;                    // lanes of a warp or warps of a CTA that wait for different things
inline int order;                      // of the warps: 0 ascending, 1 descending, 2 + k: warp k last
inline std::function<void()> body;

inline void pause() { swapcontext(&lanes[current].context, &scheduler); }

// All lanes of the warp bring a value; returns them.
inline const uint32_t* exchange(int kind, uint32_t v) {
    Warp& w = warps[current / 32];
    const unsigned phase = w.phase;
    uint32_t* const values = w.value[phase & 1];
    if (w.here == 0) w.kind = kind;
    failed = failed || w.kind != kind;
    values[current % 32] = v;
    if (++w.here == 32) {
        w.here = 0;
        ++w.phase;
    }
    while (w.phase == phase && !failed) pause();
    return values;
}

inline void barrier(int line) {
    const unsigned now = barriers;
    if (at_barrier == 0) barrier_line = line;
    failed = failed || barrier_line != line;
    if (++at_barrier == threads) {
        at_barrier = 0;
        ++barriers;
    }
    lanes[current].line = line;
    while (barriers == now && !failed) pause();
    lanes[current].line = 0;
}

inline void entry() {
    body();
    lanes[current].done = true;
    pause();
}

// One CTA; false where its threads would wait for ever.
inline bool run(int n) {
    threads = n;
    lanes.resize(n);
    warps.assign(n / 32, Warp{});
    at_barrier = 0;
    for (int i = 0; i < n; ++i) {
        Lane& l = lanes[i];
        l.stack.resize(kStack);
        l.done = false;
        l.line = 0;
        getcontext(&l.context);
        l.context.uc_stack.ss_sp = l.stack.data();
        l.context.uc_stack.ss_size = kStack;
        l.context.uc_link = &scheduler;
        makecontext(&l.context, entry, 0);
    }
    std::vector<int> turn(n / 32);
    for (int w = 0; w < n / 32; ++w) turn[w] = order == 1 ? n / 32 - 1 - w : w;
    if (order >= 2 && order - 2 < n / 32) {
        turn.erase(turn.begin() + (order - 2));
        turn.push_back(order - 2);
    }
    for (;;) {
        bool all_done = true, moved = false;
        for (int w : turn) {
            // until each lane is done or at a barrier that the CTA has not passed
            for (bool again = true; again && !failed;) {
                again = false;
                for (int i = 32 * w; i < 32 * w + 32; ++i) {
                    if (lanes[i].done) continue;
                    const unsigned phase = warps[w].phase, passed = barriers;
                    const int line = lanes[i].line, here = warps[w].here, waiting = at_barrier;
                    current = i;
                    swapcontext(&scheduler, &lanes[i].context);
                    again = again || lanes[i].done || phase != warps[w].phase || passed != barriers || line != lanes[i].line ||
                            here != warps[w].here || waiting != at_barrier;
                }
                moved = moved || again;
            }
            for (int i = 32 * w; i < 32 * w + 32; ++i) all_done = all_done && lanes[i].done;
        }
        if (failed) return false;
        if (all_done) return at_barrier == 0;
        if (!moved) return false;
    }
}

struct Index {
    struct X { operator unsigned() const { return current; } } x;
};

}  // namespace simt

inline const simt::Index threadIdx;
inline dim3 blockIdx, blockDim, gridDim;
#define __syncthreads() simt::barrier(__LINE__)

// ---- a warp's ----

inline uint32_t __ballot_sync(unsigned, bool p) {
    const uint32_t* v = simt::exchange(1, p);
    uint32_t r = 0;
    for (int i = 0; i < 32; ++i) r |= v[i] << i;
    return r;
}
inline uint32_t __reduce_or_sync(unsigned, uint32_t x) {
    const uint32_t* v = simt::exchange(2, x);
    uint32_t r = 0;
    for (int i = 0; i < 32; ++i) r |= v[i];
    return r;
}
template <typename T>
inline T __reduce_add_sync(unsigned, T x) {
    const uint32_t* v = simt::exchange(3, static_cast<uint32_t>(x));
    uint32_t r = 0;
    for (int i = 0; i < 32; ++i) r += v[i];
    return static_cast<T>(r);
}
inline int __shfl_up_sync(unsigned, int x, int d) {
    const int lane = simt::current % 32;
    return static_cast<int>(simt::exchange(4, static_cast<uint32_t>(x))[lane >= d ? lane - d : lane]);
}
inline void __syncwarp() { simt::exchange(5, 0); }

// ---- a thread's ----

template <typename T> inline T __ldg(const T* p) { return *p; }
inline int __popc(uint32_t x) { return __builtin_popcount(x); }
inline int __clz(uint32_t x) { return x == 0 ? 32 : __builtin_clz(x); }
inline uint32_t __float_as_uint(float x) { uint32_t u; std::memcpy(&u, &x, 4); return u; }
template <typename T> inline T atomicOr(T* p, T v) { const T old = *p; *p |= v; return old; }
template <typename T> inline T atomicMin(T* p, T v) { const T old = *p; *p = std::min(old, v); return old; }

struct __nv_bfloat16 { uint16_t x; };
struct __half2 { uint16_t x, y; };
// (values of the cache are not what is tested: they read as 0)
inline float2 __half22float2(__half2) { return {0.0f, 0.0f}; }

namespace mla {
constexpr int kLatent = MLA_LATENT_DIM, kScaleOff = MLA_SCALE_OFFSET, kTailOff = MLA_TAIL_OFFSET, kRope = MLA_ROPE_DIM;
inline void pdl_wait() {}
inline void pdl_launch_dependents() {}
inline uint4 ld_nc_v4(const void* p) { uint4 v; std::memcpy(&v, p, 16); return v; }
inline void e4m3x4_to_f16x2x2(uint32_t, uint32_t& lo, uint32_t& hi) { lo = hi = 0; }
inline uint32_t pack_bf16x2(float, float) { return 0; }
inline float bf16lo(uint32_t) { return 0.0f; }
inline float bf16hi(uint32_t) { return 0.0f; }
}  // namespace mla

namespace mla_host {
inline int error_word;
inline int* device_error_word() { return &error_word; }
}  // namespace mla_host

// ---- launches ----

enum cudaError_t { cudaSuccess, cudaErrorLaunchFailure };
enum { cudaLaunchAttributeProgrammaticStreamSerialization };
using cudaStream_t = void*;
struct cudaLaunchAttribute { int id; struct { int programmaticStreamSerializationAllowed; } val; };
struct cudaLaunchConfig_t {
    dim3 gridDim, blockDim;
    size_t dynamicSmemBytes;
    cudaStream_t stream;
    cudaLaunchAttribute* attrs;
    int numAttrs;
};
inline cudaError_t cudaGetLastError() { return cudaSuccess; }

template <typename K, typename... A>
cudaError_t cudaLaunchKernelEx(const cudaLaunchConfig_t* cfg, K kernel, A... args) {
    gridDim = cfg->gridDim;
    blockDim = cfg->blockDim;
    simt::failed = false;
    simt::body = [&]() { kernel(args...); };
    for (unsigned b = 0; b < cfg->gridDim.x; ++b) {
        blockIdx.x = b;
        if (!simt::run(static_cast<int>(cfg->blockDim.x))) return cudaErrorLaunchFailure;
    }
    return cudaSuccess;
}
