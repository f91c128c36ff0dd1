// hip_runtime.h -- what the scan kernels use of HIP, on the CPU (test infrastructure).
//
// A workgroup is one thread of the host, its lanes are fibers that change over at every
// cross-lane operation and barrier; shared memory is local to that thread.  Workgroups of a
// launch run side by side, so atomics are real ones.  Range-checked buffer accesses do what the
// hardware does with them; every other access goes to memory as it is, where guard pages lie
// around each tensor.
#pragma once

#include <math.h>
#include <sched.h>
#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#define __global__
#define __device__
#define __host__
#define __forceinline__ inline
#define __launch_bounds__(...)
#define __shared__ static thread_local

using std::max;
using std::min;

struct uint3 {
    unsigned x, y, z;
};
struct dim3 {
    unsigned x, y, z;
    dim3(unsigned x = 1, unsigned y = 1, unsigned z = 1) : x(x), y(y), z(z) {}
};
typedef int hipError_t;
typedef void *hipStream_t;
enum { hipSuccess = 0, hipErrorInvalidValue = 1 };
hipError_t hipLaunchKernel(const void *fn, dim3 grid, dim3 block, void **args, size_t lds, hipStream_t s);

extern thread_local uint3 threadIdx, blockIdx;
extern thread_local dim3 blockDim, gridDim;

// cross-lane operations of a whole wave (scan_host.cpp)
void host_barrier();
uint32_t host_exchange(uint32_t value, int from);  // the value of lane `from` of the wave
bool host_all(bool p);

inline void __syncthreads() { host_barrier(); }
inline int __all(int p) { return host_all(p != 0); }

inline float __uint_as_float(uint32_t u) {
    float f;
    memcpy(&f, &u, 4);
    return f;
}
inline uint32_t __float_as_uint(float f) {
    uint32_t u;
    memcpy(&u, &f, 4);
    return u;
}
inline int host_lane() { return threadIdx.x & 63; }
inline int __shfl_up(int v, int d) { return (int)host_exchange((uint32_t)v, host_lane() >= d ? host_lane() - d : host_lane()); }
inline int __shfl_down(int v, int d) { return (int)host_exchange((uint32_t)v, host_lane() + d < 64 ? host_lane() + d : host_lane()); }
inline float __shfl_up(float v, int d) { return __uint_as_float((uint32_t)__shfl_up((int)__float_as_uint(v), d)); }
inline float __shfl_down(float v, int d) { return __uint_as_float((uint32_t)__shfl_down((int)__float_as_uint(v), d)); }

inline uint32_t atomicAdd(uint32_t *p, uint32_t v) { return __atomic_fetch_add(p, v, __ATOMIC_RELAXED); }
#define __HIP_MEMORY_SCOPE_AGENT 0
#define __hip_atomic_load(p, order, scope) __atomic_load_n(p, order)
#define __hip_atomic_store(p, v, order, scope) __atomic_store_n(p, v, order)

#define __builtin_amdgcn_sched_barrier(x)
#define __builtin_amdgcn_s_sleep(x) sched_yield()
#define __builtin_amdgcn_readfirstlane(x) ((int)host_exchange((uint32_t)(x), 0))
inline float host_med3(float a, float b, float c) { return a != a ? b : max(b, min(a, c)); }
#define __builtin_amdgcn_fmed3f(a, b, c) host_med3(a, b, c)
// gdr_mfma.hpp declares these; no kernel here calls them
#define __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, x, y, z) (c)
#define __builtin_amdgcn_global_load_lds(src, dst, size, offset, aux) (void)0

// range-checked buffers: words past the end read 0 and are not stored
struct HostBuffer {
    char *base;
    uint32_t bytes;
};
#define __amdgpu_buffer_rsrc_t HostBuffer
typedef unsigned int host_u2 __attribute__((ext_vector_type(2)));
typedef unsigned int host_u4 __attribute__((ext_vector_type(4)));

template <class E, int N, class R> inline R host_load(HostBuffer r, uint32_t at) {
    E e[N];
    for (int i = 0; i < N; ++i) {
        e[i] = 0;
        const uint64_t o = (uint64_t)at + i * sizeof(E);
        if (o + sizeof(E) <= r.bytes) memcpy(&e[i], r.base + o, sizeof(E));
    }
    R out;
    memcpy(&out, e, sizeof(e));
    return out;
}
template <class E, int N, class R> inline void host_store(R v, HostBuffer r, uint32_t at) {
    E e[N];
    memcpy(e, &v, sizeof(e));
    for (int i = 0; i < N; ++i) {
        const uint64_t o = (uint64_t)at + i * sizeof(E);
        if (o + sizeof(E) <= r.bytes) memcpy(r.base + o, &e[i], sizeof(E));
    }
}
#define __builtin_amdgcn_make_buffer_rsrc(p, stride, n, flags) (HostBuffer{(char *)(p), (uint32_t)(n)})
#define __builtin_amdgcn_raw_buffer_load_b16(r, at, s, aux) host_load<uint16_t, 1, uint16_t>(r, at)
#define __builtin_amdgcn_raw_buffer_load_b32(r, at, s, aux) host_load<uint32_t, 1, uint32_t>(r, at)
#define __builtin_amdgcn_raw_buffer_load_b64(r, at, s, aux) host_load<uint32_t, 2, host_u2>(r, at)
#define __builtin_amdgcn_raw_buffer_load_b128(r, at, s, aux) host_load<uint32_t, 4, host_u4>(r, at)
#define __builtin_amdgcn_raw_buffer_store_b16(v, r, at, s, aux) host_store<uint16_t, 1, uint16_t>(v, r, at)
#define __builtin_amdgcn_raw_buffer_store_b32(v, r, at, s, aux) host_store<uint32_t, 1, uint32_t>(v, r, at)
#define __builtin_amdgcn_raw_buffer_store_b64(v, ...) host_store64(v, __VA_ARGS__)
#define __builtin_amdgcn_raw_buffer_store_b128(v, ...) host_store128(v, __VA_ARGS__)
inline void host_store64(host_u2 v, HostBuffer r, uint32_t at, int, int) { host_store<uint32_t, 2, host_u2>(v, r, at); }
inline void host_store128(host_u4 v, HostBuffer r, uint32_t at, int, int) { host_store<uint32_t, 4, host_u4>(v, r, at); }
