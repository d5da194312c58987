// Strided views of caller tensors: host-side checks (alignment, overlap) and vector access, shared by
// the operators around the attention.
#pragma once

#include <string.h>

#include "common.cuh"

namespace ssa {

// ---- host --------------------------------------------------------------------------------------

inline int64_t extent_of(const ssa_heads_t& v, int64_t N, int32_t D) {
    return (N - 1) * v.token_stride + (int64_t)(v.heads - 1) * v.head_stride + D;
}

inline bool check_view(const ssa_heads_t* v, int64_t N, int32_t D, size_t es, bool written) {
    if (!v || !v->data || v->heads < 1 || v->heads > 65535) return false;
    if (v->token_stride < 0 || v->head_stride < 0) return false;
    // the last element's offset stays inside 62 bits, products included
    const int64_t most = (int64_t)1 << 35;
    if ((N > 1 && v->token_stride > most) || (v->heads > 1 && v->head_stride > most)) return false;
    if ((uintptr_t)v->data % es) return false;
    if (written) {
        const int64_t ts = N > 1 ? v->token_stride : INT64_MAX, hs = v->heads > 1 ? v->head_stride : INT64_MAX;
        const bool heads_inside = hs >= D && (N == 1 || v->heads == 1 ? ts >= D : ts >= (v->heads - 1) * hs + D);
        const bool tokens_inside = ts >= D && (N == 1 || v->heads == 1 ? hs >= D : hs >= (N - 1) * ts + D);
        if (!heads_inside && !tokens_inside) return false;
    }
    return true;
}

inline bool same_view(const ssa_heads_t& a, const ssa_heads_t& b, int64_t N) {
    return a.data == b.data && a.heads == b.heads && (N == 1 || a.token_stride == b.token_stride) &&
           (a.heads == 1 || a.head_stride == b.head_stride);
}

// Whether two views share no element, as far as this can tell: their ranges do not meet, or they are
// parts of one row of equal token stride, or of equal head stride.
inline bool disjoint(const ssa_heads_t& a, const ssa_heads_t& b, int64_t N, int32_t D, size_t es) {
    const uintptr_t pa = (uintptr_t)a.data, pb = (uintptr_t)b.data;
    if (pa + (uintptr_t)extent_of(a, N, D) * es <= pb || pb + (uintptr_t)extent_of(b, N, D) * es <= pa) return true;
    const int64_t d = ((int64_t)pb - (int64_t)pa) / (int64_t)es;
    auto apart = [d](int64_t period, int64_t ea, int64_t eb) {
        const int64_t o = ((d % period) + period) % period;
        return o >= ea && o + eb <= period;
    };
    if (N > 1 && a.token_stride == b.token_stride && a.token_stride > 0 &&
        apart(a.token_stride, (int64_t)(a.heads - 1) * a.head_stride + D, (int64_t)(b.heads - 1) * b.head_stride + D))
        return true;
    const int64_t s = a.head_stride;
    return s > 0 && b.head_stride == s && (N == 1 || (a.token_stride % s == 0 && b.token_stride % s == 0)) &&
           apart(s, D, D);
}

// Largest vector (elements) at which every row of a view starts aligned.
inline int view_vector(const ssa_heads_t& v, int64_t N, size_t es, int most) {
    while (most > 1 && ((uintptr_t)v.data % (most * es) || (N > 1 && v.token_stride % most) ||
                        (v.heads > 1 && v.head_stride % most)))
        most >>= 1;
    return most;
}

// fp32 arrays of a call start at a multiple of their size (null passes).
template <typename... P>
inline bool aligned4(P... p) {
    return (((uintptr_t)p | ...) & 3) == 0;
}

// Whether fp32 arrays share no memory (null: no array).
struct Span {
    const float* p;
    int64_t n;
};
inline bool apart(const Span& a, const Span& b) {
    const uintptr_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
    return !a.p || !b.p || pa + 4 * (uintptr_t)a.n <= pb || pb + 4 * (uintptr_t)b.n <= pa;
}

// Makes the plan's device current for the scope.
struct DeviceScope {
    int before = 0;
    bool ok = true, moved = false;
    explicit DeviceScope(int device) {
        if (cudaGetDevice(&before) != cudaSuccess) before = device;
        if (before != device) {
            moved = true;
            ok = cudaSetDevice(device) == cudaSuccess;
        }
    }
    ~DeviceScope() {
        if (moved) cudaSetDevice(before);
    }
};

// Multiprocessors of a device, asked once per device.
inline int sm_count(int device) {
    static std::atomic<int> known[64];
    if (device >= 0 && device < 64) {
        const int n = known[device].load(std::memory_order_relaxed);
        if (n) return n;
    }
    int n = 148;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) n = 148;
    if (device >= 0 && device < 64) known[device].store(n, std::memory_order_relaxed);
    return n;
}

// Lets a kernel take any dynamic shared memory that an SM has beside 8 KB of its own; asked for once per kernel and device.
template <auto KERNEL>
bool allow_smem(int device) {
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = device >= 0 && device < 64 ? (uint64_t)1 << device : 0;
    if (bit && (done.load(std::memory_order_relaxed) & bit)) return true;
    if (cudaFuncSetAttribute((const void*)KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (227 - 8) * 1024) != cudaSuccess)
        return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// ---- device ------------------------------------------------------------------------------------

template <int BYTES> struct Chunk;
template <> struct Chunk<16> { using type = uint4; };
template <> struct Chunk<8> { using type = uint2; };
template <> struct Chunk<4> { using type = uint32_t; };
template <> struct Chunk<2> { using type = uint16_t; };

// One chunk from global to this thread's place in shared memory, without waiting (2 bytes, which the
// asynchronous copy does not take: through a register). `cp_wait<N>`: all but the last N groups have landed.
template <int BYTES>
__device__ __forceinline__ void cp_async(void* smem, const void* global) {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(smem);
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(global) : "memory");
    else if constexpr (BYTES >= 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(global), "n"(BYTES) : "memory");
    else
        *(uint16_t*)smem = *(const uint16_t*)global;
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Two fp32 operations in one instruction (each rounded as its scalar form): elements (i, i + 1) of arrays.
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmul.rn.f32x2 d, a, b;\nmov.b64 {%0, %1}, d;\n}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nadd.rn.f32x2 d, a, b;\nmov.b64 {%0, %1}, d;\n}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0, float c1) {
    asm("{\n.reg .b64 a, b, c, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%6, %7};\n"
        "fma.rn.f32x2 d, a, b, c;\nmov.b64 {%0, %1}, d;\n}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}

// V elements of T as one load, and as floats.
template <typename T, int V>
struct Vec {
    using C = typename Chunk<V * (int)sizeof(T)>::type;
    static __device__ __forceinline__ void unpack(const C& raw, float (&e)[V]) {
        T v[V];
        memcpy(v, &raw, sizeof(v));
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] = Elem<T>::to_f(v[j]);
    }
    static __device__ __forceinline__ C pack(const float (&e)[V]) {
        T v[V];
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = Elem<T>::from_f(e[j]);
        C raw;
        memcpy(&raw, v, sizeof(v));
        return raw;
    }
};

}  // namespace ssa
