// Vectors of consecutive elements widened to float32: VEC = 4 or 8 bf16 or 4 float32
// at addresses that are multiples of the vector, or 1 element.
#pragma once

#include "common.cuh"

namespace gdn {

template <typename T, int VEC> struct Raw;  // what one load brings
template <> struct Raw<float, 4> { float4 r; };
template <> struct Raw<__nv_bfloat16, 8> { uint4 r; };
template <> struct Raw<__nv_bfloat16, 4> { uint2 r; };
template <> struct Raw<float, 1> { float r; };
template <> struct Raw<__nv_bfloat16, 1> { __nv_bfloat16 r; };

template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T *p) {
    return *reinterpret_cast<const Raw<T, VEC> *>(p);
}

__device__ __forceinline__ void widen(const Raw<float, 4> &v, float (&x)[4]) {
    x[0] = v.r.x; x[1] = v.r.y; x[2] = v.r.z; x[3] = v.r.w;
}
__device__ __forceinline__ void widen(const Raw<__nv_bfloat16, 8> &v, float (&x)[8]) {
    const uint32_t w[4] = {v.r.x, v.r.y, v.r.z, v.r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // bf16 is the upper half of a float32
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void widen(const Raw<__nv_bfloat16, 4> &v, float (&x)[4]) {
    x[0] = __uint_as_float(v.r.x << 16);
    x[1] = __uint_as_float(v.r.x & 0xffff0000u);
    x[2] = __uint_as_float(v.r.y << 16);
    x[3] = __uint_as_float(v.r.y & 0xffff0000u);
}
__device__ __forceinline__ void widen(const Raw<float, 1> &v, float (&x)[1]) { x[0] = v.r; }
__device__ __forceinline__ void widen(const Raw<__nv_bfloat16, 1> &v, float (&x)[1]) {
    x[0] = __bfloat162float(v.r);
}

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T *p, float (&x)[VEC]) {
    widen(load_raw<T, VEC>(p), x);
}

__device__ __forceinline__ void store_vec(float *p, const float (&x)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store_vec(__nv_bfloat16 *p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_vec(__nv_bfloat16 *p, const float (&x)[4]) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                                               *reinterpret_cast<const uint32_t *>(&hi));
}
template <typename T>
__device__ __forceinline__ void store_vec(T *p, const float (&x)[1]) { *p = from_f32<T>(x[0]); }

// A parameter (weight, bias) held in float32 or in T.
template <typename T, int VEC>
__device__ __forceinline__ void load_param(const void *p, long long at, bool f32, float (&x)[VEC]) {
    if (f32) {
        constexpr int V = VEC % 4 ? 1 : 4;  // `at` is a multiple of VEC
#pragma unroll
        for (int i = 0; i < VEC; i += V) {
            float v[V];
            load_vec<float, V>(static_cast<const float *>(p) + at + i, v);
#pragma unroll
            for (int e = 0; e < V; ++e) x[i + e] = v[e];
        }
    } else {
        load_vec<T, VEC>(static_cast<const T *>(p) + at, x);
    }
}

// acc += x y, two elements per instruction.
template <int VEC>
__device__ __forceinline__ void fma_vec(const float (&x)[VEC], const float (&y)[VEC],
                                        float (&acc)[VEC]) {
    if constexpr (VEC % 2 == 0) {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
            const float2 z = __ffma2_rn(make_float2(x[e], x[e + 1]), make_float2(y[e], y[e + 1]),
                                        make_float2(acc[e], acc[e + 1]));
            acc[e] = z.x;
            acc[e + 1] = z.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = fmaf(x[e], y[e], acc[e]);
    }
}

// x *= y
template <int VEC>
__device__ __forceinline__ void mul_vec(float (&x)[VEC], const float (&y)[VEC]) {
    if constexpr (VEC % 2 == 0) {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
            const float2 z = __fmul2_rn(make_float2(x[e], x[e + 1]), make_float2(y[e], y[e + 1]));
            x[e] = z.x;
            x[e + 1] = z.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] *= y[e];
    }
}
// x += y
template <int VEC>
__device__ __forceinline__ void add_vec(float (&x)[VEC], const float (&y)[VEC]) {
    if constexpr (VEC % 2 == 0) {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
            const float2 z = __fadd2_rn(make_float2(x[e], x[e + 1]), make_float2(y[e], y[e + 1]));
            x[e] = z.x;
            x[e + 1] = z.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] += y[e];
    }
}

// x packed to T, as one load would have brought it.
__device__ __forceinline__ Raw<float, 4> pack(const float (&x)[4], Raw<float, 4>) {
    return Raw<float, 4>{make_float4(x[0], x[1], x[2], x[3])};
}
__device__ __forceinline__ Raw<__nv_bfloat16, 8> pack(const float (&x)[8], Raw<__nv_bfloat16, 8>) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return Raw<__nv_bfloat16, 8>{make_uint4(w[0], w[1], w[2], w[3])};
}

// Copies one vector to shared memory without passing registers; the copying thread
// may read it after copy_wait, which leaves its latest `pending` committed groups
// under way.  (Vectors under 4 bytes are loaded and stored.)
template <typename T, int VEC>
__device__ __forceinline__ void copy_async(Raw<T, VEC> *to, const T *from) {
    constexpr int bytes = sizeof(Raw<T, VEC>);
    if constexpr (bytes >= 4) {
        const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(bytes)
                     : "memory");
    } else {
        *to = load_raw<T, VEC>(from);
    }
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// 1 / (1 + e^-x) by the approximate power of two and reciprocal: off by at most a few
// float32 roundings (1e-6 relative for |x| up to 10); 0 where e^-x overflows.
__device__ __forceinline__ float fast_sigmoid(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
// The same of VEC elements, two per instruction where the unit allows.
template <int VEC>
__device__ __forceinline__ void fast_sigmoid(const float (&x)[VEC], float (&s)[VEC]) {
    if constexpr (VEC % 2 == 0) {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            const float2 m = __fmul2_rn(make_float2(x[i], x[i + 1]),
                                        make_float2(-1.4426950408889634f, -1.4426950408889634f));
            float2 e;
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(m.x));
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(m.y));
            e = __fadd2_rn(e, make_float2(1.f, 1.f));
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s[i]) : "f"(e.x));
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s[i + 1]) : "f"(e.y));
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[i] = fast_sigmoid(x[i]);
    }
}

// slots[i .. i + 3], i a multiple of 4, from an array 16 bytes aligned; -1 from n on.
__device__ __forceinline__ void load_slots(const int *slots, int i, int n, int (&s)[4]) {
    if (i + 4 <= n) {
        const int4 v = *reinterpret_cast<const int4 *>(slots + i);
        s[0] = v.x; s[1] = v.y; s[2] = v.z; s[3] = v.w;
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] = i + k < n ? slots[i + k] : -1;
}
// Whether sequence i has tokens: offsets that are none leave it out, and the slot that it
// names to the others.
__device__ __forceinline__ bool has_tokens(const int *cu, int total, int i) {
    return !cu || (cu[i] >= 0 && cu[i] < cu[i + 1] && cu[i + 1] <= total);
}
// Whether one of the sequences before n that have tokens names `slot` (>= 0); each caller
// looks at its share.
__device__ __forceinline__ int slot_taken(const int *slots, const int *cu, int total, int n, int slot,
                                          int from, int step) {
    int taken = 0;
#pragma unroll 2
    for (int i = 4 * from; i < n; i += 4 * step) {
        int s[4];
        load_slots(slots, i, n, s);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (s[k] == slot) taken |= has_tokens(cu, total, i + k);
    }
    return taken;
}

}  // namespace gdn
