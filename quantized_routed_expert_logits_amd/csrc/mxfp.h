// Device helpers of microscaled 4-bit floating point (E2M1 values, one power
// of two per 32) and of rows in fp32, fp16 or bf16.
#pragma once

#include "block.h"

namespace strata_moe {

typedef float v2f __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef _Float16 v4h __attribute__((ext_vector_type(4)));
typedef __bf16 v4b __attribute__((ext_vector_type(4)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(_Float16 v) { return (float)v; }
__device__ __forceinline__ float widen(__bf16 v) { return (float)v; }

__device__ __forceinline__ void load4_vec(const float* p, float* v) {
    const float4 f = *(const float4*)p;
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
}
__device__ __forceinline__ void load4_vec(const _Float16* p, float* v) {
    const v4h f = *(const v4h*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)f[i];
}
__device__ __forceinline__ void load4_vec(const __bf16* p, float* v) {
    const uint2 f = *(const uint2*)p;
    v[0] = __uint_as_float(f.x << 16), v[1] = __uint_as_float(f.x & 0xffff0000u);
    v[2] = __uint_as_float(f.y << 16), v[3] = __uint_as_float(f.y & 0xffff0000u);
}

// 16 bytes at an element's address: the memory takes wide accesses at any of them.
typedef v4f v4f_any __attribute__((aligned(4)));
typedef v8h v8h_any __attribute__((aligned(2)));
typedef v8b v8b_any __attribute__((aligned(2)));
typedef uint32_t v4u_any __attribute__((ext_vector_type(4), aligned(2)));

// 8 neighbouring values.
__device__ __forceinline__ void load8(const float* p, float* v) {
    const v4f a = *(const v4f_any*)p, b = *(const v4f_any*)(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
}
__device__ __forceinline__ void load8(const _Float16* p, float* v) {
    const v8h f = *(const v8h_any*)p;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)f[i];
}
__device__ __forceinline__ void load8(const __bf16* p, float* v) {
    const v4u_any u = *(const v4u_any*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

// v (4 values that are exact in type T) to columns j..j+3 of a row of H.
template <typename T, typename V>
__device__ __forceinline__ void store4(T* row, int j, int H, bool vec, const float* v) {
    if (vec && j + 4 <= H) {
        V o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = (T)v[i];
        *(V*)(row + j) = o;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (j + i < H) row[j + i] = (T)v[i];
}
// v (8 values) to columns j..j+7 of a row of H, 16 bytes a store.
template <typename T, typename V>
__device__ __forceinline__ void store8(T* row, int j, int H, const float* v) {
    constexpr int n = 16 / (int)sizeof(T);
    if (j + 8 <= H) {
#pragma unroll
        for (int k = 0; k < 8; k += n) {
            V o;
#pragma unroll
            for (int i = 0; i < n; ++i) o[i] = (T)v[k + i];
            *(V*)(row + j + k) = o;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (j + i < H) row[j + i] = (T)v[i];
}

__device__ __forceinline__ void store4_any(void* base, int dtype, int64_t at, int j, int H, bool vec, const float* v) {
    if (dtype == kF32) store4<float, v4f>((float*)base + at, j, H, vec, v);
    else if (dtype == kF16) store4<_Float16, v4h>((_Float16*)base + at, j, H, vec, v);
    else store4<__bf16, v4b>((__bf16*)base + at, j, H, vec, v);
}

// v rounded to fp32 and from there to the type, as a 16-bit tensor is made of a
// 64-bit one; *o: the value as fp32.
__device__ __forceinline__ double round_to(double v, int dtype, float* o) {
    const float f = (float)v;
    *o = dtype == kF32 ? f : dtype == kF16 ? (float)(_Float16)f : (float)(__bf16)f;
    return *o;
}

// ---- 4-bit blocks
// The scale byte of a block whose largest magnitude has these fp32 bits:
// 2^(byte - 127) = 2^(floor(log2 top) - 2), not below 2^-127; 255 (NaN) for an
// infinite or NaN value.  A zero block has byte 0.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
    const uint32_t e = top >> 23;
    return e == 255 ? 255u : e < 2 ? 0u : e - 2;
}
__device__ __forceinline__ float mx_scale(uint32_t byte) {
    return __uint_as_float(byte == 255 ? 0x7fc00000u : byte ? byte << 23 : 0x00400000u);
}
// The codes of a and b (nearest, ties to even, magnitudes above 6 to 6) into
// byte B of q, a in the low half.
template <int B>
__device__ __forceinline__ uint32_t mx_code_pair(uint32_t q, float a, float b, uint32_t byte) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, a, b, mx_scale(byte), B);
}

}  // namespace strata_moe
