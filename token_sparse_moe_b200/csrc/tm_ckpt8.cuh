// tm_ckpt8.cuh -- 8-bit activation checkpoints: the format's device code, shared by the pack and
// unpack kernels and by the kernels that write or read a checkpoint in passing.
//
// A row is cut into blocks of 32 values (the last one may be shorter).  With m the largest finite
// magnitude of a block, its scale is 2^e, e the smallest integer with m <= 127 * 2^e, at least -126
// (so that 2^e and 2^-e are normal fp32 numbers) and at most 121 (so that 127 * 2^e is finite); a
// value's code is the nearest integer to x * 2^-e, ties to even, held to +-127 (which only binds above
// 127 * 2^121).  Scaling by a power of two is exact, so the codes depend on x alone: two correct
// implementations give the same ones.  Code -128 stands for a value that is not finite and reads
// back as NaN: an overflow in the forward pass is not hidden from the backward pass.  A code times
// 2^e has 7 significant bits, so it is exact in bf16 as well as in fp32.
//
// Why a power of two and a block of 32: an arbitrary scale max / 127 would use the code range fully
// (a power of two leaves its top code between 64 and 127) at the price of rounding the quotient;
// with one byte per 32 values the scales add 3 % to the bytes.
#pragma once
#include "tm_device.cuh"

namespace tml {

constexpr int kCk8Block = 32;

// exponent of a block whose largest finite magnitude has the fp32 bits `mbits`: m = f * 2^x with f
// in [0.5, 1) gives e = x - 7, or x - 6 when f > 127/128; the carry of the addition is that case.
__device__ __forceinline__ int ck8_exponent(uint32_t mbits) {
    const int e = (int)((mbits + 0x1FFFFu) >> 23) - 133;
    return e < -126 ? -126 : e;
}
__device__ __forceinline__ float ck8_scale(int e) { return __uint_as_float((uint32_t)(127 + max(e, -126)) << 23); }
__device__ __forceinline__ float ck8_inv_scale(int e) { return __uint_as_float((uint32_t)(127 - e) << 23); }

// The code of a finite |x * s| <= 127 in the low byte: adding 1.5 * 2^23 leaves the nearest integer
// (ties to even) in the low mantissa bits, two's complement.
__device__ __forceinline__ uint32_t ck8_code(float x, float s) { return __float_as_uint(fmaf(x, s, 12582912.f)); }
__device__ __forceinline__ bool nonfinite_bits(uint32_t b) { return (b & 0x7FFFFFFFu) >= 0x7F800000u; }

// Quantises one block spread over LB neighbouring lanes of a warp (aligned to LB), V values each
// (missing ones 0): codes packed four to a word in q (V == 1: in q[0]'s low byte), returns e.  All 32
// lanes of the warp call it together.
template <int V, int LB>
__device__ __forceinline__ int ck8_quantize(const float (&v)[V], uint32_t (&q)[(V + 3) / 4]) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 1; o < LB; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const bool odd = m > 0x7F7E0000u;     // above 127 * 2^121, or not finite
    if (__any_sync(0xffffffffu, odd)) {   // rare: the largest finite magnitude instead
        uint32_t f = 0u;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
            if (b < 0x7F800000u) f = max(f, b);
        }
#pragma unroll
        for (int o = 1; o < LB; o <<= 1) f = max(f, __shfl_xor_sync(0xffffffffu, f, o));
        m = f;
    }
    const int e = min(ck8_exponent(m), 121);
    const float s = ck8_inv_scale(e);
    uint32_t c[V];
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = ck8_code(v[i], s);
    if (odd) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            c[i] = nonfinite_bits(__float_as_uint(v[i])) ? 0x80u : ck8_code(fminf(fmaxf(v[i] * s, -127.f), 127.f), 1.f);
    }
    if (V == 1) {
        q[0] = c[0] & 0xFFu;
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const uint32_t lo = __byte_perm(c[(4 * i) % V], c[(4 * i + 1) % V], 0x0040);
            const uint32_t hi = __byte_perm(c[(4 * i + 2) % V], c[(4 * i + 3) % V], 0x0040);
            q[i] = __byte_perm(lo, hi, 0x5410);
        }
    }
    return e;
}

// The value of a code (a byte, two's complement) at scale s = 2^e.
__device__ __forceinline__ float ck8_value(uint32_t byte, float s) {
    const int c = (int)(int8_t)byte;
    return c == -128 ? __uint_as_float(0x7FC00000u) : (float)c * s;
}
template <int V>
__device__ __forceinline__ void ck8_values(const uint32_t (&q)[(V + 3) / 4], float s, float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = ck8_value((q[i / 4] >> (8 * (i % 4))) & 0xFFu, s);
}

// V codes to / from memory as one access (V = 1, 4 or 8 bytes, aligned to V).
template <int V>
__device__ __forceinline__ void ck8_store(int8_t* p, const uint32_t (&q)[(V + 3) / 4]) {
    if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(q[0], q[1]);
    else if constexpr (V == 4) *reinterpret_cast<uint32_t*>(p) = q[0];
    else *p = (int8_t)q[0];
}
template <int V>
__device__ __forceinline__ void ck8_load(const int8_t* p, uint32_t (&q)[(V + 3) / 4]) {
    if constexpr (V == 8) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
        q[0] = w.x;
        q[1] = w.y;
    } else if constexpr (V == 4) {
        q[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else {
        q[0] = (uint8_t)__ldg(p);
    }
}

// V values of storage type T to / from memory as one access.
template <typename T, int V>
struct Pack;
template <>
struct Pack<__nv_bfloat16, 8> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) { v[2 * i] = bf16_lo(a[i]); v[2 * i + 1] = bf16_hi(a[i]); }
    }
    __device__ __forceinline__ static void store(__nv_bfloat16* p, const float (&v)[8]) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
};
template <>
struct Pack<float, 4> {
    float4 w;
    __device__ __forceinline__ void load(const float* p) { w = __ldg(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void zero() { w = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&v)[4]) const { v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w; }
    __device__ __forceinline__ static void store(float* p, const float (&v)[4]) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <>
struct Pack<__nv_bfloat16, 1> {
    __nv_bfloat16 w;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = __ldg(p); }
    __device__ __forceinline__ void zero() { w = __float2bfloat16_rn(0.f); }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = __bfloat162float(w); }
    __device__ __forceinline__ static void store(__nv_bfloat16* p, const float (&v)[1]) { *p = __float2bfloat16_rn(v[0]); }
};
template <>
struct Pack<float, 1> {
    float w;
    __device__ __forceinline__ void load(const float* p) { w = __ldg(p); }
    __device__ __forceinline__ void zero() { w = 0.f; }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = w; }
    __device__ __forceinline__ static void store(float* p, const float (&v)[1]) { *p = v[0]; }
};

}  // namespace tml
