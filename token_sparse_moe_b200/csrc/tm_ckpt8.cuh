// tm_ckpt8.cuh -- 8-bit activation checkpoints: the format's device code, shared by the pack and
// unpack kernels and by the kernels that write or read a checkpoint in passing; and the paired fp32
// arithmetic of the row kernels.
//
// A row is cut into blocks of 32 values (the last one may be shorter).  With m the largest magnitude of
// a block, its scale is 2^e, e the smallest integer with m <= 127 * 2^e, at least -126 (so that 2^e and
// 2^-e are normal fp32 numbers) and at most 121 (so that 127 * 2^e is finite); a value's code is the
// nearest integer to x * 2^-e, ties to even, held to +-127 (which only binds above 127 * 2^121).
// Scaling by a power of two is exact, so the codes depend on x alone: two correct implementations give
// the same ones.  A block with a value that is not finite has e = 127 and codes 0, and reads back as NaN
// throughout: an overflow in the forward pass is not hidden from the backward pass, and reading costs no
// test per value (its scale is NaN).  A code times 2^e has 7 significant bits, so it is exact in bf16 as
// well as in fp32.
//
// Why a power of two and a block of 32: an arbitrary scale max / 127 would use the code range fully
// (a power of two leaves its top code between 64 and 127) at the price of rounding the quotient;
// with one byte per 32 values the scales add 3 % to the bytes.
//
// Instructions, not bytes, are what these kernels run out of first: at 6.5 TB/s an SM has about 25 issue
// slots per bf16 element read and written once.  So everything is done on pairs (Blackwell's two-wide
// fp32 add, multiply and fma), codes are rounded by adding 1.5 * 2^23 and read by placing the byte in the
// mantissa of 2^23, and maxima take three operands.
#pragma once
#include "tm_device.cuh"

namespace tml {

constexpr int kCk8Block = 32;
constexpr int kCk8NaN = 127;      // exponent of a block with a value that is not finite
// blocks of a row (the sum in 32 bits without a sign: a row may have 2^31 - 1 values)
__host__ __device__ constexpr int ck8_blocks(int width) { return (int)(((uint32_t)width + kCk8Block - 1) / kCk8Block); }

// Quotients by a fixed divisor d of 0 <= t < 2^31: (umulhi(m, t) + t) >> l, l = ceil(log2 d),
// m = floor(2^32 (2^l - d) / d) + 1 (division by an invariant integer through multiplication).
struct FastDiv {
    uint32_t d, m, l;
    __device__ __forceinline__ int div(int t) const { return (int)((__umulhi(m, (uint32_t)t) + (uint32_t)t) >> l); }
};
inline FastDiv fast_div(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    return FastDiv{d, (uint32_t)(((1ull << 32) * ((1ull << l) - d)) / d + 1), l};
}

// ------------------------------------------------------------------ pairs
__device__ __forceinline__ float2 f2(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
// max(m, |a.x|, |a.y|), NaN if any is
__device__ __forceinline__ float absmax3(float m, float2 a) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a.x), "f"(a.y));
    return r;
}

// V values of storage type T to / from memory as one access, as pairs.
template <typename T, int V>
struct Pack;
template <>
struct Pack<__nv_bfloat16, 8> {
    uint4 w;
    __device__ __forceinline__ void load(const void* p) { w = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void load_shared(const void* p) { w = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float2 (&v)[4]) const {
        v[0] = make_float2(bf16_lo(w.x), bf16_hi(w.x));
        v[1] = make_float2(bf16_lo(w.y), bf16_hi(w.y));
        v[2] = make_float2(bf16_lo(w.z), bf16_hi(w.z));
        v[3] = make_float2(bf16_lo(w.w), bf16_hi(w.w));
    }
    __device__ __forceinline__ static void store(__nv_bfloat16* p, const float2 (&v)[4]) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                                                  pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
    }
};
template <>
struct Pack<float, 4> {
    float4 w;
    __device__ __forceinline__ void load(const void* p) { w = __ldg(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void load_shared(const void* p) { w = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void zero() { w = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float2 (&v)[2]) const {
        v[0] = make_float2(w.x, w.y);
        v[1] = make_float2(w.z, w.w);
    }
    __device__ __forceinline__ static void store(float* p, const float2 (&v)[2]) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    }
};
// one value (the pair's second is 0 and is not stored): rows that start on no vector boundary
template <typename T>
struct Pack<T, 1> {
    T w;
    __device__ __forceinline__ void load(const void* p) { w = __ldg(reinterpret_cast<const T*>(p)); }
    __device__ __forceinline__ void zero() { from_f(0.f, &w); }
    __device__ __forceinline__ void get(float2 (&v)[1]) const { v[0] = make_float2(to_f(w), 0.f); }
    __device__ __forceinline__ static void store(T* p, const float2 (&v)[1]) { from_f(v[0].x, p); }
};
template <int V>
struct Pairs {
    static constexpr int N = (V + 1) / 2;
};

// ------------------------------------------------------------------ codes
// exponent of a block whose largest magnitude has the fp32 bits `mbits`: m = f * 2^x with f in [0.5, 1)
// gives e = x - 7, or x - 6 when f > 127/128; the carry of the addition is that case.
__device__ __forceinline__ int ck8_exponent(uint32_t mbits) { return max((int)((mbits + 0x1FFFFu) >> 23) - 133, -126); }
__device__ __forceinline__ float ck8_scale(int e) {
    return e == kCk8NaN ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)(127 + max(e, -126)) << 23);
}

// The rare blocks: not finite (codes 0, e = 127), or above 127 * 2^121 (held to +-127).
template <int NP>
__device__ __forceinline__ int ck8_quantize_rare(float2 (&v)[NP], uint32_t mbits) {
    const bool bad = mbits >= 0x7F800000u;
    const float s = __uint_as_float((uint32_t)(127 - 121) << 23);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        v[i].x = bad ? 0.f : fminf(fmaxf(v[i].x * s, -127.f), 127.f);
        v[i].y = bad ? 0.f : fminf(fmaxf(v[i].y * s, -127.f), 127.f);
    }
    return bad ? kCk8NaN : 121;
}

// Quantises one block spread over LB neighbouring lanes of a warp (aligned to LB), V values each as pairs
// (missing ones 0): codes packed four to a word in q (V == 1: in q[0]'s low byte), returns e.  All 32
// lanes of the warp call it together.
template <int V, int LB>
__device__ __forceinline__ int ck8_quantize(const float2 (&v)[Pairs<V>::N], uint32_t (&q)[(V + 3) / 4]) {
    constexpr int NP = Pairs<V>::N;
    float mf = 0.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) mf = absmax3(mf, v[i]);
    uint32_t m = __float_as_uint(mf);              // magnitudes order as their bits do, NaN above all
    if constexpr (LB == 32) {
        m = __reduce_max_sync(0xffffffffu, m);
    } else {
#pragma unroll
        for (int o = 1; o < LB; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    int e = ck8_exponent(m);
    float2 c[NP];
    const float2 magic = f2(12582912.f);           // 1.5 * 2^23: the nearest integer in the low bits
    if (__any_sync(0xffffffffu, m > 0x7F7E0000u)) {
        float2 t[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) t[i] = v[i];
        float s = __uint_as_float((uint32_t)(127 - min(e, 121)) << 23);
        if (m > 0x7F7E0000u) {
            e = ck8_quantize_rare<NP>(t, m);
            s = 1.f;
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) c[i] = fma2(t[i], f2(s), magic);
    } else {
        const float2 s = f2(__uint_as_float((uint32_t)(127 - e) << 23));
#pragma unroll
        for (int i = 0; i < NP; ++i) c[i] = fma2(v[i], s, magic);
    }
    if constexpr (V == 1) {
        q[0] = __float_as_uint(c[0].x) & 0xFFu;
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const uint32_t lo = __byte_perm(__float_as_uint(c[2 * i].x), __float_as_uint(c[2 * i].y), 0x0040);
            const uint32_t hi = __byte_perm(__float_as_uint(c[2 * i + 1].x), __float_as_uint(c[2 * i + 1].y), 0x0040);
            q[i] = __byte_perm(lo, hi, 0x5410);
        }
    }
    return e;
}

// Codes as integers in fp32: 2^23 + (code + 128) is the byte (top bit flipped) in the mantissa of 2^23.
template <int V>
__device__ __forceinline__ void ck8_codes(const uint32_t (&q)[(V + 3) / 4], float2 (&v)[Pairs<V>::N]) {
    const float2 off = f2(-8388736.f);
#pragma unroll
    for (int i = 0; i < Pairs<V>::N; ++i) {
        const uint32_t w = q[i / 2] ^ 0x80808080u;
        const int b = 2 * (i & 1);
        v[i] = add2(make_float2(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540 + b)),
                                __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7541 + b))), off);
    }
    if constexpr (V == 1) v[0].y = 0.f;
}
template <int V>
__device__ __forceinline__ void ck8_values(const uint32_t (&q)[(V + 3) / 4], float s, float2 (&v)[Pairs<V>::N]) {
    ck8_codes<V>(q, v);
#pragma unroll
    for (int i = 0; i < Pairs<V>::N; ++i) v[i] = mul2(v[i], f2(s));
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
template <int V>
__device__ __forceinline__ void ck8_load_shared(const uint8_t* p, uint32_t (&q)[(V + 3) / 4]) {
    if constexpr (V == 8) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        q[0] = w.x;
        q[1] = w.y;
    } else {
        q[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

}  // namespace tml
