// tm_linear.cu -- the per-token linear layer beside its tensor-core contractions (tm_linear.cuh): the forward
// of one sample, the activation's derivative with the bias gradient's column sums, the sums of partial results, the fp32
// form of the contractions on CUDA cores, and the launchers.
#include <string.h>

#include <atomic>

#include "tm_linear.cuh"
#include "tm_internal.h"

namespace tml {

// ------------------------------------------------------------------ activations in fp32
// The fp32 path calls the CUDA math functions; bf16 results take the short forms of tm_linear.cuh.
__device__ __forceinline__ float act_f32(int act, float z) {
    if (act == LIN_RELU) return max_nan(z, 0.f);
    if (act == LIN_GELU) return 0.5f * z * erfcf(-0.70710678118654752f * z);
    if (act == LIN_SILU) return z / (1.f + expf(-z));
    return z;
}
// act'(z): gelu' = Phi(z) + z phi(z); silu' = s (1 + z (1 - s)), s = sigmoid(z).  ACT is a template
// parameter of the pass over dy so that its inner loop has no branches.
template <typename T, int ACT>
__device__ __forceinline__ float2 act_slope2(float2 z) {
    if constexpr (ACT == LIN_RELU)            // NaN stays
        return make_float2(z.x > 0.f ? 1.f : (z.x == z.x ? 0.f : z.x), z.y > 0.f ? 1.f : (z.y == z.y ? 0.f : z.y));
    if constexpr (ACT == LIN_GELU && sizeof(T) == 4) {
        auto f = [](float v) {
            return fmaf(v * 0.39894228040143268f, expf(-0.5f * v * v), 0.5f * erfcf(-0.70710678118654752f * v));
        };
        return make_float2(f(z.x), f(z.y));
    }
    if constexpr (ACT == LIN_SILU && sizeof(T) == 4) {
        auto f = [](float v) {
            const float s = 1.f / (1.f + expf(-v));
            return s * fmaf(v, 1.f - s, 1.f);
        };
        return make_float2(f(z.x), f(z.y));
    }
    if constexpr (ACT == LIN_GELU) {
        // gelu'(-a) = Q(a) - a phi(a) = 1 - gelu'(a) = exp(-a^2 / 2) (M(a) - a / sqrt(2 pi)), a >= 0, with
        // M(a) = Q(a) / exp(-a^2 / 2) a polynomial of degree 4 in r = 1 / (1 + p a), the form of Abramowitz and
        // Stegun's 26.2.17, fitted here towards the smallest maximum of the absolute error up to a = 1.5 and of the
        // relative one from there to 13.5: 1.5e-6 absolutely, and in the negative tail 1.5e-4 of the slope itself, as
        // far as exp(-a^2 / 2) is a normal number.  (A polynomial in a alone takes degree 9 and more for that.)
        // a' = -a sqrt(log2(e) / 2) makes the exponent -a'^2, and with M in units of the factor of a' the sum needs no
        // product: exp2(-(a'^2 + c)) (2^c M + a'), 2^-c = sqrt(ln 2 / pi).  Past the normal numbers the
        // exponential is 0 and the sum finite; of a NaN or an infinity the slope is NaN.
        const float2 a = make_float2(-0.8493218f * fabsf(z.x), -0.8493218f * fabsf(z.y));
        const float2 x = fma2(a, a, f2(1.09013125f));
        float2 u = fma2(a, f2(-0.50601883f), f2(1.f));
        const float2 r = make_float2(rcp_approx(u.x), rcp_approx(u.y));
        u = fma2(f2(-0.253971815f), r, f2(0.748718917f));
        u = fma2(u, r, f2(0.175845459f));
        u = fma2(u, r, f2(0.393871248f));
        u = fma2(u, r, a);
        const float2 t = mul2(u, make_float2(ex2_approx(-x.x), ex2_approx(-x.y)));
        return make_float2(z.x < 0.f ? t.x : 1.f - t.x, z.y < 0.f ? t.y : 1.f - t.y);
    }
    if constexpr (ACT == LIN_SILU) {
        const float2 x = mul2(z, f2(-1.4426950408889634f));
        const float2 s = make_float2(rcp_approx(1.f + ex2_approx(x.x)), rcp_approx(1.f + ex2_approx(x.y)));
        return mul2(s, fma2(z, fma2(s, f2(-1.f), f2(1.f)), f2(1.f)));
    }
    return f2(1.f);
}

// ------------------------------------------------------------------ dz = dy act'(z), db = sum over b of dz
// dy, z, dz are [B, cols] with cols = banks * N; a thread owns V columns and walks down its block's
// rows; the sums over a block's rows go to part [gridDim.y][cols] (in a fixed order).  SRC: what z is
// read from.  dz may be NULL (no activation: dz is dy, only the sums are wanted).
// One pass, bound by memory: 8192 x 48 x 1536 bf16 with z whole 562 us with silu (6.4 TB/s), 585 with gelu; from the
// checkpoint 500 and 523 (a sixth fewer bytes, but the codes' conversion and the slope then take as long as the bus);
// under the power cap, between the two contractions, 590 to 620 and 620 to 680.
// dz is rounded to bf16, the operand type of both contractions that read it: its half step, 2^-8, is of the
// size of the one in y and dominates the error of dx and dw.
enum ZSrc : int { Z_NONE = 0, Z_FULL = 1, Z_CK8 = 2 };
constexpr int kActX = 64, kActY = 4;

template <typename T, int V, int SRC, int ACT>
__global__ void __launch_bounds__(kActX * kActY)
    act_bwd_kernel(const T* __restrict__ dy, const T* __restrict__ z, const int8_t* __restrict__ codes,
                   const int8_t* __restrict__ exps, int B, long long cols, int N, int nblk, int rows_per,
                   T* __restrict__ dz, float* __restrict__ part) {
    constexpr int NP = Pairs<V>::N, U = 4;
    __shared__ float2 sm[kActY][kActX][NP + 1];          // + 1: rows of a column's pairs in different banks
    const int tx = threadIdx.x % kActX, ty = threadIdx.x / kActX;
    const long long c = ((long long)blockIdx.x * kActX + tx) * V;
    const bool in = c < cols;
    const long long bank = in ? c / N : 0;
    const int n = in ? (int)(c - bank * N) : 0;
    const long long erow = cols / N * nblk;              // exponents per b
    const long long eoff = bank * nblk + n / kCk8Block;
    const int b0 = blockIdx.y * rows_per, b1 = min(B, b0 + rows_per);
    float2 s[NP];
#pragma unroll
    for (int k = 0; k < NP; ++k) s[k] = make_float2(0.f, 0.f);
    if (in) {
        for (int b = b0 + ty; b < b1; b += kActY * U) {
            Pack<T, V> dw[U], zw[SRC == Z_FULL ? U : 1];
            uint32_t q[SRC == Z_CK8 ? U : 1][(V + 3) / 4];
            int e[SRC == Z_CK8 ? U : 1];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = b + u * kActY;
                if (r >= b1) continue;
                dw[u].load(dy + r * cols + c);
                if constexpr (SRC == Z_FULL) zw[u].load(z + r * cols + c);
                if constexpr (SRC == Z_CK8) {
                    ck8_load<V>(codes + r * cols + c, q[u]);
                    e[u] = __ldg(exps + r * erow + eoff);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = b + u * kActY;
                if (r >= b1) continue;
                float2 d[NP];
                dw[u].get(d);
                if constexpr (SRC != Z_NONE) {
                    float2 zv[NP];
                    if constexpr (SRC == Z_FULL) zw[u].get(zv);
                    else ck8_values<V>(q[u], ck8_scale(e[u]), zv);
#pragma unroll
                    for (int k = 0; k < NP; ++k) d[k] = mul2(d[k], act_slope2<T, ACT>(zv[k]));
                    Pack<T, V>::store(dz + r * cols + c, d);
                }
#pragma unroll
                for (int k = 0; k < NP; ++k) s[k] = add2(s[k], d[k]);
            }
        }
    }
    if (!part) return;
#pragma unroll
    for (int k = 0; k < NP; ++k) sm[ty][tx][k] = s[k];
    __syncthreads();
    if (ty == 0 && in) {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            float2 t = make_float2(0.f, 0.f);
#pragma unroll
            for (int y = 0; y < kActY; ++y) t = add2(t, sm[y][tx][k]);
            float* o = part + blockIdx.y * cols + c + 2 * k;
            o[0] = t.x;
            if (V > 1) o[1] = t.y;
        }
    }
}

// out[i] = sum over r < R of part[r][i], in order
template <typename T>
__global__ void __launch_bounds__(256) sum_parts_kernel(const float* __restrict__ part, int R, long long n,
                                                        T* __restrict__ out) {
    const bool vec = (n & 3) == 0;
    const long long n4 = vec ? n / 4 : n;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n4; i += (long long)gridDim.x * 256) {
        if (vec) {
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int r = 0; r < R; ++r) {
                const float4 w = __ldg(reinterpret_cast<const float4*>(part + r * n) + i);
                s.x += w.x; s.y += w.y; s.z += w.z; s.w += w.w;
            }
            from_f(s.x, out + 4 * i);
            from_f(s.y, out + 4 * i + 1);
            from_f(s.z, out + 4 * i + 2);
            from_f(s.w, out + 4 * i + 3);
        } else {
            float s = 0.f;
            for (int r = 0; r < R; ++r) s += __ldg(part + r * n + i);
            from_f(s, out + i);
        }
    }
}

// The same for many parts of few columns (the bias gradient's): a block takes 32 columns, eight slices of the
// parts side by side, then the slices in order.  64 parts of 12288 columns: 9 us, 12 with a thread a column;
// for up to 8 parts (a split contraction's, of many columns) the slices would be a part each.
template <typename T>
__global__ void __launch_bounds__(256) sum_parts_tall_kernel(const float* __restrict__ part, int R, long long n,
                                                             T* __restrict__ out) {
    __shared__ float sm[8][33];
    const int cx = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const long long c = (long long)blockIdx.x * 32 + cx;
    float s = 0.f;
    if (c < n)
#pragma unroll 8
        for (int r = sl; r < R; r += 8) s += __ldg(part + r * n + c);
    sm[sl][cx] = s;
    __syncthreads();
    if (sl == 0 && c < n) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sm[i][cx];
        from_f(s, out + c);
    }
}

// ------------------------------------------------------------------ fp32 contractions
// D[g][m][n] = sum_k A[g][m][k] B[g][n][k] with every stride given, 64 x 64 tiles, slabs of 16, 4 x 4
// outputs a thread; the forward's epilogue as in tm_linear.cuh.  The path of the small fp32 stack: exact
// products in fp32, no tensor cores.  256 x 16 banks x 256 -> 256 27 us, 4096 x 16 x 512 -> 512 28 TFLOP/s,
// about a third of the CUDA cores' rate: bound by the shared-memory reads of a 4 x 4 tile.
struct SimtLin {
    const float *a, *b, *bias, *add;
    float *d, *z;
    int8_t *codes, *exps;
    long long ag, am, ak, bg, bn, bk, dg, dm;   // element strides (D's columns are contiguous)
    int groups, M, N, K, act, nblk;
};

__global__ void __launch_bounds__(256) linear_simt_kernel(const SimtLin p) {
    __shared__ float sa[16][68], sb[16][68];
    const int g = blockIdx.z, m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const float* A = p.a + g * p.ag;
    const float* Bm = p.b + g * p.bg;
    float acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    for (int k0 = 0; k0 < p.K; k0 += 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // the contiguous index runs across the threads
            const int e = threadIdx.x + 256 * i;
            const int ak = p.ak == 1 ? e & 15 : e >> 6, am = p.ak == 1 ? e >> 4 : e & 63;
            const int bk = p.bk == 1 ? e & 15 : e >> 6, bn = p.bk == 1 ? e >> 4 : e & 63;
            sa[ak][am] = (m0 + am < p.M && k0 + ak < p.K) ? __ldg(A + (m0 + am) * p.am + (k0 + ak) * p.ak) : 0.f;
            sb[bk][bn] = (n0 + bn < p.N && k0 + bk < p.K) ? __ldg(Bm + (n0 + bn) * p.bn + (k0 + bk) * p.bk) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            float av[4], bv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) { av[i] = sa[k][ty * 4 + i]; bv[i] = sb[k][tx * 4 + i]; }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + ty * 4 + i, n = n0 + tx * 4;
        const bool row_in = m < p.M;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (p.bias && n + j < p.N) acc[i][j] += __ldg(p.bias + (long long)g * p.N + n + j);
        const long long r = (long long)m * p.groups + g;      // row of the forward's rows
        if (p.codes) {
            uint32_t q[1];
            const float2 v2[2] = {make_float2(acc[i][0], acc[i][1]), make_float2(acc[i][2], acc[i][3])};
            const int e = ck8_quantize<4, 8>(v2, q);          // a block of 32 columns: 8 lanes
            if (row_in) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + j < p.N) p.codes[r * p.N + n + j] = (int8_t)(q[0] >> (8 * j));
                if ((n & 31) == 0 && n < p.N) p.exps[r * p.nblk + (n >> 5)] = (int8_t)e;
            }
        }
        if (!row_in) continue;
        const long long o = g * p.dg + m * p.dm + n;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (n + j >= p.N) break;
            if (p.z) p.z[o + j] = acc[i][j];
            float y = act_f32(p.act, acc[i][j]);
            if (p.add) y += __ldg(p.add + o + j);
            p.d[o + j] = y;
        }
    }
}

// ------------------------------------------------------------------ one sample
// The bf16 forward of a single sample, where the weights' one pass through memory is all there is.  A block
// owns 32 columns of a bank (one block of the checkpoint's codes), a warp four of them, its lanes along the
// contraction in vectors of 8, eight vectors of weights in flight a lane; sums in fp32, joined by shuffles in
// a fixed order; then the first warp has a column a lane.  No tile, barrier or x from shared memory: 48 banks of
// 768 -> 1536 take 20.7 us (5.5 TB/s of weights; the tensor-core tiles 24.1), 40 of 1024 -> 2048 28.5 (37.7), 1 of
// 1024 -> 2048 4.1 (9.0).  From two samples on, their x and sums crowd out the loads (33 us to the tiles' 22).
struct RowLin {
    const __nv_bfloat16 *x, *w, *bias, *res;
    __nv_bfloat16 *y, *z;
    int8_t *codes, *exps;
    int K, N, nblk;
};

template <int ACT, int SAVE>
__global__ void __launch_bounds__(256, 4) linear_row_kernel(const RowLin p) {
    __shared__ float sums[32];
    constexpr int U = 2;
    const int bank = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n0 = blockIdx.x * 32, kv = p.K / 8;
    const size_t o = (size_t)bank * p.N + n0 + lane;
    const bool in = warp == 0 && n0 + lane < p.N;
    float bias = 0.f, res = 0.f;
    if (in && p.bias) bias = to_f(__ldg(p.bias + o));
    if (in && p.res) res = to_f(__ldg(p.res + o));
    float sum = 0.f;                                       // of column 4 warp + (lane >> 3) in every lane
    if (n0 + 4 * warp < p.N) {                             // N is a multiple of 8: whole fours
        const __nv_bfloat16* w = p.w + ((size_t)bank * p.N + n0 + 4 * warp) * p.K;
        const __nv_bfloat16* x = p.x + (size_t)bank * p.K;
        float2 acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = make_float2(0.f, 0.f);
        for (int c0 = lane; c0 < kv; c0 += 32 * U) {
            Pack<__nv_bfloat16, 8> wv[U][4], xw[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + 32 * u < kv) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) wv[u][j].load(w + (size_t)j * p.K + (c0 + 32 * u) * 8);
                    xw[u].load(x + (c0 + 32 * u) * 8);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + 32 * u < kv) {
                    float2 xv[4];
                    xw[u].get(xv);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float2 v[4];
                        wv[u][j].get(v);
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[j] = fma2(v[k], xv[k], acc[j]);
                    }
                }
        }
        // four sums over the warp: halves exchanged, so that after two steps a lane holds one column's
        float t[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) t[j] = acc[j].x + acc[j].y;
        const bool h1 = lane & 16, h0 = lane & 8;
        const float a = (h1 ? t[2] : t[0]) + __shfl_xor_sync(0xffffffffu, h1 ? t[0] : t[2], 16);
        const float b = (h1 ? t[3] : t[1]) + __shfl_xor_sync(0xffffffffu, h1 ? t[1] : t[3], 16);
        sum = (h0 ? b : a) + __shfl_xor_sync(0xffffffffu, h0 ? a : b, 8);
#pragma unroll
        for (int k = 4; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    }
    if ((lane & 7) == 0) sums[4 * warp + (lane >> 3)] = sum;
    __syncthreads();
    if (warp != 0) return;
    float v = in ? sums[lane] + bias : 0.f;
    if constexpr (SAVE == LIN_KEEP_CK8) {
        const float2 one[1] = {make_float2(v, 0.f)};
        uint32_t q[1];
        const int e = ck8_quantize<1, 32>(one, q);
        if (in) p.codes[o] = (int8_t)q[0];
        if (lane == 0) p.exps[bank * p.nblk + blockIdx.x] = (int8_t)e;
    }
    if (!in) return;
    if constexpr (SAVE == LIN_KEEP_FULL) p.z[o] = __float2bfloat16(v);
    p.y[o] = __float2bfloat16(lin_act2<ACT>(make_float2(v, 0.f)).x + res);
}

cudaError_t launch_linear_row(int banks, int act, int save, const RowLin& p, cudaStream_t st) {
    ProfileScope ps_("linear_row", st);
    const dim3 grid((p.N + 31) / 32, banks);
#define X(ACT_, SAVE_) \
    if (act == ACT_ && (act == LIN_NONE || save == SAVE_)) linear_row_kernel<ACT_, SAVE_><<<grid, 256, 0, st>>>(p);
    X(LIN_NONE, LIN_KEEP_NOTHING)
    X(LIN_RELU, LIN_KEEP_NOTHING) X(LIN_RELU, LIN_KEEP_FULL) X(LIN_RELU, LIN_KEEP_CK8)
    X(LIN_GELU, LIN_KEEP_NOTHING) X(LIN_GELU, LIN_KEEP_FULL) X(LIN_GELU, LIN_KEEP_CK8)
    X(LIN_SILU, LIN_KEEP_NOTHING) X(LIN_SILU, LIN_KEEP_FULL) X(LIN_SILU, LIN_KEEP_CK8)
#undef X
    return cudaGetLastError();
}

// ------------------------------------------------------------------ launchers
cudaError_t launch_linear_simt(const SimtLin& p, cudaStream_t st) {
    ProfileScope ps_("linear_f32", st);
    const dim3 grid((p.N + 63) / 64, (p.M + 63) / 64, p.groups);
    linear_simt_kernel<<<grid, 256, 0, st>>>(p);
    return cudaGetLastError();
}

template <int BN, bool PAIR, bool A_MN, bool B_MN, int ACT, int SAVE, bool F32OUT>
static cudaError_t launch_linear_one(const LinMaps& m, const LinParams& p, int sms, cudaStream_t st) {
    using C = LinCfg<BN, PAIR>;
    auto kern = linear_gemm_kernel<BN, PAIR, A_MN, B_MN, ACT, SAVE, F32OUT>;
    static std::atomic<bool> configured[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev].store(true, std::memory_order_release);
    }
    ProfileScope ps_(A_MN ? "linear_dw" : B_MN ? "linear_dx" : "linear", st);
    if (!PAIR) {
        kern<<<p.ntile < sms ? p.ntile : sms, C::NTHREADS, C::SMEM_BYTES, st>>>(m.a, m.b, m.o, m.r, p);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3((unsigned)(2 * (p.ntile < sms / 2 ? p.ntile : sms / 2)), 1, 1);
    cfg.blockDim = dim3(C::NTHREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, m.a, m.b, m.o, m.r, p);
}

// The two shapes of tile: pairs of 256 x 256, single CTAs of 128 x 128.
template <bool A_MN, bool B_MN, int ACT, int SAVE, bool F32OUT>
static cudaError_t launch_linear_shape(bool pair, const LinMaps& m, const LinParams& p, int sms, cudaStream_t st) {
    if (pair) return launch_linear_one<256, true, A_MN, B_MN, ACT, SAVE, F32OUT>(m, p, sms, st);
    return launch_linear_one<128, false, A_MN, B_MN, ACT, SAVE, F32OUT>(m, p, sms, st);
}

cudaError_t launch_linear_fwd(bool pair, int act, int save, const LinMaps& m, const LinParams& p, int sms,
                              cudaStream_t st) {
    if (act == LIN_NONE) return launch_linear_shape<false, false, LIN_NONE, LIN_KEEP_NOTHING, false>(pair, m, p, sms, st);
#define X(ACT_, SAVE_) \
    if (act == ACT_ && save == SAVE_) return launch_linear_shape<false, false, ACT_, SAVE_, false>(pair, m, p, sms, st);
    X(LIN_RELU, LIN_KEEP_NOTHING) X(LIN_RELU, LIN_KEEP_FULL) X(LIN_RELU, LIN_KEEP_CK8)
    X(LIN_GELU, LIN_KEEP_NOTHING) X(LIN_GELU, LIN_KEEP_FULL) X(LIN_GELU, LIN_KEEP_CK8)
    X(LIN_SILU, LIN_KEEP_NOTHING) X(LIN_SILU, LIN_KEEP_FULL) X(LIN_SILU, LIN_KEEP_CK8)
#undef X
    return cudaErrorInvalidValue;
}
cudaError_t launch_linear_dx(bool pair, const LinMaps& m, const LinParams& p, int sms, cudaStream_t st) {
    return launch_linear_shape<false, true, LIN_NONE, LIN_KEEP_NOTHING, false>(pair, m, p, sms, st);
}
// more than one split: fp32 partial sums
cudaError_t launch_linear_dw(bool pair, const LinMaps& m, const LinParams& p, int sms, cudaStream_t st) {
    if (p.splits.d > 1) return launch_linear_shape<true, true, LIN_NONE, LIN_KEEP_NOTHING, true>(pair, m, p, sms, st);
    return launch_linear_shape<true, true, LIN_NONE, LIN_KEEP_NOTHING, false>(pair, m, p, sms, st);
}

cudaError_t launch_sum_parts(int dtype, const float* part, int R, long long n, void* out, cudaStream_t st) {
    ProfileScope ps_("sum_parts", st);
    if (R > 8 && n <= (1LL << 24)) {
        const int grid = (int)((n + 31) / 32);
        if (dtype == 1) sum_parts_tall_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(part, R, n, (__nv_bfloat16*)out);
        else sum_parts_tall_kernel<float><<<grid, 256, 0, st>>>(part, R, n, (float*)out);
        return cudaGetLastError();
    }
    const long long per = (n & 3) == 0 ? n / 4 : n;
    const long long grid = (per + 255) / 256 < 148 * 16 ? (per + 255) / 256 : 148 * 16;
    if (dtype == 1) sum_parts_kernel<__nv_bfloat16><<<(int)grid, 256, 0, st>>>(part, R, n, (__nv_bfloat16*)out);
    else sum_parts_kernel<float><<<(int)grid, 256, 0, st>>>(part, R, n, (float*)out);
    return cudaGetLastError();
}

// Row chunks of the derivative pass: enough blocks for every SM several times over, at least 16 rows
// each, at most 64 partial sums per column.
int act_bwd_chunks(int dtype, int B, long long cols, int N, int sms) {
    const int V = dtype == 1 ? 8 : (N % 4 == 0 ? 4 : 1);
    const long long gx = (cols / V + kActX - 1) / kActX;
    long long r = (8LL * sms + gx - 1) / gx;
    if (r > (B + 15) / 16) r = (B + 15) / 16;
    if (r > 64) r = 64;
    return (int)(r < 1 ? 1 : r);
}

template <typename T, int V>
static void launch_act_bwd_v(const void* dy, const void* z, const int8_t* codes, const int8_t* exps, int act, int B,
                             long long cols, int N, int chunks, void* dz, float* part, cudaStream_t st) {
    const dim3 grid((unsigned)((cols / V + kActX - 1) / kActX), chunks);
    const int per = (B + chunks - 1) / chunks;
    const int nblk = (N + kCk8Block - 1) / kCk8Block;
#define X(SRC_, ACT_)                                                                                       \
    act_bwd_kernel<T, V, SRC_, ACT_><<<grid, kActX * kActY, 0, st>>>((const T*)dy, (const T*)z, codes, exps, B, cols, \
                                                                     N, nblk, per, (T*)dz, part)
    if (act == LIN_NONE) X(Z_NONE, LIN_NONE);
    else if (codes && act == LIN_RELU) X(Z_CK8, LIN_RELU);
    else if (codes && act == LIN_GELU) X(Z_CK8, LIN_GELU);
    else if (codes) X(Z_CK8, LIN_SILU);
    else if (act == LIN_RELU) X(Z_FULL, LIN_RELU);
    else if (act == LIN_GELU) X(Z_FULL, LIN_GELU);
    else X(Z_FULL, LIN_SILU);
#undef X
}

cudaError_t launch_act_bwd(int dtype, const void* dy, const void* z, const int8_t* codes, const int8_t* exps, int act,
                           int B, long long cols, int N, int chunks, void* dz, float* part, cudaStream_t st) {
    ProfileScope ps_("act_bwd", st);
    if (dtype == 1)
        launch_act_bwd_v<__nv_bfloat16, 8>(dy, z, codes, exps, act, B, cols, N, chunks, dz, part, st);
    else if (N % 4 == 0)
        launch_act_bwd_v<float, 4>(dy, z, codes, exps, act, B, cols, N, chunks, dz, part, st);
    else
        launch_act_bwd_v<float, 1>(dy, z, codes, exps, act, B, cols, N, chunks, dz, part, st);
    return cudaGetLastError();
}

}  // namespace tml
