// tm_ckpt8.cu -- packing rows into 8-bit checkpoints and unpacking them (the format: tm_ckpt8.cuh).
//
// Both are one pass over the data, bound by memory: packing n bf16 values reads 2n bytes and writes
// n + n / 32.  134 M values: pack 66 us, unpack 64 (6.1 to 6.4 TB/s).  A thread handles U vectors of 16 bytes whose loads are all issued before the first is
// used; a block of 32 values is spread over 32 / V neighbouring lanes, which share its maximum by
// shuffles.
#include "tm_ckpt8.cuh"
#include "tm_internal.h"

namespace tml {

constexpr int kCk8Threads = 256;

// The vectors of a thread: unit u of a row holds its values u*V .. u*V + V-1; a row has upr units (its
// last block filled up to 32 / V of them).  FLAT: rows are whole blocks, so unit u of the whole tensor
// is its values u*V .. and block u / (32 / V).  Otherwise a thread's units, which are a grid's threads
// apart, advance row and unit by constants and a carry instead of a division each.  (Units are counted without a
// sign: a row of nearly 2^31 values, filled up to whole blocks, has 2^31 of them.)
template <typename T, int V, int U, bool PACK, bool FLAT>
__global__ void __launch_bounds__(kCk8Threads)
    ck8_kernel(T* __restrict__ x, int8_t* __restrict__ codes, int8_t* __restrict__ exps, long long rows, int width,
               int nblk) {
    constexpr int LB = kCk8Block / V;
    const uint32_t upr = (uint32_t)nblk * LB;
    const long long total = rows * upr;
    const long long nth = (long long)gridDim.x * blockDim.x;
    long long t0 = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    long long row = 0, drow = 0;
    uint32_t s = 0, ds = 0;
    if (!FLAT) {
        drow = nth / upr;
        ds = (uint32_t)(nth - drow * upr);
        row = t0 / upr;
        s = (uint32_t)(t0 - row * upr);
    }
    // t0 - lane is the warp's first unit: the loop is uniform across the warp (the shuffles need it)
    for (; t0 - (threadIdx.x & 31) < total; t0 += U * nth) {
        long long xo[U], eo[U];
        bool in[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (FLAT) {
                const long long u = t0 + i * nth;
                in[i] = u < total;
                xo[i] = u * V;
                eo[i] = u / LB;
            } else {
                in[i] = row < rows && s * V < (uint32_t)width;
                xo[i] = row * width + s * V;
                eo[i] = row * nblk + s / LB;
                row += drow;
                s += ds;
                if (s >= upr) { s -= upr; ++row; }
            }
        }
        const bool first = threadIdx.x % LB == 0;       // upr and nth are multiples of LB: a block's first lane
        if constexpr (PACK) {
            Pack<T, V> w[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (in[i]) w[i].load(x + xo[i]);
                else w[i].zero();
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                float2 v[Pairs<V>::N];
                w[i].get(v);
                uint32_t q[(V + 3) / 4];
                const int e = ck8_quantize<V, LB>(v, q);
                if (in[i]) {
                    ck8_store<V>(codes + xo[i], q);
                    if (first) exps[eo[i]] = (int8_t)e;
                }
            }
        } else {
            uint32_t q[U][(V + 3) / 4];
            int e[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (in[i]) {
                    ck8_load<V>(codes + xo[i], q[i]);
                    e[i] = __ldg(exps + eo[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (!in[i]) continue;
                float2 v[Pairs<V>::N];
                ck8_values<V>(q[i], ck8_scale(e[i]), v);
                Pack<T, V>::store(x + xo[i], v);
            }
        }
    }
}

template <typename T, int V, bool PACK>
static cudaError_t launch_ck8_one(void* x, void* codes, void* exps, long long rows, int width, int sms,
                                  cudaStream_t st) {
    constexpr int U = 4;
    const int nblk = ck8_blocks(width);
    const long long total = rows * nblk * (kCk8Block / V);
    const long long all = (total + kCk8Threads - 1) / kCk8Threads, per = (all + U - 1) / U;
    // small inputs: one unit a thread, so that all SMs take part
    long long grid = per > 2LL * sms ? per : (all < 2LL * sms ? all : 2LL * sms);
    if (grid > (1 << 20)) grid = 1 << 20;
    ProfileScope ps_(PACK ? "ckpt8_pack" : "ckpt8_unpack", st);
    if (V > 1 && width % kCk8Block == 0)
        ck8_kernel<T, V, U, PACK, (V > 1)><<<(int)grid, kCk8Threads, 0, st>>>((T*)x, (int8_t*)codes, (int8_t*)exps, rows, width, nblk);
    else
        ck8_kernel<T, V, U, PACK, false><<<(int)grid, kCk8Threads, 0, st>>>((T*)x, (int8_t*)codes, (int8_t*)exps, rows, width, nblk);
    return cudaGetLastError();
}

// pack: x -> codes, exps; else codes, exps -> x.  16-byte vectors when every row starts on one, else
// one value a thread.
cudaError_t launch_ckpt8(bool pack, int dtype, void* x, void* codes, void* exps, long long rows, int width, int sms,
                         cudaStream_t st) {
    if (dtype == 1) {
        if (width % 8 == 0)
            return pack ? launch_ck8_one<__nv_bfloat16, 8, true>(x, codes, exps, rows, width, sms, st)
                        : launch_ck8_one<__nv_bfloat16, 8, false>(x, codes, exps, rows, width, sms, st);
        return pack ? launch_ck8_one<__nv_bfloat16, 1, true>(x, codes, exps, rows, width, sms, st)
                    : launch_ck8_one<__nv_bfloat16, 1, false>(x, codes, exps, rows, width, sms, st);
    }
    if (width % 4 == 0)
        return pack ? launch_ck8_one<float, 4, true>(x, codes, exps, rows, width, sms, st)
                    : launch_ck8_one<float, 4, false>(x, codes, exps, rows, width, sms, st);
    return pack ? launch_ck8_one<float, 1, true>(x, codes, exps, rows, width, sms, st)
                : launch_ck8_one<float, 1, false>(x, codes, exps, rows, width, sms, st);
}

}  // namespace tml
