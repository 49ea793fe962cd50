// tm_ckpt8.cu -- packing rows into 8-bit checkpoints and unpacking them (the format: tm_ckpt8.cuh).
//
// Both are one pass over the data, bound by memory: packing n bf16 values reads 2n bytes and writes
// n + n / 32.  A thread handles U vectors of 16 bytes whose loads are all issued before the first is
// used; a block of 32 values is spread over 32 / V neighbouring lanes, which share its maximum by
// shuffles.
#include "tm_ckpt8.cuh"
#include "tm_internal.h"

namespace tml {

constexpr int kCk8Threads = 256;

// The vectors of a thread: unit u of a row holds its values u*V .. u*V + V-1; a row has upr units (its
// last block filled up to 32 / V of them).  A thread's units are a grid's threads apart, so row and
// unit advance by constants and a carry instead of a division each.
struct Ck8Walk {
    long long row;
    int s;
};

template <typename T, int V, int U, bool PACK>
__global__ void __launch_bounds__(kCk8Threads)
    ck8_kernel(T* __restrict__ x, int8_t* __restrict__ codes, int8_t* __restrict__ exps, long long rows, int width,
               int nblk) {
    constexpr int LB = kCk8Block / V;
    const int upr = nblk * LB;
    const long long total = rows * upr;
    const long long nth = (long long)gridDim.x * blockDim.x;
    const long long t0 = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const long long drow = nth / upr;
    const int ds = (int)(nth - drow * upr);
    Ck8Walk p{t0 / upr, 0};
    p.s = (int)(t0 - p.row * upr);
    // t0 - lane is the warp's first unit: the loop is uniform across the warp (the shuffles need it)
    for (long long wu = t0 - (threadIdx.x & 31); wu < total; wu += U * nth) {
        Ck8Walk at[U];
        bool in[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            at[i] = p;
            in[i] = p.row < rows && p.s * V < width;
            p.row += drow;
            p.s += ds;
            if (p.s >= upr) { p.s -= upr; ++p.row; }
        }
        if constexpr (PACK) {
            Pack<T, V> w[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (in[i]) w[i].load(x + at[i].row * width + at[i].s * V);
                else w[i].zero();
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                float v[V];
                w[i].get(v);
                uint32_t q[(V + 3) / 4];
                const int e = ck8_quantize<V, LB>(v, q);
                if (in[i]) {
                    ck8_store<V>(codes + at[i].row * width + at[i].s * V, q);
                    if (at[i].s % LB == 0) exps[at[i].row * nblk + at[i].s / LB] = (int8_t)e;
                }
            }
        } else {
            uint32_t q[U][(V + 3) / 4];
            int e[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                e[i] = 0;
                if (in[i]) {
                    ck8_load<V>(codes + at[i].row * width + at[i].s * V, q[i]);
                    e[i] = __ldg(exps + at[i].row * nblk + at[i].s / LB);
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (!in[i]) continue;
                float v[V];
                ck8_values<V>(q[i], ck8_scale(e[i]), v);
                Pack<T, V>::store(x + at[i].row * width + at[i].s * V, v);
            }
        }
    }
}

template <typename T, int V, bool PACK>
static cudaError_t launch_ck8_one(void* x, void* codes, void* exps, long long rows, int width, int sms,
                                  cudaStream_t st) {
    constexpr int U = 4;
    const int nblk = (width + kCk8Block - 1) / kCk8Block;
    const long long total = rows * nblk * (kCk8Block / V);
    const long long per = (long long)kCk8Threads * U;
    long long grid = (total + per - 1) / per;
    // small inputs: one unit a thread, so that all SMs take part
    if (grid < sms) grid = (total + kCk8Threads - 1) / kCk8Threads < sms ? (total + kCk8Threads - 1) / kCk8Threads : sms;
    if (grid > (1 << 20)) grid = 1 << 20;
    ProfileScope ps_(PACK ? "ckpt8_pack" : "ckpt8_unpack", st);
    ck8_kernel<T, V, U, PACK><<<(int)grid, kCk8Threads, 0, st>>>((T*)x, (int8_t*)codes, (int8_t*)exps, rows, width, nblk);
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
