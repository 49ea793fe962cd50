// tm_norm.cu -- layer normalisation of token rows, forward and backward.
//
//   z = x + residual;  mu = mean(z);  s = 1 / sqrt(mean((z - mu)^2) + eps);  n = (z - mu) s;
//   y = n * gain + bias
//   dn = dy * gain;  dz = s (dn - mean(dn) - n mean(dn n));  dgain = sum dy n;  dbias = sum dy
// x is read through a RowMap: the rows as they are, or the Mix view of a token tensor (the residual,
// y, dy and the saved rows are always plain rows [B, banks, W]).
//
// All of it is bound by memory: a row stays in registers between its statistics and its use, so each
// tensor crosses the bus once.  G threads share a row: 8 or 16 lanes for rows of at most 8 or 16
// vectors (so that narrow rows leave no lanes idle), a warp up to 1024 columns, 4 to 16 warps beyond.
// Statistics are two passes over the registers in fp32 (the mean first, then the centred squares): the
// one-pass form sum(z^2) - mean^2 loses the variance of rows whose mean is large.
#include <atomic>

#include "tm_ckpt8.cuh"
#include "tm_internal.h"

namespace tml {

// Sums of the G threads of a row (a power of two), the same in all of them and in a fixed order.
// G > 32: the whole block works on one row; `red` holds one float per warp and is free again after
// the next call's first barrier (two buffers in turn).
template <int G>
__device__ __forceinline__ float row_sum(float v, float* red, int& turn) {
    constexpr int L = G < 32 ? G : 32;
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (G > 32) {
        constexpr int NW = G / 32;
        float* r = red + turn * NW;
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) v += r[i];
    }
    return v;
}

struct NormParams {
    const void* x;
    const void* res;           // NULL: none
    const void* gain;          // NULL: ones
    const void* bias;          // NULL: zeros
    RowMap map;                // where x (and dx) lie
    int B;
    float eps;
    // forward
    void* y;
    float* mean;               // [B * banks], forward: may be NULL
    float* rstd;
    int8_t* codes;             // checkpoint of z, written by the forward, read by the backward (NULL: none)
    int8_t* exps;
    // backward
    const void* dy;
    void* dx;
    void* dres;                // mixed rows: the gradient of the residual rows (NULL: not wanted)
    float* part;               // [blocks][2][W] partial sums of dgain, dbias (NULL: not wanted)
};

template <int G>
struct NormBlock {
    static constexpr int THREADS = G > 32 ? G : 256;
    static constexpr int ROWS = THREADS / G;
};

// A row's statistics, checkpoint and output from its z in registers (the forward after its loads).
template <typename T, int V, int NV, int G>
__device__ __forceinline__ void ln_fwd_row(const NormParams& p, const float (&z)[NV][V], bool live, long long row,
                                           int gl, float* red, int& turn) {
    const int W = p.map.W;
    const size_t ro = (size_t)row * W;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) sum += z[i][k];
    const float mu = row_sum<G>(sum, red, turn) / (float)W;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if ((gl + G * i) * V < W) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float d = z[i][k] - mu;
                sq = fmaf(d, d, sq);
            }
        }
    }
    const float rs = 1.0f / sqrtf(row_sum<G>(sq, red, turn) / (float)W + p.eps);
    if (live && gl == 0) {
        if (p.mean) p.mean[row] = mu;
        if (p.rstd) p.rstd[row] = rs;
    }
    if (p.codes) {
        constexpr int LB = kCk8Block / V;
        const int nblk = (W + kCk8Block - 1) / kCk8Block;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (gl + G * i) * V;
            uint32_t q[(V + 3) / 4];
            const int e = ck8_quantize<V, LB>(z[i], q);
            if (live && c < W) {
                ck8_store<V>(p.codes + ro + c, q);
                if (c % kCk8Block == 0) p.exps[row * nblk + c / kCk8Block] = (int8_t)e;
            }
        }
    }
    if (!live) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (gl + G * i) * V;
        if (c >= W) continue;
        float g[V], o[V];
        Pack<T, V> w;
        if (p.gain) {
            w.load((const T*)p.gain + c);
            w.get(g);
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) g[k] = 1.f;
        }
        if (p.bias) w.load((const T*)p.bias + c);
        else w.zero();
        w.get(o);
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] = fmaf((z[i][k] - mu) * rs, g[k], o[k]);
        Pack<T, V>::store((T*)p.y + ro + c, o);
    }
}

// Forward: one row per G threads, NV vectors of V values a thread.
template <typename T, int V, int NV, int G>
__global__ void __launch_bounds__(NormBlock<G>::THREADS) ln_fwd_kernel(const NormParams p) {
    __shared__ float red[2 * (G > 32 ? G / 32 : 1)];
    int turn = 0;
    const int W = p.map.W;
    const int gl = threadIdx.x % G;
    const long long nrows = (long long)p.B * p.map.banks;
    const long long row = (long long)blockIdx.x * NormBlock<G>::ROWS + threadIdx.x / G;
    const bool live = row < nrows;          // lanes past the last row take part in the shuffles
    const int b = live ? (int)(row / p.map.banks) : 0;
    const int bank = live ? (int)(row - (long long)b * p.map.banks) : 0;
    const size_t ro = (size_t)(live ? row : 0) * W;
    Pack<T, V> xw[NV], rw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (gl + G * i) * V;
        xw[i].zero();
        rw[i].zero();
        if (live && c < W) {
            xw[i].load((const T*)p.x + row_elem(p.map, b, bank, c));
            if (p.res) rw[i].load((const T*)p.res + ro + c);
        }
    }
    float z[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float r[V];
        xw[i].get(z[i]);
        rw[i].get(r);
#pragma unroll
        for (int k = 0; k < V; ++k) z[i][k] += r[k];
    }
    ln_fwd_row<T, V, NV, G>(p, z, live, live ? row : 0, gl, red, turn);
}

// What the backward pass reads of one row: dy, and x (+ residual) or the checkpoint of their sum.
template <typename T, int V, int NV, bool CK>
struct NormRow {
    Pack<T, V> dw[NV];
    Pack<T, V> xw[CK ? 1 : NV], rw[CK ? 1 : NV];
    uint32_t q[CK ? NV : 1][(V + 3) / 4];
    int e[CK ? NV : 1];

    template <int G>
    __device__ __forceinline__ void load(const NormParams& p, bool live, long long row, int b, int bank, int gl) {
        const int W = p.map.W;
        const size_t ro = (size_t)row * W;
        const int nblk = (W + kCk8Block - 1) / kCk8Block;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (gl + G * i) * V;
            dw[i].zero();
            if constexpr (CK) {
                e[i] = 0;
#pragma unroll
                for (int k = 0; k < (V + 3) / 4; ++k) q[i][k] = 0u;
            } else {
                xw[i].zero();
                rw[i].zero();
            }
            if (live && c < W) {
                dw[i].load((const T*)p.dy + ro + c);
                if constexpr (CK) {
                    ck8_load<V>(p.codes + ro + c, q[i]);
                    e[i] = __ldg(p.exps + row * nblk + c / kCk8Block);
                } else {
                    xw[i].load((const T*)p.x + row_elem(p.map, b, bank, c));
                    if (p.res) rw[i].load((const T*)p.res + ro + c);
                }
            }
        }
    }
    // n = (z - mu) rs of vector i (columns past the row give values that are not used)
    __device__ __forceinline__ void normalised(int i, float mu, float rs, float (&n)[V]) const {
        if constexpr (CK) {
            ck8_values<V>(q[i], ck8_scale(e[i]), n);
        } else {
            float r[V];
            xw[i].get(n);
            rw[i].get(r);
#pragma unroll
            for (int k = 0; k < V; ++k) n[k] += r[k];
        }
#pragma unroll
        for (int k = 0; k < V; ++k) n[k] = (n[k] - mu) * rs;
    }
};

template <typename T, int V>
__device__ __forceinline__ void norm_gain(const NormParams& p, int c, float (&g)[V]) {
    if (p.gain) {
        Pack<T, V> w;
        w.load((const T*)p.gain + c);
        w.get(g);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) g[k] = 1.f;
    }
}

// One row of the backward pass: its dz by vectors handed to `emit`, its part of dgain and dbias added
// to dg and db.
template <typename T, int V, int NV, int G, bool CK, class Emit>
__device__ __forceinline__ void ln_bwd_row(const NormParams& p, const NormRow<T, V, NV, CK>& r, float mu, float rs,
                                           int gl, float* red, int& turn, float (&dg)[NV][V], float (&db)[NV][V],
                                           Emit emit) {
    const int W = p.map.W;
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (gl + G * i) * V;
        if (c < W) {
            float n[V], d[V], g[V];
            r.normalised(i, mu, rs, n);
            r.dw[i].get(d);
            norm_gain<T, V>(p, c, g);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                dg[i][k] = fmaf(d[k], n[k], dg[i][k]);
                db[i][k] += d[k];
                const float dn = d[k] * g[k];
                s1 += dn;
                s2 = fmaf(dn, n[k], s2);
            }
        }
    }
    const float m1 = row_sum<G>(s1, red, turn) / (float)W;
    const float m2 = row_sum<G>(s2, red, turn) / (float)W;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (gl + G * i) * V;
        if (c < W) {
            float n[V], d[V], g[V];
            r.normalised(i, mu, rs, n);
            r.dw[i].get(d);
            norm_gain<T, V>(p, c, g);
#pragma unroll
            for (int k = 0; k < V; ++k) d[k] = rs * (fmaf(d[k], g[k], -m1) - n[k] * m2);
            emit(c, d);
        }
    }
}

// The block's sums of dgain and dbias over its row groups, in a fixed order: through shared memory,
// one of the two at a time; sm holds ROWS * W floats.
template <int V, int NV, int G>
__device__ __forceinline__ void ln_store_partials(const NormParams& p, float* sm, int gl, const float (&dg)[NV][V],
                                                  const float (&db)[NV][V]) {
    constexpr int ROWS = NormBlock<G>::ROWS;
    const int W = p.map.W;
    float* out = p.part + (size_t)blockIdx.x * 2 * W;
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (gl + G * i) * V;
            if (c < W) {
#pragma unroll
                for (int k = 0; k < V; ++k) sm[(threadIdx.x / G) * W + c + k] = which == 0 ? dg[i][k] : db[i][k];
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < W; c += blockDim.x) {
            float s = 0.f;
            for (int r = 0; r < ROWS; ++r) s += sm[r * W + c];
            out[which * W + c] = s;
        }
    }
}

// Backward, one row per G threads at a time over a grid-stride of rows (a persistent grid, so that the
// sums of dgain and dbias stay in registers).
template <typename T, int V, int NV, int G, bool CK>
__global__ void __launch_bounds__(NormBlock<G>::THREADS) ln_bwd_kernel(const NormParams p) {
    extern __shared__ float sm[];
    __shared__ float red[2 * (G > 32 ? G / 32 : 1)];
    int turn = 0;
    constexpr int ROWS = NormBlock<G>::ROWS;
    const int W = p.map.W;
    const int gl = threadIdx.x % G;
    const long long nrows = (long long)p.B * p.map.banks;
    const bool mixed = p.map.layout == 1;
    float dg[NV][V], db[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) dg[i][k] = db[i][k] = 0.f;
    // the next row's loads are in flight while this one is worked on
    struct At {
        long long row;
        bool live;
        int b, bank;
        float mu, rs;
    };
    auto at = [&](long long base) -> At {
        At a;
        a.row = base + threadIdx.x / G;
        a.live = a.row < nrows;             // a group without a row works on zeros, which add nothing
        a.b = a.live ? (int)(a.row / p.map.banks) : 0;
        a.bank = a.live ? (int)(a.row - (long long)a.b * p.map.banks) : 0;
        a.mu = a.live ? __ldg(p.mean + a.row) : 0.f;
        a.rs = a.live ? __ldg(p.rstd + a.row) : 0.f;
        return a;
    };
    const long long step = (long long)gridDim.x * ROWS;
    long long base = (long long)blockIdx.x * ROWS;
    NormRow<T, V, NV, CK> rn;
    At an = at(base);
    rn.template load<G>(p, an.live, an.row, an.b, an.bank, gl);
    for (; base < nrows; base += step) {
        const NormRow<T, V, NV, CK> r = rn;
        const At a = an;
        if (base + step < nrows) {
            an = at(base + step);
            rn.template load<G>(p, an.live, an.row, an.b, an.bank, gl);
        }
        ln_bwd_row<T, V, NV, G, CK>(p, r, a.mu, a.rs, gl, red, turn, dg, db, [&](int c, const float(&d)[V]) {
            if (!a.live) return;
            Pack<T, V>::store((T*)p.dx + row_elem(p.map, a.b, a.bank, c), d);
            if (mixed && p.dres) Pack<T, V>::store((T*)p.dres + (size_t)a.row * W + c, d);
        });
    }
    if (p.part) ln_store_partials<V, NV, G>(p, sm, gl, dg, db);
}

// Backward of LN(Mix(X) + X) (T = H, W = D): dX = dz + Revert(dz), where an element of Revert(dz) comes
// from another row of the same sample.  A block works on one sample at a time: its warps turn the
// sample's rows into dz in shared memory (fp32), then all threads add the two parts and write dX.
template <typename T, int V, int NV, bool CK, int THREADS>
__global__ void __launch_bounds__(THREADS) ln_bwd_self_kernel(const NormParams p) {
    extern __shared__ float sm[];
    int turn = 0;
    const int W = p.map.W, H = p.map.banks, dh = p.map.dh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float dg[NV][V], db[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) dg[i][k] = db[i][k] = 0.f;
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        for (int h = warp; h < H; h += THREADS / 32) {
            const long long row = (long long)b * H + h;
            NormRow<T, V, NV, CK> r;
            const float mu = __ldg(p.mean + row), rs = __ldg(p.rstd + row);
            r.template load<32>(p, true, row, b, h, lane);
            ln_bwd_row<T, V, NV, 32, CK>(p, r, mu, rs, lane, nullptr, turn, dg, db, [&](int c, const float(&d)[V]) {
#pragma unroll
                for (int k = 0; k < V; k += 4)
                    *reinterpret_cast<float4*>(sm + (size_t)h * W + c + k) = make_float4(d[k], d[k + 1], d[k + 2], d[k + 3]);
            });
        }
        __syncthreads();
        const int nvec = H * W / V;
        T* out = (T*)p.dx + (size_t)b * H * W;
        for (int i = threadIdx.x; i < nvec; i += THREADS) {
            const int e = i * V;
            const int t = e / W, c = e - t * W;              // token t, column c = h * dh + j
            const int h = c / dh, j = c - h * dh;
            const float* a = sm + e;
            const float* r = sm + h * W + t * dh + j;        // row h of the Mix view holds it at t * dh + j
            float o[V];
#pragma unroll
            for (int k = 0; k < V; ++k) o[k] = a[k] + r[k];
            Pack<T, V>::store(out + e, o);
        }
        __syncthreads();
    }
    if (p.part) {
        // the warps' sums, in a fixed order; sm is free (the last barrier is behind every read)
        float* out = p.part + (size_t)blockIdx.x * 2 * W;
        // as many warps' rows as the sample's H * W floats hold at a time
        const int room = H < THREADS / 32 ? H : THREADS / 32;
        for (int which = 0; which < 2; ++which) {
            for (int w0 = 0; w0 < THREADS / 32; w0 += room) {
                __syncthreads();
                if (warp >= w0 && warp < w0 + room) {
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const int c = (lane + 32 * i) * V;
                        if (c < W) {
#pragma unroll
                            for (int k = 0; k < V; ++k) sm[(warp - w0) * W + c + k] = which == 0 ? dg[i][k] : db[i][k];
                        }
                    }
                }
                __syncthreads();
                const int n = min(room, THREADS / 32 - w0);
                for (int c = threadIdx.x; c < W; c += THREADS) {
                    float s = w0 == 0 ? 0.f : out[which * W + c];
                    for (int r = 0; r < n; ++r) s += sm[r * W + c];
                    out[which * W + c] = s;
                }
            }
        }
    }
}

// ------------------------------------------------------------------ whole samples: LN(Mix(X) + X)
// With T = H and X as the residual too, everything a sample's rows read is the sample itself, one
// contiguous piece of memory.  Blocks bring samples into shared memory by bulk copies, a ring of NB
// slots ahead of the arithmetic, so that the scattered reads of the Mix view (pieces of dh columns, one
// per token) cost shared-memory cycles instead of L1 lookups, and loads stay in flight while rows are
// worked on.  A token row of a slot is `ld` bytes, padded so that ld = dh * esz modulo 128: the pieces
// of 8 lanes then fall into different banks.
struct SampleRing {
    uint8_t* base;             // slots, then one barrier each
    uint64_t* full;
    uint32_t slot_bytes;
    int nb;
};

// Token rows of one sample (rows x bytes each, contiguous in memory) into a slot.  One thread.
__device__ __forceinline__ void sample_load(const SampleRing& r, int slot, const void* src, int rows, uint32_t bytes,
                                            uint32_t ld) {
    uint64_t* bar = r.full + slot;
    mbar_arrive_expect_tx(bar, rows * bytes);
    uint8_t* dst = r.base + slot * r.slot_bytes;
    for (int t = 0; t < rows; ++t) bulk_load(dst + t * ld, (const uint8_t*)src + (size_t)t * bytes, bytes, bar);
}

template <typename T, int V>
__device__ __forceinline__ void smem_vec(const uint8_t* p, float (&v)[V]) {
    Pack<T, V> w;
    w.w = *reinterpret_cast<const decltype(w.w)*>(p);
    w.get(v);
}

template <typename T, int V, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) ln_sample_fwd_kernel(const NormParams p, uint32_t ld, int nb) {
    extern __shared__ __align__(128) uint8_t sms[];
    __shared__ uint64_t bars[8];
    const int W = p.map.W, H = p.map.banks, dh = p.map.dh;
    const uint32_t bytes = W * sizeof(T);
    const SampleRing ring{sms, bars, H * ld, nb};
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int turn = 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < nb; ++i) mbar_init(&bars[i], 1);
        fence_barrier_init();
    }
    __syncthreads();
    const T* x = (const T*)p.x;
    const size_t per = (size_t)H * W;
    // load i of this block is sample blockIdx.x + i * gridDim.x, in slot i % nb
    const int mine = blockIdx.x < p.B ? (p.B - 1 - blockIdx.x) / gridDim.x + 1 : 0;
    if (threadIdx.x == 0)
        for (int i = 0; i < nb && i < mine; ++i)
            sample_load(ring, i, x + (blockIdx.x + (size_t)i * gridDim.x) * per, H, bytes, ld);
    // byte offsets of this lane's vectors in a token row, and of the Mix view's pieces
    int moff[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (lane + 32 * i) * V, t = c / dh;
        moff[i] = t * (int)ld + (c - t * dh) * (int)sizeof(T);
    }
    int slot = 0;
    uint32_t ph = 0;
    int done = 0;
    for (; done < mine; ++done) {
        const bool ok = mbar_wait(&bars[slot], ph, 0x810);
        if (!__syncthreads_and(ok)) break;
        const uint8_t* sx = sms + slot * ring.slot_bytes;
        const long long b = blockIdx.x + (long long)done * gridDim.x;
        for (int h = warp; h < H; h += THREADS / 32) {
            float z[NV][V];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (lane + 32 * i) * V;
#pragma unroll
                for (int k = 0; k < V; ++k) z[i][k] = 0.f;
                if (c < W) {
                    float r[V];
                    smem_vec<T, V>(sx + moff[i] + h * dh * (int)sizeof(T), z[i]);
                    smem_vec<T, V>(sx + h * ld + c * (int)sizeof(T), r);
#pragma unroll
                    for (int k = 0; k < V; ++k) z[i][k] += r[k];
                }
            }
            ln_fwd_row<T, V, NV, 32>(p, z, true, b * H + h, lane, nullptr, turn);
        }
        __syncthreads();
        if (threadIdx.x == 0 && done + nb < mine)
            sample_load(ring, slot, x + (b + (size_t)nb * gridDim.x) * per, H, bytes, ld);
        if (++slot == nb) { slot = 0; ph ^= 1; }
    }
    if (done < mine && threadIdx.x == 0)    // given up: the loads in flight land before the block ends
        for (int i = 0; i < nb && done + i < mine; ++i) {
            mbar_wait(&bars[slot], ph, 0x811);
            if (++slot == nb) { slot = 0; ph ^= 1; }
        }
}

// Backward of the same, dX = dz + Revert(dz).  Mix(X) + X is symmetric under exchange of a token and a
// head (its element (row h, column t * dh + j) is X[t][h * dh + j] + X[h][t * dh + j]), and so is dX:
// dX[t][h * dh + j] = dz[t][h * dh + j] + dz[h][t * dh + j] = dX[h][t * dh + j].  A sample takes two
// slots (X or the checkpoint's codes, and dy).  First its rows' two means, with dgain and dbias on the
// way, a warp a row; then every pair of elements once, from the same shared memory: dz is never stored.
template <typename T, int V, int NV, bool CK, int THREADS>
__global__ void __launch_bounds__(THREADS) ln_sample_bwd_kernel(const NormParams p, uint32_t ld, uint32_t ldc, int nb) {
    extern __shared__ __align__(128) uint8_t sms[];
    __shared__ uint64_t bars[8];
    constexpr int NW = THREADS / 32;
    const int W = p.map.W, H = p.map.banks, dh = p.map.dh;
    const int nblk = (W + kCk8Block - 1) / kCk8Block;
    constexpr int ES = sizeof(T);
    const uint32_t bytes = W * ES;
    const SampleRing ring{sms, bars, H * ld, nb};
    float4* rowc = reinterpret_cast<float4*>(sms + (size_t)nb * ring.slot_bytes);   // [H] {rs, mu, -rs m1, -rs^2 m2}
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int turn = 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < nb; ++i) mbar_init(&bars[i], 1);
        fence_barrier_init();
    }
    __syncthreads();
    const size_t per = (size_t)H * W;
    const int mine = blockIdx.x < p.B ? (p.B - 1 - blockIdx.x) / gridDim.x + 1 : 0;
    // load 2 i is sample i's X (or codes), load 2 i + 1 its dy; load l goes to slot l % nb
    auto load = [&](int l, int slot) {
        const size_t b = blockIdx.x + (size_t)(l >> 1) * gridDim.x;
        if (l & 1) sample_load(ring, slot, (const T*)p.dy + b * per, H, bytes, ld);
        else if (CK) sample_load(ring, slot, p.codes + b * per, H, W, ldc);
        else sample_load(ring, slot, (const T*)p.x + b * per, H, bytes, ld);
    };
    if (threadIdx.x == 0)
        for (int l = 0; l < nb && l < 2 * mine; ++l) load(l, l);
    float dg[NV][V], db[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) dg[i][k] = db[i][k] = 0.f;
    int moff[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (lane + 32 * i) * V, t = c / dh;
        moff[i] = t * (int)ld + (c - t * dh) * ES;
    }
    const int vpd = dh / V;                                // vectors of a piece
    const int npair = (H + 1) / 2 * (H + 1) * vpd;
    int slot = 0;
    uint32_t ph = 0;
    int done = 0;
    for (; done < mine; ++done) {
        const int slot2 = slot + 1 == nb ? 0 : slot + 1;
        const bool ok = mbar_wait(&bars[slot], ph, 0x812) && mbar_wait(&bars[slot2], slot2 ? ph : ph ^ 1, 0x813);
        if (!__syncthreads_and(ok)) break;
        const uint8_t* sx = sms + slot * ring.slot_bytes;
        const uint8_t* sd = sms + slot2 * ring.slot_bytes;
        const long long b = blockIdx.x + (long long)done * gridDim.x;
        const int8_t* ex = CK ? p.exps + b * H * nblk : nullptr;
        for (int h = warp; h < H; h += NW) {
            const float mu = __ldg(p.mean + b * H + h), rs = __ldg(p.rstd + b * H + h);
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (lane + 32 * i) * V;
                if (c < W) {
                    float n[V], d[V], g[V];
                    if constexpr (CK) {
                        uint32_t q[(V + 3) / 4];
                        if constexpr (V == 8) {
                            const uint2 w = *reinterpret_cast<const uint2*>(sx + h * ldc + c);
                            q[0] = w.x;
                            q[1] = w.y;
                        } else {
                            q[0] = *reinterpret_cast<const uint32_t*>(sx + h * ldc + c);
                        }
                        ck8_values<V>(q, ck8_scale(__ldg(ex + h * nblk + c / kCk8Block)), n);
                    } else {
                        float r[V];
                        smem_vec<T, V>(sx + moff[i] + h * dh * ES, n);
                        smem_vec<T, V>(sx + h * ld + c * ES, r);
#pragma unroll
                        for (int k = 0; k < V; ++k) n[k] += r[k];
                    }
                    smem_vec<T, V>(sd + h * ld + c * ES, d);
                    norm_gain<T, V>(p, c, g);
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        n[k] = (n[k] - mu) * rs;
                        dg[i][k] = fmaf(d[k], n[k], dg[i][k]);
                        db[i][k] += d[k];
                        const float dn = d[k] * g[k];
                        s1 += dn;
                        s2 = fmaf(dn, n[k], s2);
                    }
                }
            }
            const float m1 = row_sum<32>(s1, nullptr, turn) / (float)W;
            const float m2 = row_sum<32>(s2, nullptr, turn) / (float)W;
            if (lane == 0) rowc[h] = make_float4(rs, mu, -rs * m1, -rs * rs * m2);
        }
        __syncthreads();
        // pairs (t <= h): rows i and H-1-i of the triangle together are H + 1 pieces
        T* out = (T*)p.dx + b * per;
        for (int u = threadIdx.x; u < npair; u += THREADS) {
            const int j = u % vpd * V;
            const int k2 = u / vpd;
            const int i = k2 / (H + 1), k = k2 - i * (H + 1);
            int t, h;
            if (k < H - i) {
                t = i;
                h = i + k;
            } else {
                t = H - 1 - i;
                h = t + k - (H - i);
                if (t == i) continue;                      // odd H: the middle row is its own partner
            }
            const int ca = h * dh + j, cb = t * dh + j;
            float za[V], zb[V], da[V], dd[V], ga[V], gb[V];
            if constexpr (CK) {
                uint32_t q[(V + 3) / 4];
                auto codes = [&](int r, int c, float(&v)[V]) {
                    if constexpr (V == 8) {
                        const uint2 w = *reinterpret_cast<const uint2*>(sx + r * ldc + c);
                        q[0] = w.x;
                        q[1] = w.y;
                    } else {
                        q[0] = *reinterpret_cast<const uint32_t*>(sx + r * ldc + c);
                    }
                    ck8_values<V>(q, ck8_scale(__ldg(ex + r * nblk + c / kCk8Block)), v);
                };
                codes(t, ca, za);
                codes(h, cb, zb);
            } else {
                smem_vec<T, V>(sx + t * ld + ca * ES, za);
                smem_vec<T, V>(sx + h * ld + cb * ES, zb);
#pragma unroll
                for (int e = 0; e < V; ++e) za[e] = zb[e] = za[e] + zb[e];
            }
            smem_vec<T, V>(sd + t * ld + ca * ES, da);
            smem_vec<T, V>(sd + h * ld + cb * ES, dd);
            norm_gain<T, V>(p, ca, ga);
            norm_gain<T, V>(p, cb, gb);
            const float4 ra = rowc[t], rb = rowc[h];
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float a = fmaf(za[e] - ra.y, ra.w, fmaf(da[e] * ga[e], ra.x, ra.z));
                const float c = fmaf(zb[e] - rb.y, rb.w, fmaf(dd[e] * gb[e], rb.x, rb.z));
                o[e] = a + c;
            }
            Pack<T, V>::store(out + (size_t)t * W + ca, o);
            if (t != h) Pack<T, V>::store(out + (size_t)h * W + cb, o);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            if (2 * done + nb < 2 * mine) load(2 * done + nb, slot);
            if (2 * done + 1 + nb < 2 * mine) load(2 * done + 1 + nb, slot2);
        }
        slot += 2;
        if (slot >= nb) { slot -= nb; ph ^= 1; }
    }
    if (done < mine) {                       // given up: the loads in flight land before the block ends
        if (threadIdx.x == 0)
            for (int l = 2 * done; l < 2 * mine && l < 2 * done + nb; ++l) {
                mbar_wait(&bars[slot], ph, 0x814);
                if (++slot == nb) { slot = 0; ph ^= 1; }
            }
        return;
    }
    if (!p.part) return;
    // the warps' sums of dgain and dbias in a fixed order, through the slots (every read is behind the
    // last barrier): `room` warps' rows at a time
    float* sm = reinterpret_cast<float*>(sms);
    float* out = p.part + (size_t)blockIdx.x * 2 * W;
    const int fit = (int)((size_t)nb * ring.slot_bytes / (W * sizeof(float)));
    const int room = fit < NW ? fit : NW;
    for (int which = 0; which < 2; ++which) {
        for (int w0 = 0; w0 < NW; w0 += room) {
            __syncthreads();
            if (warp >= w0 && warp < w0 + room) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = (lane + 32 * i) * V;
                    if (c < W) {
#pragma unroll
                        for (int k = 0; k < V; ++k) sm[(warp - w0) * W + c + k] = which == 0 ? dg[i][k] : db[i][k];
                    }
                }
            }
            __syncthreads();
            const int n = min(room, NW - w0);
            for (int c = threadIdx.x; c < W; c += THREADS) {
                float s = w0 == 0 ? 0.f : out[which * W + c];
                for (int r = 0; r < n; ++r) s += sm[r * W + c];
                out[which * W + c] = s;
            }
        }
    }
}

// out0[c] = sum over n of part[n][0][c], out1[c] of part[n][1][c] (either may be NULL), fixed order: 8
// slices of the n partials per column, then the slices.  Grid: ceil(2 W / 32) blocks of 32 x 8 threads.
template <typename T>
__global__ void __launch_bounds__(256) norm_reduce_kernel(const float* __restrict__ part, int n, int W,
                                                          T* __restrict__ out0, T* __restrict__ out1) {
    __shared__ float sm[8][33];
    const int cx = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cx;
    float s = 0.f;
    if (c < 2 * W)
        for (int i = sl; i < n; i += 8) s += __ldg(part + (size_t)i * 2 * W + c);
    sm[sl][cx] = s;
    __syncthreads();
    if (sl == 0 && c < 2 * W) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sm[i][cx];
        T* o = c < W ? out0 : out1;
        if (o) from_f(s, o + (c < W ? c : c - W));
    }
}

// ------------------------------------------------------------------ launchers
// Rows of W columns in vectors of V: the threads per row G and vectors per thread NV.
#define TM_NORM_SIZES_8(X) X(8, 1, 8) X(8, 1, 16) X(8, 3, 8) X(8, 1, 32) X(8, 3, 16) X(8, 2, 32) X(8, 3, 32) X(8, 4, 32) X(8, 4, 128) X(8, 4, 512)
#define TM_NORM_SIZES_4(X) X(4, 1, 8) X(4, 1, 16) X(4, 1, 32) X(4, 3, 16) X(4, 2, 32) X(4, 3, 32) X(4, 4, 32) X(4, 8, 32) X(4, 8, 128) X(4, 8, 512)
#define TM_NORM_SIZES_1(X) X(1, 4, 32) X(1, 16, 32) X(1, 16, 128) X(1, 32, 512)

int norm_max_width() { return 16384; }

static int norm_vec(int dtype, int W) { return dtype == 1 ? (W % 8 == 0 ? 8 : 1) : (W % 4 == 0 ? 4 : 1); }

template <typename T>
static cudaError_t launch_ln_fwd_t(const NormParams& p, int vec, cudaStream_t st) {
    const long long nrows = (long long)p.B * p.map.banks;
#define X(V_, NV_, G_)                                                                                  \
    if (vec == V_ && p.map.W <= V_ * NV_ * G_) {                                                        \
        const long long grid = (nrows + NormBlock<G_>::ROWS - 1) / NormBlock<G_>::ROWS;                 \
        ln_fwd_kernel<T, V_, NV_, G_><<<(unsigned)grid, NormBlock<G_>::THREADS, 0, st>>>(p);            \
        return cudaGetLastError();                                                                      \
    }
    if constexpr (sizeof(T) == 2) { TM_NORM_SIZES_8(X) }
    else { TM_NORM_SIZES_4(X) }
    TM_NORM_SIZES_1(X)
#undef X
    return cudaErrorInvalidValue;
}

// ---- sample kernels (X the residual too): the ring's slots and block size
constexpr size_t kSampleSmem = 225 * 1024;
// bytes of a padded token row (piece: bytes of dh columns; a multiple of 16)
static uint32_t sample_ld(uint32_t bytes, uint32_t piece) {
    if (piece < 16) piece = 16;
    return bytes + (piece + 128 - bytes % 128) % 128;
}
// Slots for `need` at least and 4 at most: two blocks an SM where that leaves each the slots it wants.
static int sample_slots(size_t slot, size_t extra, int need) {
    const size_t half = kSampleSmem / 2 - extra, whole = kSampleSmem - extra;
    int nb = (int)(half / slot);
    if (nb < need + 1) nb = (int)(whole / slot);
    return nb < need ? 0 : (nb > 4 ? 4 : nb);
}
// Samples of at least 8 KB; smaller ones leave a block's threads idle, and the row kernels take them.
constexpr size_t kSampleLeast = 8 * 1024;

template <class K>
static cudaError_t norm_resident(K kern, int threads, size_t smem_most, std::atomic<int>* cache, int* per_sm);
static long long norm_bwd_blocks(long long nrows, int rows_per_block, int per_sm, size_t smem, int sms);

template <typename T, int V, int NV>
static cudaError_t launch_sample_fwd(const NormParams& p, uint32_t ld, int nb, int sms, cudaStream_t st) {
    constexpr int THREADS = 512;
    auto kern = ln_sample_fwd_kernel<T, V, NV, THREADS>;
    static std::atomic<int> cache[64];
    int per_sm = 0;
    cudaError_t e = norm_resident(kern, THREADS, kSampleSmem, cache, &per_sm);
    if (e != cudaSuccess) return e;
    const size_t smem = (size_t)nb * p.map.banks * ld;
    kern<<<(unsigned)norm_bwd_blocks(p.B, 1, per_sm, smem, sms), THREADS, smem, st>>>(p, ld, nb);
    return cudaGetLastError();
}
template <typename T>
static cudaError_t launch_sample_fwd_t(const NormParams& p, uint32_t ld, int nb, int sms, cudaStream_t st) {
    constexpr int V = sizeof(T) == 2 ? 8 : 4;
    const int nv = (p.map.W + 32 * V - 1) / (32 * V);
    if (nv == 1) return launch_sample_fwd<T, V, 1>(p, ld, nb, sms, st);
    if (nv == 2) return launch_sample_fwd<T, V, 2>(p, ld, nb, sms, st);
    if (nv == 3) return launch_sample_fwd<T, V, 3>(p, ld, nb, sms, st);
    if (nv == 4) return launch_sample_fwd<T, V, 4>(p, ld, nb, sms, st);
    if constexpr (V == 4) return launch_sample_fwd<T, V, 8>(p, ld, nb, sms, st);
    return cudaErrorInvalidValue;
}

template <typename T, int V, int NV, bool CK>
static cudaError_t launch_sample_bwd(const NormParams& p, uint32_t ld, uint32_t ldc, int nb, int sms, int* nblk,
                                     cudaStream_t st) {
    constexpr int THREADS = 512;
    auto kern = ln_sample_bwd_kernel<T, V, NV, CK, THREADS>;
    static std::atomic<int> cache[64];
    int per_sm = 0;
    cudaError_t e = norm_resident(kern, THREADS, kSampleSmem, cache, &per_sm);
    if (e != cudaSuccess) return e;
    const size_t smem = (size_t)nb * p.map.banks * ld + p.map.banks * sizeof(float4);
    const long long grid = norm_bwd_blocks(p.B, 1, per_sm, smem, sms);
    *nblk = (int)grid;
    kern<<<(unsigned)grid, THREADS, smem, st>>>(p, ld, ldc, nb);
    return cudaGetLastError();
}
template <typename T, bool CK>
static cudaError_t launch_sample_bwd_t(const NormParams& p, uint32_t ld, uint32_t ldc, int nb, int sms, int* nblk,
                                       cudaStream_t st) {
    constexpr int V = sizeof(T) == 2 ? 8 : 4;
    const int nv = (p.map.W + 32 * V - 1) / (32 * V);
    if (nv == 1) return launch_sample_bwd<T, V, 1, CK>(p, ld, ldc, nb, sms, nblk, st);
    if (nv == 2) return launch_sample_bwd<T, V, 2, CK>(p, ld, ldc, nb, sms, nblk, st);
    if (nv == 3) return launch_sample_bwd<T, V, 3, CK>(p, ld, ldc, nb, sms, nblk, st);
    if (nv == 4) return launch_sample_bwd<T, V, 4, CK>(p, ld, ldc, nb, sms, nblk, st);
    if constexpr (V == 4) return launch_sample_bwd<T, V, 8, CK>(p, ld, ldc, nb, sms, nblk, st);
    return cudaErrorInvalidValue;
}

cudaError_t launch_ln_fwd(int dtype, const NormParams& p, int sms, cudaStream_t st) {
    ProfileScope ps_("layer_norm", st);
    const int esz = dtype == 1 ? 2 : 4;
    if (p.map.layout == 1 && p.res == p.x && p.map.T == p.map.banks && p.map.W <= 1024 &&
        (size_t)p.map.banks * p.map.W * esz >= kSampleLeast) {
        const uint32_t ld = sample_ld(p.map.W * esz, p.map.dh * esz);
        const int nb = sample_slots((size_t)p.map.banks * ld, 0, 1);
        if (nb) return dtype == 1 ? launch_sample_fwd_t<__nv_bfloat16>(p, ld, nb, sms, st)
                                  : launch_sample_fwd_t<float>(p, ld, nb, sms, st);
    }
    const int vec = norm_vec(dtype, p.map.W);
    return dtype == 1 ? launch_ln_fwd_t<__nv_bfloat16>(p, vec, st) : launch_ln_fwd_t<float>(p, vec, st);
}

// Blocks per SM that the backward's persistent grid may have at most (its partial sums are sized by it).
constexpr int kNormBlocksPerSm = 4;

// Resident blocks per SM of a kernel without its dynamic shared memory, which is also allowed up to
// `smem_most` here; asked once per kernel (the caller's `cache`) and device.
template <class K>
static cudaError_t norm_resident(K kern, int threads, size_t smem_most, std::atomic<int>* cache, int* per_sm) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool keep = dev >= 0 && dev < 64;
    if (keep && (*per_sm = cache[dev].load(std::memory_order_acquire)) > 0) return cudaSuccess;
    if (smem_most > 48 * 1024) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_most);
        if (e != cudaSuccess) return e;
    }
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(per_sm, kern, threads, 0);
    if (e != cudaSuccess) return e;
    if (*per_sm < 1) *per_sm = 1;
    if (keep) cache[dev].store(*per_sm, std::memory_order_release);
    return cudaSuccess;
}

// Grid of a persistent launch: one block per `rows_per_block` rows, at most as many as are resident.
static long long norm_bwd_blocks(long long nrows, int rows_per_block, int per_sm, size_t smem, int sms) {
    const long long by_smem = (long long)((227 * 1024) / (smem + 1024));
    if (per_sm > by_smem) per_sm = (int)(by_smem > 0 ? by_smem : 1);
    if (per_sm > kNormBlocksPerSm) per_sm = kNormBlocksPerSm;
    const long long want = (nrows + rows_per_block - 1) / rows_per_block;
    const long long cap = (long long)per_sm * sms;
    return want < cap ? want : cap;
}

template <typename T, int V, int NV, int G, bool CK>
static cudaError_t launch_ln_bwd_one(const NormParams& p, int sms, int* nblk, cudaStream_t st) {
    constexpr int ROWS = NormBlock<G>::ROWS;
    const size_t smem = p.part ? (size_t)ROWS * p.map.W * sizeof(float) : 0;
    auto kern = ln_bwd_kernel<T, V, NV, G, CK>;
    static std::atomic<int> cache[64];
    int per_sm = 0;
    cudaError_t e = norm_resident(kern, NormBlock<G>::THREADS, (size_t)ROWS * V * NV * G * sizeof(float), cache, &per_sm);
    if (e != cudaSuccess) return e;
    const long long grid = norm_bwd_blocks((long long)p.B * p.map.banks, ROWS, per_sm, smem, sms);
    *nblk = (int)grid;
    kern<<<(unsigned)grid, NormBlock<G>::THREADS, smem, st>>>(p);
    return cudaGetLastError();
}

template <typename T, bool CK>
static cudaError_t launch_ln_bwd_t(const NormParams& p, int vec, int sms, int* nblk, cudaStream_t st) {
#define X(V_, NV_, G_) \
    if (vec == V_ && p.map.W <= V_ * NV_ * G_) return launch_ln_bwd_one<T, V_, NV_, G_, CK>(p, sms, nblk, st);
    if constexpr (sizeof(T) == 2) { TM_NORM_SIZES_8(X) }
    else { TM_NORM_SIZES_4(X) }
    TM_NORM_SIZES_1(X)
#undef X
    return cudaErrorInvalidValue;
}

constexpr int kSelfThreads = 512;
constexpr size_t kSelfSmem = 220 * 1024;

// The sample of LN(Mix(X) + X)'s backward has to fit the shared memory as fp32, a row one warp.
bool ln_self_supported(int H, int W) { return (size_t)H * W * 4 <= kSelfSmem && W <= 1024; }

template <typename T, int V, int NV, bool CK>
static cudaError_t launch_ln_self_one(const NormParams& p, int sms, int* nblk, cudaStream_t st) {
    const size_t smem = (size_t)p.map.banks * p.map.W * sizeof(float);
    auto kern = ln_bwd_self_kernel<T, V, NV, CK, kSelfThreads>;
    static std::atomic<int> cache[64];
    int per_sm = 0;
    cudaError_t e = norm_resident(kern, kSelfThreads, kSelfSmem, cache, &per_sm);
    if (e != cudaSuccess) return e;
    const long long grid = norm_bwd_blocks(p.B, 1, per_sm, smem, sms);
    *nblk = (int)grid;
    kern<<<(unsigned)grid, kSelfThreads, smem, st>>>(p);
    return cudaGetLastError();
}

template <typename T, bool CK>
static cudaError_t launch_ln_self_t(const NormParams& p, int sms, int* nblk, cudaStream_t st) {
    constexpr int V = sizeof(T) == 2 ? 8 : 4;
    const int W = p.map.W;
    if (W <= 32 * V) return launch_ln_self_one<T, V, 1, CK>(p, sms, nblk, st);
    if (W <= 64 * V) return launch_ln_self_one<T, V, 2, CK>(p, sms, nblk, st);
    if constexpr (V == 8) {
        if (W <= 96 * V) return launch_ln_self_one<T, V, 3, CK>(p, sms, nblk, st);
        return launch_ln_self_one<T, V, 4, CK>(p, sms, nblk, st);
    } else {
        if (W <= 128 * V) return launch_ln_self_one<T, V, 4, CK>(p, sms, nblk, st);
        return launch_ln_self_one<T, V, 8, CK>(p, sms, nblk, st);
    }
}

// Floats of the partial sums that the backward may write.
size_t ln_part_floats(long long nrows, int W, int sms) {
    const long long cap = (long long)kNormBlocksPerSm * sms;
    return (size_t)(nrows < cap ? nrows : cap) * 2 * W;
}

// self: x is the residual too (mixed rows), dx = dz + Revert(dz).  dgain, dbias: NULL where not wanted
// (p.part then NULL if neither is).
cudaError_t launch_ln_bwd(int dtype, const NormParams& p, bool self, void* dgain, void* dbias, int sms,
                          cudaStream_t st) {
    int nblk = 0;
    const bool ck = p.codes != nullptr;
    cudaError_t e;
    {
        ProfileScope ps_("layer_norm_bwd", st);
        const int vec = norm_vec(dtype, p.map.W), esz = dtype == 1 ? 2 : 4;
        const uint32_t ld = sample_ld(p.map.W * esz, p.map.dh * esz), ldc = sample_ld(p.map.W, p.map.dh);
        int nb = 0;
        if (self && (size_t)p.map.banks * p.map.W * esz >= kSampleLeast && (!ck || p.map.W % 16 == 0))
            nb = sample_slots((size_t)p.map.banks * ld, p.map.banks * sizeof(float4), 2);
        if (nb)
            e = dtype == 1 ? (ck ? launch_sample_bwd_t<__nv_bfloat16, true>(p, ld, ldc, nb, sms, &nblk, st)
                                 : launch_sample_bwd_t<__nv_bfloat16, false>(p, ld, ldc, nb, sms, &nblk, st))
                           : (ck ? launch_sample_bwd_t<float, true>(p, ld, ldc, nb, sms, &nblk, st)
                                 : launch_sample_bwd_t<float, false>(p, ld, ldc, nb, sms, &nblk, st));
        else if (self)
            e = dtype == 1 ? (ck ? launch_ln_self_t<__nv_bfloat16, true>(p, sms, &nblk, st)
                                 : launch_ln_self_t<__nv_bfloat16, false>(p, sms, &nblk, st))
                           : (ck ? launch_ln_self_t<float, true>(p, sms, &nblk, st)
                                 : launch_ln_self_t<float, false>(p, sms, &nblk, st));
        else
            e = dtype == 1 ? (ck ? launch_ln_bwd_t<__nv_bfloat16, true>(p, vec, sms, &nblk, st)
                                 : launch_ln_bwd_t<__nv_bfloat16, false>(p, vec, sms, &nblk, st))
                           : (ck ? launch_ln_bwd_t<float, true>(p, vec, sms, &nblk, st)
                                 : launch_ln_bwd_t<float, false>(p, vec, sms, &nblk, st));
        if (e != cudaSuccess) return e;
    }
    if (!p.part) return cudaSuccess;
    ProfileScope ps_("norm_reduce", st);
    const int grid = (2 * p.map.W + 31) / 32;
    if (dtype == 1)
        norm_reduce_kernel<<<grid, 256, 0, st>>>(p.part, nblk, p.map.W, (__nv_bfloat16*)dgain, (__nv_bfloat16*)dbias);
    else
        norm_reduce_kernel<<<grid, 256, 0, st>>>(p.part, nblk, p.map.W, (float*)dgain, (float*)dbias);
    return cudaGetLastError();
}

}  // namespace tml
