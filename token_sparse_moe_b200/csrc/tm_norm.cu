// tm_norm.cu -- layer normalisation of token rows, forward and backward.
//
//   z = x + residual;  mu = mean(z);  s = 1 / sqrt(mean((z - mu)^2) + eps);  n = (z - mu) s;
//   y = n * gain + bias
//   dn = dy * gain;  dz = s (dn - mean(dn) - n mean(dn n));  dgain = sum dy n;  dbias = sum dy
// x is read through a RowMap: the rows as they are, or the Mix view of a token tensor (the residual,
// y, dy and the saved rows are always plain rows [B, banks, W]).
//
// A row stays in registers between its statistics and its use, so each tensor crosses the bus once.  G
// threads share a row: 8 or 16 lanes for rows of at most 8 or 16 vectors (so that narrow rows leave few
// lanes idle), a warp up to 1024 columns, 4 to 16 warps beyond.  Grids are persistent: gain and bias sit in
// shared memory as fp32, the sums of dgain and dbias in registers, and the next row's loads are in flight
// while a row is worked on.  What is then left to bound them is the issue of instructions as much as memory
// (see tm_ckpt8.cuh): the arithmetic is in pairs throughout.  4096 x 16 rows of 1024 bf16 with a residual, nothing
// in the L2 (kernels alone): forward 61 us (6.6 TB/s), with the checkpoint 78 (quantising is as much arithmetic as the
// norm); backward from x and the residual 100 (5.4 TB/s), from the checkpoint 78 (4.3).  Rows of the Mix view with a
// residual of their own, 4096 x 48 x 768 (pieces of 16 columns): forward 140, backward 288, from the checkpoint 192.
// Statistics are two passes over the registers in fp32 (the mean first, then the centred squares): the
// one-pass form sum(z^2) - mean^2 loses the variance of rows whose mean is large.
#include <atomic>

#include "tm_ckpt8.cuh"
#include "tm_internal.h"

namespace tml {

// Sums of the G threads of a row (a power of two), the same in all of them and in a fixed order.
// G > 32: the whole block works on one row; `red` holds one pair per warp and is free again after
// the next call's barrier (two buffers in turn).
template <int G>
__device__ __forceinline__ float2 row_sum2(float2 v, float2* red, int& turn) {
    constexpr int L = G < 32 ? G : 32;
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1)
        v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
    if constexpr (G > 32) {
        constexpr int NW = G / 32;
        float2* r = red + turn * NW;
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
        __syncthreads();
        v = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NW; ++i) v = add2(v, r[i]);
    }
    return v;
}
template <int G>
__device__ __forceinline__ float row_sum(float v, float2* red, int& turn) {
    if constexpr (G > 32) return row_sum2<G>(make_float2(v, 0.f), red, turn).x;
    constexpr int L = G < 32 ? G : 32;
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct NormParams {
    const void* x;
    const void* res;           // NULL: none
    const void* gain;          // NULL: ones
    const void* bias;          // NULL: zeros
    RowMap map;                // where x (and dx) lie
    int B;
    float eps, inv_w;          // 1 / W
    FastDiv banks;             // row = b * banks + bank
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
    static constexpr int THREADS = G > 32 ? G : 128;
    static constexpr int ROWS = THREADS / G;
};

// Where a thread's vectors lie in a row of x: from the row's start in the row layout, from the sample's
// head piece in the mixed one (column c = t * dh + j at t * D + j).
template <int V, int NV, int G>
struct NormCols {
    int off[NV];
    __device__ __forceinline__ NormCols(const RowMap& m, int gl) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (gl + G * i) * V;
            off[i] = c;
            if (m.layout == 1) {
                const int t = c / m.dh;
                off[i] = t * m.D + c - t * m.dh;
            }
        }
    }
};
// Start of a row of x (rows <= 2^28).
__device__ __forceinline__ size_t norm_row(const NormParams& p, int row) {
    if (p.map.layout == 0) return (size_t)row * p.map.W;
    const int b = p.banks.div(row);
    return (size_t)b * p.map.T * p.map.D + (size_t)(row - b * (int)p.banks.d) * p.map.dh;
}

// A vector of gain or bias [W] in shared memory as fp32.  V = 8: the two halves of each vector apart, so
// that neighbouring lanes read neighbouring 16 bytes.
template <typename T, int V>
__device__ __forceinline__ void stage_vec(float* s, const void* g, int W, float none) {
    for (int c = threadIdx.x; c < W; c += blockDim.x) {
        const int at = V == 8 ? (c & 4 ? W / 2 : 0) + (c >> 3) * 4 + (c & 3) : c;
        s[at] = g ? to_f(__ldg((const T*)g + c)) : none;
    }
}
template <int V>
__device__ __forceinline__ void staged(const float* s, int W, int c, float2 (&v)[Pairs<V>::N]) {
    if constexpr (V == 1) {
        v[0] = make_float2(s[c], 0.f);
    } else {
        const float4 a = *reinterpret_cast<const float4*>(s + (V == 8 ? (c >> 3) * 4 : c));
        v[0] = make_float2(a.x, a.y);
        v[1] = make_float2(a.z, a.w);
        if constexpr (V == 8) {
            const float4 b = *reinterpret_cast<const float4*>(s + W / 2 + (c >> 3) * 4);
            v[2] = make_float2(b.x, b.y);
            v[3] = make_float2(b.z, b.w);
        }
    }
}

// A row's statistics, checkpoint and output from its z in registers (zeros past the row).
template <typename T, int V, int NV, int G>
__device__ __forceinline__ void ln_fwd_row(const NormParams& p, float2 (&z)[NV][Pairs<V>::N], bool live, int row,
                                           int gl, const float* sg, const float* sb, float2* red, int& turn) {
    constexpr int NP = Pairs<V>::N;
    const int W = p.map.W;
    const size_t ro = (size_t)row * W;
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < NP; ++k) s2 = add2(s2, z[i][k]);
    const float mu = row_sum<G>(s2.x + s2.y, red, turn) * p.inv_w;
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
                if (c % kCk8Block == 0) p.exps[(size_t)row * nblk + c / kCk8Block] = (int8_t)e;
            }
        }
    }
    // z - mu in place of z
    s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if ((gl + G * i) * V < W) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                z[i][k] = add2(z[i][k], f2(-mu));
                if (V == 1) z[i][k].y = 0.f;
                s2 = fma2(z[i][k], z[i][k], s2);
            }
        }
    }
    const float rs = rsqrtf(row_sum<G>(s2.x + s2.y, red, turn) * p.inv_w + p.eps);
    if (!live) return;
    if (gl == 0) {
        if (p.mean) p.mean[row] = mu;
        if (p.rstd) p.rstd[row] = rs;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (gl + G * i) * V;
        if (c >= W) continue;
        float2 g[NP], o[NP];
        staged<V>(sg, W, c, g);
        staged<V>(sb, W, c, o);
#pragma unroll
        for (int k = 0; k < NP; ++k) o[k] = fma2(mul2(z[i][k], f2(rs)), g[k], o[k]);
        Pack<T, V>::store((T*)p.y + ro + c, o);
    }
}

// Forward: one row per G threads at a time, NV vectors of V values a thread.  Dynamic shared memory: gain
// and bias.
template <typename T, int V, int NV, int G>
__global__ void __launch_bounds__(NormBlock<G>::THREADS) ln_fwd_kernel(const NormParams p) {
    extern __shared__ __align__(16) float nsm[];
    __shared__ float2 red[2 * (G > 32 ? G / 32 : 1)];
    constexpr int NP = Pairs<V>::N, ROWS = NormBlock<G>::ROWS;
    int turn = 0;
    const int W = p.map.W;
    const int gl = threadIdx.x % G;
    const int nrows = p.B * p.map.banks;
    const int step = gridDim.x * ROWS;
    const NormCols<V, NV, G> cols(p.map, gl);
    Pack<T, V> xw[NV], rw[NV];
    auto load = [&](int row) {
        const bool live = row < nrows;      // lanes past the last row take part in the shuffles, on zeros
        const T* x = (const T*)p.x + norm_row(p, live ? row : 0);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (gl + G * i) * V;
            xw[i].zero();
            rw[i].zero();
            if (live && c < W) {
                xw[i].load(x + cols.off[i]);
                if (p.res) rw[i].load((const T*)p.res + (size_t)row * W + c);
            }
        }
    };
    int base = blockIdx.x * ROWS;
    load(base + threadIdx.x / G);
    float *sg = nsm, *sb = nsm + W;
    stage_vec<T, V>(sg, p.gain, W, 1.f);
    stage_vec<T, V>(sb, p.bias, W, 0.f);
    __syncthreads();
    for (; base < nrows; base += step) {
        float2 z[NV][NP];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float2 r[NP];
            xw[i].get(z[i]);
            rw[i].get(r);
#pragma unroll
            for (int k = 0; k < NP; ++k) z[i][k] = add2(z[i][k], r[k]);
        }
        const int row = base + threadIdx.x / G;
        if (base + step < nrows) load(row + step);
        const bool live = row < nrows;
        ln_fwd_row<T, V, NV, G>(p, z, live, live ? row : 0, gl, sg, sb, red, turn);
    }
}

// What the backward pass reads of one row: dy, and x (+ residual) or the checkpoint of their sum.
template <typename T, int V, int NV, bool CK>
struct NormRow {
    static constexpr int NP = Pairs<V>::N;
    Pack<T, V> dw[NV];
    Pack<T, V> xw[CK ? 1 : NV], rw[CK ? 1 : NV];
    uint32_t q[CK ? NV : 1][(V + 3) / 4];
    int e[CK ? NV : 1];

    template <int G>
    __device__ __forceinline__ void load(const NormParams& p, bool live, int row, const NormCols<V, NV, G>& cols, int gl) {
        const int W = p.map.W;
        const size_t ro = (size_t)row * W;
        const T* x = CK ? nullptr : (const T*)p.x + norm_row(p, row);
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
                    e[i] = __ldg(p.exps + (size_t)row * nblk + c / kCk8Block);
                } else {
                    xw[i].load(x + cols.off[i]);
                    if (p.res) rw[i].load((const T*)p.res + ro + c);
                }
            }
        }
    }
    // n = (z - mu) rs of vector i (columns past the row give values that are not used)
    __device__ __forceinline__ void normalised(int i, float mu, float rs, float2 (&n)[NP]) const {
        if constexpr (CK) {
            // code * 2^e is exact, so z - mu is rounded once, whatever the mean (code * (2^e rs) - mu rs, a
            // multiplication less, is off by |mu| rs roundings)
            ck8_codes<V>(q[i], n);
            const float a = ck8_scale(e[i]);
#pragma unroll
            for (int k = 0; k < NP; ++k) n[k] = mul2(fma2(n[k], f2(a), f2(-mu)), f2(rs));
        } else {
            float2 r[NP];
            xw[i].get(n);
            rw[i].get(r);
#pragma unroll
            for (int k = 0; k < NP; ++k) n[k] = mul2(add2(add2(n[k], r[k]), f2(-mu)), f2(rs));
        }
    }
};

// One row of the backward pass: its dz by vectors handed to `emit`, its part of dgain and dbias added
// to dg and db.  Up to 24 values a thread, n and dn stay in registers between the sums and dz; beyond
// that they are made again.
template <typename T, int V, int NV, int G, bool CK, class Emit>
__device__ __forceinline__ void ln_bwd_row(const NormParams& p, const NormRow<T, V, NV, CK>& r, float mu, float rs,
                                           int gl, const float* sg, float2* red, int& turn,
                                           float2 (&dg)[NV][Pairs<V>::N], float2 (&db)[NV][Pairs<V>::N], Emit emit) {
    constexpr int NP = Pairs<V>::N;
    constexpr bool KEEP = V * NV <= 24;
    const int W = p.map.W;
    float2 n[KEEP ? NV : 1][NP], dn[KEEP ? NV : 1][NP];
    auto make = [&](int i, int c, float2(&nn)[NP], float2(&dd)[NP], float2(&d)[NP]) {
        float2 g[NP];
        r.normalised(i, mu, rs, nn);
        r.dw[i].get(d);
        staged<V>(sg, W, c, g);
#pragma unroll
        for (int k = 0; k < NP; ++k) dd[k] = mul2(d[k], g[k]);
    };
    float2 s1 = make_float2(0.f, 0.f), s2 = s1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (gl + G * i) * V, a = KEEP ? i : 0;
        if (c < W) {
            float2 d[NP];
            make(i, c, n[a], dn[a], d);
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                dg[i][k] = fma2(d[k], n[a][k], dg[i][k]);
                db[i][k] = add2(db[i][k], d[k]);
                s1 = add2(s1, dn[a][k]);
                s2 = fma2(dn[a][k], n[a][k], s2);
            }
        }
    }
    const float2 m = row_sum2<G>(make_float2(s1.x + s1.y, s2.x + s2.y), red, turn);
    const float2 m1 = f2(-rs * (m.x * p.inv_w)), m2 = f2(-rs * (m.y * p.inv_w));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (gl + G * i) * V, a = KEEP ? i : 0;
        if (c < W) {
            float2 d[NP];
            if (!KEEP) make(i, c, n[a], dn[a], d);
#pragma unroll
            for (int k = 0; k < NP; ++k) d[k] = fma2(dn[a][k], f2(rs), fma2(n[a][k], m2, m1));
            emit(i, c, d);
        }
    }
}

template <int V, int NV>
__device__ __forceinline__ void zero_sums(float2 (&dg)[NV][Pairs<V>::N], float2 (&db)[NV][Pairs<V>::N]) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < Pairs<V>::N; ++k) dg[i][k] = db[i][k] = make_float2(0.f, 0.f);
}

// The block's sums of dgain and dbias over its row groups (group grp's thread gl holds columns (gl + G i) V ..),
// in a fixed order: through shared memory, one of the two at a time and `room` groups at a time; sm holds
// room * W floats and is free when this is called.
template <int V, int NV, int G>
__device__ __forceinline__ void ln_store_partials(const NormParams& p, float* sm, int room, int groups, int grp, int gl,
                                                  const float2 (&dg)[NV][Pairs<V>::N],
                                                  const float2 (&db)[NV][Pairs<V>::N]) {
    const int W = p.map.W;
    float* out = p.part + (size_t)blockIdx.x * 2 * W;
    for (int which = 0; which < 2; ++which) {
        for (int g0 = 0; g0 < groups; g0 += room) {
            __syncthreads();
            if (grp >= g0 && grp < g0 + room) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = (gl + G * i) * V;
                    if (c < W) {
                        float* o = sm + (grp - g0) * W + c;
#pragma unroll
                        for (int k = 0; k < Pairs<V>::N; ++k) {
                            const float2 v = which == 0 ? dg[i][k] : db[i][k];
                            o[2 * k] = v.x;
                            if (V > 1) o[2 * k + 1] = v.y;
                        }
                    }
                }
            }
            __syncthreads();
            const int n = min(room, groups - g0);
            for (int c = threadIdx.x; c < W; c += blockDim.x) {
                float s = g0 == 0 ? 0.f : out[which * W + c];
                for (int r = 0; r < n; ++r) s += sm[r * W + c];
                out[which * W + c] = s;
            }
        }
    }
}

// Backward, one row per G threads at a time.  Dynamic shared memory: gain, then (p.part) ROWS * W floats.
template <typename T, int V, int NV, int G, bool CK>
__global__ void __launch_bounds__(NormBlock<G>::THREADS) ln_bwd_kernel(const NormParams p) {
    extern __shared__ __align__(16) float nsm[];
    __shared__ float2 red[2 * (G > 32 ? G / 32 : 1)];
    constexpr int NP = Pairs<V>::N, ROWS = NormBlock<G>::ROWS;
    // loads a row ahead where the registers allow it
    constexpr bool AHEAD = V * NV * (int)sizeof(T) <= (CK ? 64 : 48);
    int turn = 0;
    const int W = p.map.W;
    const int gl = threadIdx.x % G;
    const int nrows = p.B * p.map.banks;
    const bool mixed = p.map.layout == 1;
    const NormCols<V, NV, G> cols(p.map, gl);
    float2 dg[NV][NP], db[NV][NP];
    zero_sums<V, NV>(dg, db);
    struct At {
        int row;                            // < 0: a group without a row, on zeros, which add nothing
        float mu, rs;
    };
    NormRow<T, V, NV, CK> rn;
    auto fetch = [&](int base) -> At {
        At a;
        const int row = base + threadIdx.x / G;
        const bool live = row < nrows;
        a.row = live ? row : -1;
        a.mu = live ? __ldg(p.mean + row) : 0.f;
        a.rs = live ? __ldg(p.rstd + row) : 0.f;
        rn.template load<G>(p, live, live ? row : 0, cols, gl);
        return a;
    };
    const int step = gridDim.x * ROWS;
    int base = blockIdx.x * ROWS;
    At an = fetch(base);
    stage_vec<T, V>(nsm, p.gain, W, 1.f);
    __syncthreads();
    for (; base < nrows; base += step) {
        if (!AHEAD && base != (int)blockIdx.x * ROWS) an = fetch(base);
        const NormRow<T, V, NV, CK> r = rn;
        const At a = an;
        if (AHEAD && base + step < nrows) an = fetch(base + step);
        T* dx = (T*)p.dx + norm_row(p, max(a.row, 0));
        ln_bwd_row<T, V, NV, G, CK>(p, r, a.mu, a.rs, gl, nsm, red, turn, dg, db, [&](int i, int c, const float2(&d)[NP]) {
            if (a.row < 0) return;
            Pack<T, V>::store(dx + cols.off[i], d);
            if (mixed && p.dres) Pack<T, V>::store((T*)p.dres + (size_t)a.row * W + c, d);
        });
    }
    if (p.part) ln_store_partials<V, NV, G>(p, nsm + W, ROWS, ROWS, threadIdx.x / G, gl, dg, db);
}

// Backward of LN(Mix(X) + X) (T = H, W = D) for samples that the ring of ln_sample_bwd_kernel does not take:
// dX = dz + Revert(dz), where an element of Revert(dz) comes from another row of the same sample.  A block
// works on one sample at a time: its warps turn the sample's rows into dz in shared memory (fp32), then all
// threads add the two parts and write dX.  Dynamic shared memory: gain, then H * W floats.
template <typename T, int V, int NV, bool CK, int THREADS>
__global__ void __launch_bounds__(THREADS) ln_bwd_self_kernel(const NormParams p) {
    extern __shared__ __align__(16) float nsm[];
    constexpr int NP = Pairs<V>::N;
    int turn = 0;
    const int W = p.map.W, H = p.map.banks, dh = p.map.dh;
    float* sm = nsm + W;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    stage_vec<T, V>(nsm, p.gain, W, 1.f);
    __syncthreads();
    const NormCols<V, NV, 32> cols(p.map, lane);
    float2 dg[NV][NP], db[NV][NP];
    zero_sums<V, NV>(dg, db);
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        for (int h = warp; h < H; h += THREADS / 32) {
            const int row = b * H + h;
            NormRow<T, V, NV, CK> r;
            const float mu = __ldg(p.mean + row), rs = __ldg(p.rstd + row);
            r.template load<32>(p, true, row, cols, lane);
            ln_bwd_row<T, V, NV, 32, CK>(p, r, mu, rs, lane, nsm, nullptr, turn, dg, db, [&](int, int c, const float2(&d)[NP]) {
#pragma unroll
                for (int k = 0; k < NP; k += 2)
                    *reinterpret_cast<float4*>(sm + (size_t)h * W + c + 2 * k) = make_float4(d[k].x, d[k].y, d[k + 1].x, d[k + 1].y);
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
            float2 o[NP];
#pragma unroll
            for (int k = 0; k < NP; ++k) o[k] = make_float2(a[2 * k] + r[2 * k], a[2 * k + 1] + r[2 * k + 1]);
            Pack<T, V>::store(out + e, o);
        }
        __syncthreads();
    }
    if (p.part) ln_store_partials<V, NV, 32>(p, sm, min(H, THREADS / 32), THREADS / 32, warp, lane, dg, db);
}

// ------------------------------------------------------------------ whole samples: LN(Mix(X) + X)
// With T = H and X as the residual too, everything a sample's rows read is the sample itself, one
// contiguous piece of memory.  Blocks bring samples into shared memory by bulk copies, a ring of NB
// slots ahead of the arithmetic, so that the scattered reads of the Mix view (pieces of dh columns, one
// per token) cost shared-memory cycles instead of L1 lookups, and loads stay in flight while rows are
// worked on.  A token row of a slot is `ld` bytes, padded so that ld = dh * esz modulo 128: the pieces
// of 8 lanes then fall into different banks.  A slot takes `per_slot` samples (the last of a tensor fewer):
// what a slot costs besides its rows -- waits, barriers, the latency of its first loads -- is paid once for all.
struct SampleGeo {
    uint32_t ld;               // bytes of a padded token row, and
    uint32_t ldc;              // of a padded row of the checkpoint's codes (the backward's)
    int nb;                    // slots (the forward's)
    int per_slot, nslots;      // samples a slot, and slots' worth of samples in the tensor
    FastDiv heads;             // rows a sample
};
struct SampleRing {
    uint8_t* base;             // slots
    uint64_t* full;            // one barrier each
    uint32_t slot_bytes;
    int nb;
};

// Token rows of a slot's samples (rows x bytes each, contiguous in memory), by one warp.
__device__ __forceinline__ void sample_load(const SampleRing& r, int slot, const void* src, int rows, uint32_t bytes,
                                            uint32_t ld) {
    uint64_t* bar = r.full + slot;
    const int lane = threadIdx.x & 31;
    if (lane == 0) mbar_arrive_expect_tx(bar, rows * bytes);
    __syncwarp();
    uint8_t* dst = r.base + slot * r.slot_bytes;
    for (int t = lane; t < rows; t += 32) bulk_load(dst + t * ld, (const uint8_t*)src + (size_t)t * bytes, bytes, bar);
}

// Waits for a phase by one lane of the warp; then every lane sees for itself that it is complete.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, unsigned where) {
    bool ok = true;
    if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, where);
    ok = __all_sync(0xffffffffu, ok);
    mbar_try_wait(bar, parity);
    return ok;
}

// Working warps of the sample kernels, beside the one that loads (issuing a sample's 48 row copies takes
// a warp some 4000 cycles): rows of up to 64 vectors leave room for several blocks an SM, whose loads,
// arithmetic and stores then overlap; wider rows come in samples that fill an SM.  300 MB of bf16 forward, 8 / 24
// warps: 32 x 512 101 / 145 us, 16 x 256 121 / 230, 32 x 768 125 / 122, 48 x 768 128 / 111.
constexpr int sample_warps(int nv) { return nv <= 2 ? 8 : 24; }

// Dynamic shared memory: nb slots, then gain and bias.
template <typename T, int V, int NV, int NW>
__global__ void __launch_bounds__(NW * 32 + 32, NV <= 2 ? 3 : 1)
    ln_sample_fwd_kernel(const NormParams p, const SampleGeo geo) {
    extern __shared__ __align__(128) uint8_t sms[];
    __shared__ uint64_t bars[8];               // [slot] loaded, [4 + slot] read by every warp
    constexpr int NP = Pairs<V>::N, ES = sizeof(T);
    const int W = p.map.W, H = p.map.banks, dh = p.map.dh;
    const uint32_t bytes = W * ES, ld = geo.ld;
    const int nb = geo.nb, all = geo.per_slot * H;
    const SampleRing ring{sms, bars, all * ld, nb};
    float* sg = reinterpret_cast<float*>(sms + (size_t)nb * ring.slot_bytes);
    float* sb = sg + W;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int turn = 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < nb; ++i) {
            mbar_init(&bars[i], 1);
            mbar_init(&bars[4 + i], NW);
        }
        fence_barrier_init();
    }
    __syncthreads();
    // group i of samples of this block is blockIdx.x + i * gridDim.x, in slot i % nb
    const int mine = blockIdx.x < geo.nslots ? (geo.nslots - 1 - blockIdx.x) / gridDim.x + 1 : 0;
    auto first_row = [&](int i) { return (blockIdx.x + i * (int)gridDim.x) * all; };
    auto rows_of = [&](int i) { return min(all, p.B * H - first_row(i)); };
    auto load = [&](int i, int slot) {
        const int r0 = first_row(i);
        sample_load(ring, slot, (const T*)p.x + (size_t)r0 * W, rows_of(i), bytes, ld);
    };
    if (warp == NW) {
        int slot = 0, i = 0;
        uint32_t ph = 0;
        for (; i < mine; ++i) {
            if (i >= nb && !warp_wait(&bars[4 + slot], ph ^ 1, 0x815)) break;
            load(i, slot);
            if (++slot == nb) { slot = 0; ph ^= 1; }
            if (i == 0) break;                 // the first on its way, then the vectors of all rows
        }
        stage_vec<T, V>(sg, p.gain, W, 1.f);
        stage_vec<T, V>(sb, p.bias, W, 0.f);
        __syncthreads();
        for (++i; i < mine; ++i) {
            if (i >= nb && !warp_wait(&bars[4 + slot], ph ^ 1, 0x815)) break;
            load(i, slot);
            if (++slot == nb) { slot = 0; ph ^= 1; }
        }
        if (i < mine)                          // given up: the loads in flight land before the block ends
            for (int k = 0; k < nb && k < i; ++k) {
                if (slot == 0) { slot = nb; ph ^= 1; }
                --slot;
                mbar_wait(&bars[slot], ph, 0x811);
            }
        return;
    }
    stage_vec<T, V>(sg, p.gain, W, 1.f);
    stage_vec<T, V>(sb, p.bias, W, 0.f);
    // byte offsets of the Mix view's pieces that this lane's vectors are
    int moff[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (lane + 32 * i) * V, t = c / dh;
        moff[i] = t * (int)ld + (c - t * dh) * ES;
    }
    __syncthreads();
    // warps go from sample to sample on their own
    int slot = 0;
    uint32_t ph = 0;
    for (int done = 0; done < mine; ++done) {
        if (!warp_wait(&bars[slot], ph, 0x810)) break;
        const uint8_t* sx = sms + slot * ring.slot_bytes;
        const int r0 = first_row(done), rows = rows_of(done);
        for (int r = warp; r < rows; r += NW) {
            const int s0 = geo.heads.div(r) * H;             // the sample's first row, head r - s0
            const uint8_t* mx = sx + s0 * ld + (r - s0) * dh * ES;
            float2 z[NV][NP];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (lane + 32 * i) * V;
                Pack<T, V> a, w;
                a.zero();
                w.zero();
                if (c < W) {
                    a.load_shared(mx + moff[i]);
                    w.load_shared(sx + r * ld + c * ES);
                }
                float2 rv[NP];
                a.get(z[i]);
                w.get(rv);
#pragma unroll
                for (int k = 0; k < NP; ++k) z[i][k] = add2(z[i][k], rv[k]);
            }
            ln_fwd_row<T, V, NV, 32>(p, z, true, r0 + r, lane, sg, sb, nullptr, turn);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[4 + slot]);
        if (++slot == nb) { slot = 0; ph ^= 1; }
    }
}

// Backward of the same, dX = dz + Revert(dz).  Mix(X) + X is symmetric under exchange of a token and a
// head (its element (row h, column t * dh + j) is X[t][h * dh + j] + X[h][t * dh + j]), and so is dX:
// dX[t][h * dh + j] = dz[t][h * dh + j] + dz[h][t * dh + j] = dX[h][t * dh + j].  First a sample's row
// means, with dgain and dbias on the way, a warp a row; then every pair of elements once: dz is never stored.  Three slots: X (or the
// checkpoint's codes) of this sample and of the next, and dy.  The second step reads dy again through the
// L2, where the first's copy has just come from, so that the next dy is on its way meanwhile: with dy kept
// in its slot to the end, two samples of 73 KB do not fit, and a third of the time went by waiting for the
// next one.  Every warp issues some of a sample's row copies (all of them take one warp some 4000 cycles).
// Bf16: 8192 x 32 x 512 205 us (3.9 TB/s), 4096 x 48 x 768 235; from the checkpoint 257 and 296.  Not the bus
// but a sample's two steps bound it, with a barrier after each and 16 warps an SM: the sums of dgain and dbias
// stay in 32 to 64 registers a thread, and more warps (20 or 24) spilled and took 310 to 400.  So the checkpoint, a
// sixth fewer bytes but its codes converted in both steps, saves memory here and costs time.  Fp32: 4096 x 32 x 512 152
// us, from the checkpoint 183; samples of 48 x 768 do not fit three slots and take ln_bwd_self_kernel, 2048 of them
// 432, and 250 from the checkpoint, without the scattered reads of x.
// Dynamic shared memory: 3 slots, gain, and per row of a slot its constants, statistics and sums.
template <typename T, int NV, bool CK, int NW>
__global__ void __launch_bounds__(NW * 32, NW <= 12 ? 2 : 1)
    ln_sample_bwd_kernel(const NormParams p, const SampleGeo geo) {
    extern __shared__ __align__(128) uint8_t sms[];
    __shared__ uint64_t bars[3];       // loaded: X slots 0 and 1, dy
    constexpr int V = sizeof(T) == 2 ? 8 : 4, NP = Pairs<V>::N, ES = sizeof(T);
    const int W = p.map.W, H = p.map.banks, dh = p.map.dh;
    const int nblk = (W + kCk8Block - 1) / kCk8Block;
    const uint32_t bytes = W * ES, ld = geo.ld, ldc = geo.ldc;
    constexpr bool MULTI = NV <= 2;    // wider rows: one sample a slot, which spares the registers of its walk
    const int all = MULTI ? geo.per_slot * H : H;
    const SampleRing ring{sms, bars, all * ld, 3};
    float* sg = reinterpret_cast<float*>(sms + (size_t)3 * ring.slot_bytes);
    float4* rowc = reinterpret_cast<float4*>(sg + W);      // {rs, mu, -rs m1, -rs^2 m2}
    float2* rowstat = reinterpret_cast<float2*>(rowc + all); // {mu, rs}
    float2* rowsum = rowstat + all;                          // sums of dn and dn n
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int turn = 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; ++i) mbar_init(&bars[i], 1);
        fence_barrier_init();
    }
    __syncthreads();
    const int mine = blockIdx.x < geo.nslots ? (geo.nslots - 1 - blockIdx.x) / gridDim.x + 1 : 0;
    auto first_row = [&](int i) { return (blockIdx.x + i * (int)gridDim.x) * all; };
    auto rows_of = [&](int i) { return MULTI ? min(all, p.B * H - first_row(i)) : all; };
    float2 dg[NV][NP], db[NV][NP];
    zero_sums<V, NV>(dg, db);
    // this block's i-th group of samples, row copies dealt out to the warps: X or codes into slot i % 2, dy into
    // slot 2
    auto load = [&](int i, int slot, const void* src, uint32_t row_bytes, uint32_t row_ld) {
        const int rows = rows_of(i);
        src = (const uint8_t*)src + (size_t)first_row(i) * row_bytes;
        if (threadIdx.x == 0) mbar_arrive_expect_tx(&bars[slot], rows * row_bytes);
        uint8_t* dst = sms + slot * ring.slot_bytes;
        for (int t = lane * NW + warp; t < rows; t += 32 * NW)
            bulk_load(dst + t * row_ld, (const uint8_t*)src + (size_t)t * row_bytes, row_bytes, &bars[slot]);
    };
    auto load_x = [&](int i) {
        if (CK) load(i, i & 1, p.codes, W, ldc);
        else load(i, i & 1, p.x, bytes, ld);
    };
    auto load_d = [&](int i) { load(i, 2, p.dy, bytes, ld); };
    if (mine > 0) {
        load_x(0);
        load_d(0);
    }
    stage_vec<T, V>(sg, p.gain, W, 1.f);
    int moff[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (lane + 32 * i) * V, t = c / dh;
        moff[i] = t * (int)ld + (c - t * dh) * ES;
    }
    // the second step's vectors: per sample (H + 1) / 2 folded rows of H + 1 pieces of vpd vectors; this
    // thread's first and the step to its next
    constexpr int TH = NW * 32;
    const int vpd = dh / V, folds = (H + 1) / 2, npair = folds * (H + 1) * vpd;
    // (vector of a piece, piece and folded row in 10 bits each, as registers are short here)
    auto walk = [&](int v) { return v % vpd | v / vpd % (H + 1) << 10 | v / vpd / (H + 1) % folds << 20; };
    const int jki0 = walk(threadIdx.x), djki = walk(TH);
    const int s0 = MULTI ? threadIdx.x / npair * H : 0, ds = MULTI ? TH / npair * H : 0;
    // thread r holds row r's statistics a group ahead (a slot has at most 256 rows, the smallest block's threads)
    float2 stat = make_float2(0.f, 0.f);
    auto fetch_stat = [&](int i) {
        const int r = first_row(i) + threadIdx.x;
        if (threadIdx.x < rows_of(i)) stat = make_float2(__ldg(p.mean + r), __ldg(p.rstd + r));
    };
    if (mine > 0) fetch_stat(0);
    __syncthreads();
    int done = 0;
    for (; done < mine; ++done) {
        const uint32_t phx = (done >> 1) & 1, phd = done & 1;
        // one warp waits for the data, the others at the barrier; it also says that every warp is done with
        // the last sample, its slot of X and its row constants
        const bool ok = warp != 0 || (warp_wait(&bars[done & 1], phx, 0x812) && warp_wait(&bars[2], phd, 0x813));
        if (threadIdx.x < all) rowstat[threadIdx.x] = stat;
        if (!__syncthreads_and(ok)) break;
        mbar_try_wait(&bars[done & 1], phx);           // complete: each thread sees it for itself
        mbar_try_wait(&bars[2], phd);
        if (done + 1 < mine) load_x(done + 1);
        const uint8_t* sx = sms + (done & 1) * ring.slot_bytes;
        const uint8_t* sd = sms + 2 * ring.slot_bytes;
        const int r0 = first_row(done), rows = rows_of(done);
        const int8_t* ex = CK ? p.exps + (size_t)r0 * nblk : nullptr;
        for (int r = warp; r < rows; r += NW) {
            const int sr = MULTI ? geo.heads.div(r) * H : 0; // the sample's first row, head r - sr
            const uint8_t* mx = sx + sr * ld + (r - sr) * dh * ES;
            const float2 st = rowstat[r];
            float2 s1 = make_float2(0.f, 0.f), s2 = s1;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (lane + 32 * i) * V;
                if (c < W) {
                    float2 n[NP], d[NP], g[NP];
                    Pack<T, V> w;
                    if constexpr (CK) {
                        uint32_t q[(V + 3) / 4];
                        ck8_load_shared<V>(sx + r * ldc + c, q);
                        ck8_values<V>(q, ck8_scale(__ldg(ex + r * nblk + c / kCk8Block)), n);
                    } else {
                        float2 x[NP];
                        w.load_shared(mx + moff[i]);
                        w.get(n);
                        w.load_shared(sx + r * ld + c * ES);
                        w.get(x);
#pragma unroll
                        for (int k = 0; k < NP; ++k) n[k] = add2(n[k], x[k]);
                    }
                    w.load_shared(sd + r * ld + c * ES);
                    w.get(d);
                    staged<V>(sg, W, c, g);
#pragma unroll
                    for (int k = 0; k < NP; ++k) {
                        n[k] = mul2(add2(n[k], f2(-st.x)), f2(st.y));
                        dg[i][k] = fma2(d[k], n[k], dg[i][k]);
                        db[i][k] = add2(db[i][k], d[k]);
                        const float2 dn = mul2(d[k], g[k]);
                        s1 = add2(s1, dn);
                        s2 = fma2(dn, n[k], s2);
                    }
                }
            }
            const float2 m = row_sum2<32>(make_float2(s1.x + s1.y, s2.x + s2.y), nullptr, turn);
            if (lane == 0) rowsum[r] = m;
        }
        if (done + 1 < mine) fetch_stat(done + 1);
        // the second step's pairs (t <= h): rows i and H-1-i of the triangle together are H + 1 pieces; the
        // first two vectors of dy are on their way before the barriers, then always the next two
        const int nvec = MULTI ? rows / H * npair : npair;
        T* out = (T*)p.dx + (size_t)r0 * W;
        const T* dyb = (const T*)p.dy + (size_t)r0 * W;
        // piece k of folded row i of the sample whose first row is s, vector j of it: advanced by TH with carries
        int jki = jki0, s = s0, left = nvec - threadIdx.x;
        struct Pair {
            uint32_t rows, cols;                // t | h << 16, rows of the slot, and their columns; none: cols = ~0
        };
        Pair q[2];
        Pack<T, V> wa[2], wb[2];
        auto fetch = [&](int at) {
            const int j = jki & 1023, k = jki >> 10 & 1023, i = jki >> 20;
            const bool low = k >= H - i;
            const int t = low ? H - 1 - i : i;
            const int h = low ? k - 1 : i + k;  // t + k - (H - i), or i + k
            Pair& c = q[at];
            if (left <= 0 || (low && t == i)) { // odd H: the middle row is its own partner
                c.cols = ~0u;
            } else {
                const int ct = h * dh + j * V, ch = t * dh + j * V;
                c.rows = (s + t) | (s + h) << 16;
                c.cols = ct | ch << 16;
                wa[at].load(dyb + ((s + t) * W + ct));
                wb[at].load(dyb + ((s + h) * W + ch));
            }
            left -= TH;
            jki += djki;
            if (MULTI) s += ds;
            if ((jki & 1023) >= vpd) jki += (1 << 10) - vpd;
            if ((jki >> 10 & 1023) > H) jki += (1 << 20) - ((H + 1) << 10);
            if (MULTI && (jki >> 20) >= folds) {
                jki -= folds << 20;
                s += H;
            }
        };
        fetch(0);
        fetch(1);
        __syncthreads();
        if (done + 1 < mine) load_d(done + 1);
        if (threadIdx.x < rows) {
            const float2 m = rowsum[threadIdx.x];
            const float2 st = rowstat[threadIdx.x];
            rowc[threadIdx.x] = make_float4(st.y, st.x, -st.y * (m.x * p.inv_w), -st.y * st.y * (m.y * p.inv_w));
        }
        __syncthreads();
        // z of the vector at column c of row r of the checkpoint
        auto codes = [&](int r, int c, float2(&v)[NP]) {
            uint32_t q[(V + 3) / 4];
            ck8_load_shared<V>(sx + r * ldc + c, q);
            ck8_values<V>(q, ck8_scale(__ldg(ex + r * nblk + c / kCk8Block)), v);
        };
        auto step = [&](int at) {
            const Pair c = q[at];
            float2 za[NP], zb[NP], da[NP], dd[NP], ga[NP], gb[NP];
            wa[at].get(da);
            wb[at].get(dd);
            fetch(at);
            if (c.cols == ~0u) return;
            const int rt = c.rows & 0xffff, rh = c.rows >> 16, ct = c.cols & 0xffff, ch = c.cols >> 16;
            if constexpr (CK) {
                codes(rt, ct, za);
                codes(rh, ch, zb);
            } else {
                Pack<T, V> w;
                w.load_shared(sx + rt * ld + ct * ES);
                w.get(za);
                w.load_shared(sx + rh * ld + ch * ES);
                w.get(zb);
#pragma unroll
                for (int e = 0; e < NP; ++e) za[e] = add2(za[e], zb[e]);
            }
            staged<V>(sg, W, ct, ga);
            staged<V>(sg, W, ch, gb);
            const float4 ra = rowc[rt], rb = rowc[rh];
            float2 o[NP];
            if constexpr (CK) {
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    const float2 a = fma2(add2(za[e], f2(-ra.y)), f2(ra.w), fma2(mul2(da[e], ga[e]), f2(ra.x), f2(ra.z)));
                    const float2 d = fma2(add2(zb[e], f2(-rb.y)), f2(rb.w), fma2(mul2(dd[e], gb[e]), f2(rb.x), f2(rb.z)));
                    o[e] = add2(a, d);
                }
            } else {
                // one z: its two factors together, row h's centre expressed from row t's
                const float2 wz = f2(ra.w + rb.w), cz = f2(ra.z + fmaf(ra.y - rb.y, rb.w, rb.z));
#pragma unroll
                for (int e = 0; e < NP; ++e)
                    o[e] = fma2(mul2(da[e], ga[e]), f2(ra.x),
                                fma2(mul2(dd[e], gb[e]), f2(rb.x), fma2(add2(za[e], f2(-ra.y)), wz, cz)));
            }
            Pack<T, V>::store(out + (rt * W + ct), o);
            if (rt != rh) Pack<T, V>::store(out + (rh * W + ch), o);
        };
        for (int v = threadIdx.x; v < nvec; v += 2 * TH) {
            step(0);
            if (v + TH < nvec) step(1);
        }
    }
    if (done < mine) {
        // given up, before anything of this group was started: the loads in flight are its own two
        if (threadIdx.x == 0) {
            mbar_wait(&bars[done & 1], (done >> 1) & 1, 0x814);
            mbar_wait(&bars[2], done & 1, 0x816);
        }
        return;
    }
    if (p.part) {                                // (its first barrier is behind every read of the slots)
        const int fit = (int)((size_t)3 * ring.slot_bytes / (W * sizeof(float)));
        ln_store_partials<V, NV, 32>(p, reinterpret_cast<float*>(sms), min(fit, NW), NW, warp, lane, dg, db);
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
// Rows of W columns in vectors of V: vectors per thread NV and threads per row G, the first that holds W.
#define TM_NORM_BF16(X) \
    X(8, 1, 8) X(8, 1, 16) X(8, 1, 32) X(8, 3, 16) X(8, 2, 32) X(8, 3, 32) X(8, 4, 32) X(8, 2, 128) X(8, 4, 128) X(8, 4, 512)
#define TM_NORM_F32(X) \
    X(4, 1, 8) X(4, 1, 16) X(4, 1, 32) X(4, 2, 32) X(4, 3, 32) X(4, 4, 32) X(4, 8, 32) X(4, 4, 128) X(4, 8, 128) X(4, 8, 512)
#define TM_NORM_ODD(X) X(1, 4, 32) X(1, 16, 32) X(1, 16, 128) X(1, 32, 512)

int norm_max_width() { return 16384; }

// rows that start on 16-byte boundaries
static bool norm_vec(int dtype, int W) { return W % (dtype == 1 ? 8 : 4) == 0; }

// Blocks per SM that a persistent grid may have at most (the backward's partial sums are sized by it).
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

// Grid of a persistent launch: one block per `rows_per_block` rows, at most as many as are resident and
// `most` per SM.
static long long norm_blocks(long long nrows, int rows_per_block, int per_sm, size_t smem, int sms, int most) {
    const long long by_smem = (long long)((227 * 1024) / (smem + 1024));
    if (per_sm > by_smem) per_sm = (int)(by_smem > 0 ? by_smem : 1);
    if (per_sm > most) per_sm = most;
    const long long want = (nrows + rows_per_block - 1) / rows_per_block;
    const long long cap = (long long)per_sm * sms;
    return want < cap ? want : cap;
}

template <typename T, int V, int NV, int G>
static cudaError_t launch_ln_fwd_one(const NormParams& p, int sms, cudaStream_t st) {
    constexpr int ROWS = NormBlock<G>::ROWS;
    const size_t smem = 2 * (size_t)p.map.W * sizeof(float);
    auto kern = ln_fwd_kernel<T, V, NV, G>;
    static std::atomic<int> cache[64];
    int per_sm = 0;
    cudaError_t e = norm_resident(kern, NormBlock<G>::THREADS, 2 * (size_t)V * NV * G * sizeof(float), cache, &per_sm);
    if (e != cudaSuccess) return e;
    const long long grid = norm_blocks((long long)p.B * p.map.banks, ROWS, per_sm, smem, sms, 16);
    kern<<<(unsigned)grid, NormBlock<G>::THREADS, smem, st>>>(p);
    return cudaGetLastError();
}

template <typename T>
static cudaError_t launch_ln_fwd_t(const NormParams& p, bool vec, int sms, cudaStream_t st) {
#define X(V_, NV_, G_) \
    if (p.map.W <= V_ * NV_ * G_) return launch_ln_fwd_one<T, V_, NV_, G_>(p, sms, st);
    if (vec) {
        if constexpr (sizeof(T) == 2) { TM_NORM_BF16(X) }
        else { TM_NORM_F32(X) }
    } else {
        TM_NORM_ODD(X)
    }
#undef X
    return cudaErrorInvalidValue;
}

template <typename T, int V, int NV, int G, bool CK>
static cudaError_t launch_ln_bwd_one(const NormParams& p, int sms, int* nblk, cudaStream_t st) {
    constexpr int ROWS = NormBlock<G>::ROWS;
    const size_t smem = (size_t)(1 + (p.part ? ROWS : 0)) * p.map.W * sizeof(float);
    auto kern = ln_bwd_kernel<T, V, NV, G, CK>;
    static std::atomic<int> cache[64];
    int per_sm = 0;
    cudaError_t e =
        norm_resident(kern, NormBlock<G>::THREADS, (size_t)(1 + ROWS) * V * NV * G * sizeof(float), cache, &per_sm);
    if (e != cudaSuccess) return e;
    const long long grid = norm_blocks((long long)p.B * p.map.banks, ROWS, per_sm, smem, sms, kNormBlocksPerSm);
    *nblk = (int)grid;
    kern<<<(unsigned)grid, NormBlock<G>::THREADS, smem, st>>>(p);
    return cudaGetLastError();
}

template <typename T, bool CK>
static cudaError_t launch_ln_bwd_t(const NormParams& p, bool vec, int sms, int* nblk, cudaStream_t st) {
#define X(V_, NV_, G_) \
    if (p.map.W <= V_ * NV_ * G_) return launch_ln_bwd_one<T, V_, NV_, G_, CK>(p, sms, nblk, st);
    if (vec) {
        if constexpr (sizeof(T) == 2) { TM_NORM_BF16(X) }
        else { TM_NORM_F32(X) }
    } else {
        TM_NORM_ODD(X)
    }
#undef X
    return cudaErrorInvalidValue;
}

// Kernels whose warps take a whole row of a sample: NV by W.
#define TM_NORM_WARP_ROWS(FN, T, V, W, ...)                      \
    if (W <= 32 * V) return FN<T, V, 1, ##__VA_ARGS__> TM_ARGS;  \
    if (W <= 64 * V) return FN<T, V, 2, ##__VA_ARGS__> TM_ARGS;  \
    if (W <= 96 * V) return FN<T, V, 3, ##__VA_ARGS__> TM_ARGS;  \
    if (W <= 128 * V) return FN<T, V, 4, ##__VA_ARGS__> TM_ARGS; \
    if constexpr (V == 4) return FN<T, V, 8, ##__VA_ARGS__> TM_ARGS;

constexpr int kSelfThreads = 512;
constexpr size_t kSelfSmem = 220 * 1024;     // of a sample in fp32; the gain comes on top
constexpr size_t kSampleSmem = 226 * 1024;
// The forward's samples of at least 8 KB (which makes rows of 181 or more values): smaller ones have narrow
// rows, of which the row kernel works on several a warp.  300 MB of bf16, sample / row kernel: 48 x 768 112 /
// 119 us, 16 x 512 102 / 107, 16 x 256 126 / 137, 8 x 256 126 / 131, 13 x 104 300 / 157, 8 x 128 240 / 134.
// (The backward's samples may be of any size: dX needs the sample's other rows, and the fallback that keeps dz
// in shared memory as fp32 takes 689 us for 48 x 768 and 904 for 8 x 128 where this one takes 234 and 376.)
constexpr size_t kSampleLeast = 8 * 1024;

// The sample of LN(Mix(X) + X)'s backward has to fit the shared memory as fp32, a row one warp.
bool ln_self_supported(int H, int W) { return (size_t)H * W * 4 <= kSelfSmem && W <= 1024; }

template <typename T, int V, int NV, bool CK>
static cudaError_t launch_ln_self(const NormParams& p, int sms, int* nblk, cudaStream_t st) {
    const size_t smem = (size_t)(p.map.banks + 1) * p.map.W * sizeof(float);
    auto kern = ln_bwd_self_kernel<T, V, NV, CK, kSelfThreads>;
    static std::atomic<int> cache[64];
    int per_sm = 0;
    cudaError_t e = norm_resident(kern, kSelfThreads, kSelfSmem + 4096, cache, &per_sm);
    if (e != cudaSuccess) return e;
    const long long grid = norm_blocks(p.B, 1, per_sm, smem, sms, kNormBlocksPerSm);
    *nblk = (int)grid;
    kern<<<(unsigned)grid, kSelfThreads, smem, st>>>(p);
    return cudaGetLastError();
}
template <typename T, bool CK>
static cudaError_t launch_ln_self_t(const NormParams& p, int sms, int* nblk, cudaStream_t st) {
    constexpr int V = sizeof(T) == 2 ? 8 : 4;
#define TM_ARGS (p, sms, nblk, st)
    TM_NORM_WARP_ROWS(launch_ln_self, T, V, p.map.W, CK)
#undef TM_ARGS
    return cudaErrorInvalidValue;
}

// ---- sample kernels (X the residual too)
// bytes of a padded token row of `bytes` (a multiple of 16, as the bulk copies into it need, whose every row
// starts at a multiple of this); piece: bytes of dh columns
static uint32_t sample_ld(uint32_t bytes, uint32_t piece) {
    piece = (piece + 15) & ~15u;
    return bytes + (piece % 128 + 128 - bytes % 128) % 128;
}
// Dynamic shared memory of each of `blocks` blocks on an SM: 228 KB less 1 KB a block for the system and 1 KB
// for the kernels' own static part.
static size_t sample_room(int blocks) { return blocks == 1 ? kSampleSmem : (228 * 1024) / blocks - 2048; }
static size_t sample_bwd_smem(int rows, int W, uint32_t ld) {
    return (size_t)3 * rows * ld + W * sizeof(float) + rows * (sizeof(float4) + 2 * sizeof(float2));
}
// Samples of a slot: as many as let two of the backward's blocks share an SM (some 32 KB; backward of 300 MB
// of bf16 in samples of 8 x 256: 476 us one by one, 260 in 16 KB, 229 in 32 KB), where there are enough for
// every block to take two slots; never more than 256 rows.
static int samples_per_slot(int B, int H, int W, uint32_t ld, int sms) {
    const size_t fixed = sample_bwd_smem(0, W, ld), each = sample_bwd_smem(H, W, ld) - fixed;
    size_t n = (sample_room(2) - fixed) / each;
    if (n > (size_t)256 / H) n = 256 / H;
    if (n > (size_t)B / (4 * sms)) n = B / (4 * sms);
    return n > 1 ? (int)n : 1;
}
// The kernels' geometry for H rows of W values of esz bytes a sample.
static SampleGeo sample_geo(int B, int H, int W, int dh, int esz, int sms) {
    const bool wide = W > 64 * (16 / esz);
    SampleGeo g;
    g.ld = sample_ld(W * esz, dh * esz);
    g.ldc = sample_ld(W, dh);
    g.nb = 0;
    g.per_slot = wide ? 1 : samples_per_slot(B, H, W, g.ld, sms);
    g.nslots = (B + g.per_slot - 1) / g.per_slot;
    g.heads = fast_div(H);
    return g;
}
// Slots of the forward's ring, 4 at most (0: none fits): as many blocks an SM, up to 3, as leave each two
// slots, so that loads run ahead.
static int sample_slots(size_t slot, size_t extra) {
    for (int blocks = 3; blocks >= 1; --blocks) {
        const size_t room = sample_room(blocks);
        if (room <= extra) continue;
        const int nb = (int)((room - extra) / slot);
        if (nb >= 2 || (blocks == 1 && nb >= 1)) return nb > 4 ? 4 : nb;
    }
    return 0;
}

template <typename T, int V, int NV>
static cudaError_t launch_sample_fwd(const NormParams& p, const SampleGeo& g, int sms, cudaStream_t st) {
    constexpr int NW = sample_warps(NV), THREADS = NW * 32 + 32;
    auto kern = ln_sample_fwd_kernel<T, V, NV, NW>;
    static std::atomic<int> cache[64];
    int per_sm = 0;
    cudaError_t e = norm_resident(kern, THREADS, kSampleSmem, cache, &per_sm);
    if (e != cudaSuccess) return e;
    const size_t smem = (size_t)g.nb * g.per_slot * p.map.banks * g.ld + 2 * p.map.W * sizeof(float);
    kern<<<(unsigned)norm_blocks(g.nslots, 1, per_sm, smem, sms, 16), THREADS, smem, st>>>(p, g);
    return cudaGetLastError();
}
template <typename T>
static cudaError_t launch_sample_fwd_t(const NormParams& p, const SampleGeo& g, int sms, cudaStream_t st) {
    constexpr int V = sizeof(T) == 2 ? 8 : 4;
#define TM_ARGS (p, g, sms, st)
    TM_NORM_WARP_ROWS(launch_sample_fwd, T, V, p.map.W)
#undef TM_ARGS
    return cudaErrorInvalidValue;
}

template <typename T, int NV, bool CK, int NW>
static cudaError_t launch_sample_bwd(const NormParams& p, const SampleGeo& g, int sms, int* nblk, cudaStream_t st) {
    constexpr int THREADS = NW * 32;
    auto kern = ln_sample_bwd_kernel<T, NV, CK, NW>;
    static std::atomic<int> cache[64];
    int per_sm = 0;
    cudaError_t e = norm_resident(kern, THREADS, kSampleSmem, cache, &per_sm);
    if (e != cudaSuccess) return e;
    const size_t smem = sample_bwd_smem(g.per_slot * p.map.banks, p.map.W, g.ld);
    const long long grid = norm_blocks(g.nslots, 1, per_sm, smem, sms, kNormBlocksPerSm);
    *nblk = (int)grid;
    kern<<<(unsigned)grid, THREADS, smem, st>>>(p, g);
    return cudaGetLastError();
}
template <typename T, bool CK>
static cudaError_t launch_sample_bwd_t(const NormParams& p, const SampleGeo& g, int sms, int* nblk, cudaStream_t st) {
    const int W = p.map.W;
    constexpr int V = sizeof(T) == 2 ? 8 : 4;
#define X(NV, NW) \
    if (W <= 32 * V * NV) return launch_sample_bwd<T, NV, CK, NW>(p, g, sms, nblk, st);
    X(1, 8) X(2, 8)
    if constexpr (V == 8) { X(3, 16) }
    X(4, 16)
    if constexpr (V == 4) { X(8, 16) }
#undef X
    return cudaErrorInvalidValue;
}

cudaError_t launch_ln_fwd(int dtype, const NormParams& p, int sms, cudaStream_t st) {
    ProfileScope ps_("layer_norm", st);
    const int esz = dtype == 1 ? 2 : 4;
    if (p.map.layout == 1 && p.res == p.x && p.map.T == p.map.banks && p.map.W <= 1024 &&
        (size_t)p.map.banks * p.map.W * esz >= kSampleLeast) {
        SampleGeo g = sample_geo(p.B, p.map.banks, p.map.W, p.map.dh, esz, sms);
        g.nb = sample_slots((size_t)g.per_slot * p.map.banks * g.ld, 2 * p.map.W * sizeof(float));
        if (g.nb) return dtype == 1 ? launch_sample_fwd_t<__nv_bfloat16>(p, g, sms, st)
                                    : launch_sample_fwd_t<float>(p, g, sms, st);
    }
    const bool vec = norm_vec(dtype, p.map.W);
    return dtype == 1 ? launch_ln_fwd_t<__nv_bfloat16>(p, vec, sms, st) : launch_ln_fwd_t<float>(p, vec, sms, st);
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
        const int esz = dtype == 1 ? 2 : 4;
        const bool vec = norm_vec(dtype, p.map.W);
        const SampleGeo g = sample_geo(p.B, p.map.banks, p.map.W, p.map.dh, esz, sms);
        const bool sample = self && p.map.banks <= 256 &&
                            (!ck || (p.map.W % 16 == 0 && g.ldc <= g.ld)) &&
                            sample_bwd_smem(g.per_slot * p.map.banks, p.map.W, g.ld) <= kSampleSmem;
#define X(FN, ...)                                                                                            \
    e = dtype == 1 ? (ck ? FN<__nv_bfloat16, true>(__VA_ARGS__) : FN<__nv_bfloat16, false>(__VA_ARGS__))      \
                   : (ck ? FN<float, true>(__VA_ARGS__) : FN<float, false>(__VA_ARGS__))
        if (sample) X(launch_sample_bwd_t, p, g, sms, &nblk, st);
        else if (self) X(launch_ln_self_t, p, sms, &nblk, st);
        else X(launch_ln_bwd_t, p, vec, sms, &nblk, st);
#undef X
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
