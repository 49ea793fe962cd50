// tm_linear.cuh -- the three contractions of the per-token linear layer on tcgen05 tensor cores:
//   forward   D[b, n] = sum_k x[b, k] W[n, k]     epilogue: + bias, activation, + residual, and the
//                                                 pre-activation saved whole or as an 8-bit checkpoint
//   dX        D[b, k] = sum_n dz[b, n] W[n, k]    epilogue: + dx_add
//   dW        D[n, k] = sum_b dz[b, n] x[b, k]    fp32 partial sums when the batch axis is split
// one problem per bank.  None of the operands is copied or transposed first: an operand whose
// contraction index is not the contiguous one (W in dX, both in dW) is loaded by TMA as it lies --
// boxes of 64 contiguous elements by 64 contraction rows -- and multiplied as an MN-major operand.
//
// Tile: 128 rows x BN columns, contraction in slabs of 64, 128-byte swizzle; edges in any direction
// are the tensor maps' business (loads past an extent give zeros, stores past it are dropped), so
// sizes need only be multiples of 8 (16-byte strides).  Persistent CTAs, one per SM: warp 0 issues the
// TMA loads, warp 1 the MMAs, warps 2-9 are the epilogue (two per TMEM lane quarter, each half of the
// columns).  Two accumulators in TMEM let the epilogue of a tile overlap the MMAs of the next.
//
// Epilogue: 32 columns at a time.  Eight warps share the activation: per 128 x 256 tile it costs one
// exponential per element (2048 cycles of the SM's 16 per cycle), which a contraction of 512 or more
// covers.  The output leaves through a 2 KB box per warp (32 rows x 64 bytes, 64-byte swizzle), two of
// them in turn so that a bulk store reads one while the other is filled.
#pragma once
#include "tm_ckpt8.cuh"
#include "tm_gemm.cuh"

namespace tml {

enum LinAct : int { LIN_NONE = 0, LIN_RELU = 1, LIN_GELU = 2, LIN_SILU = 3 };
// what the forward keeps of the pre-activation
enum LinSave : int { LIN_KEEP_NOTHING = 0, LIN_KEEP_FULL = 1, LIN_KEEP_CK8 = 2 };

struct LinParams {
    int groups;                // banks
    int rows, cols, depth;     // extents of D and of the contraction, per bank
    int mt, nt;                // tiles
    int splits, split_slabs;   // the contraction in `splits` runs of at most split_slabs slabs of 64
    const __nv_bfloat16* bias;   // [groups, cols] or NULL
    const __nv_bfloat16* add;    // residual / dx_add in D's layout or NULL
    size_t add_row, add_group;   // its strides: rows, groups
    int8_t* codes;             // LIN_KEEP_CK8: [rows * groups, cols]
    int8_t* exps;              //               [rows * groups, nblk]
    int nblk;
};

template <int BN, int SAVE>
struct LinCfg {
    static constexpr int BM = 128;
    static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int EPI_WARPS = 8;
    static constexpr int NTHREADS = 32 * (2 + EPI_WARPS);
    static constexpr int STG_BYTES = EPI_WARPS * 4096;
    static constexpr int STAGES = (232448 - 1024 - 256 - STG_BYTES) / STAGE_BYTES;
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + STG_BYTES + 1024 + 256;
    static constexpr int TMEM_COLS = 2 * BN;
    static_assert(SMEM_BYTES <= 232448 && STAGES >= 3 && (16 * STAGES + 48) <= 256, "shared memory budget");
    static_assert(TMEM_COLS == 256 || TMEM_COLS == 512, "tensor memory");
};

// MN-major operand, 128-byte swizzle: rows of 64 contiguous (M or N) elements, one row per contraction
// index; 8-row groups 1024 bytes apart, the next 64 elements of the M / N extent 64 rows (8192 bytes)
// on.  16 contraction rows (one MMA) are 2048 bytes.
__device__ __forceinline__ uint64_t umma_sdesc_mn128(uint32_t saddr) {
    uint64_t d = 0;
    d |= uint64_t((saddr >> 4) & 0x3FFFu);
    d |= uint64_t(8192u >> 4) << 16;       // leading byte offset: between 64-element blocks of M / N
    d |= uint64_t(1024u >> 4) << 32;       // stride byte offset: between groups of 8 contraction rows
    d |= uint64_t(1u) << 46;               // descriptor version for sm_100
    d |= uint64_t(2u) << 61;               // SWIZZLE_128B
    return d;
}
constexpr uint32_t kIdescAMn = 1u << 15, kIdescBMn = 1u << 16;

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float ex2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Upper tail of the normal distribution, Q(a) = erfc(a / sqrt 2) / 2, a >= 0, for results that are
// rounded to bf16: log2 Q is nearly a parabola, so a polynomial of degree 5 (fitted to log2 Q on
// [0, 6] by weighted least squares towards the smallest maximum) and one exponential give Q to a
// relative 3.7e-4, a fifth of bf16's half step; past 6, where Q < 1e-9, it falls on monotonically.
__device__ __forceinline__ float2 gauss_tail2(float2 a) {
    float2 p = make_float2(-2.01684350e-4f, -2.01684350e-4f);
    p = __ffma2_rn(p, a, make_float2(4.46760561e-3f, 4.46760561e-3f));
    p = __ffma2_rn(p, a, make_float2(-4.28327359e-2f, -4.28327359e-2f));
    p = __ffma2_rn(p, a, make_float2(-4.72785681e-1f, -4.72785681e-1f));
    p = __ffma2_rn(p, a, make_float2(-1.14439976f, -1.14439976f));
    p = __ffma2_rn(p, a, make_float2(-1.00053179f, -1.00053179f));
    return make_float2(ex2_approx(p.x), ex2_approx(p.y));
}

// Two activations.  gelu(z) = z Phi(z) = max(z, 0) - |z| Q(|z|): both terms keep their relative
// precision in the negative tail.  silu(z) = z / (1 + e^-z), one reciprocal for two (of the product of
// the denominators; z is held above -44 inside the exponential, where silu is below 1e-17, so that the
// product stays finite).  NaN comes out as NaN, +inf as +inf, -inf as 0 (relu, gelu) or -0 or NaN (silu).
template <int ACT>
__device__ __forceinline__ float2 lin_act2(float2 z) {
    if constexpr (ACT == LIN_RELU) return make_float2(max_nan(z.x, 0.f), max_nan(z.y, 0.f));
    if constexpr (ACT == LIN_GELU) {
        const float2 a = make_float2(fminf(fabsf(z.x), 16.f), fminf(fabsf(z.y), 16.f));
        const float2 q = gauss_tail2(a);
        return make_float2(fmaf(-a.x, q.x, max_nan(z.x, 0.f)), fmaf(-a.y, q.y, max_nan(z.y, 0.f)));
    }
    if constexpr (ACT == LIN_SILU) {
        const float kL = -1.4426950408889634f;   // -log2(e)
        const float d0 = 1.f + ex2_approx(kL * fmaxf(z.x, -44.f)), d1 = 1.f + ex2_approx(kL * fmaxf(z.y, -44.f));
        const float r = rcp_approx(d0 * d1);
        return make_float2(z.x * (r * d1), z.y * (r * d0));
    }
    return z;
}

template <int BN, bool A_MN, bool B_MN, int ACT, int SAVE, bool F32OUT>
__global__ void __launch_bounds__(LinCfg<BN, SAVE>::NTHREADS, 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmZ,
                       const LinParams p) {
    using C = LinCfg<BN, SAVE>;
    constexpr int STAGES = C::STAGES;
    const int ntile = p.groups * p.splits * p.mt * p.nt;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * C::STAGE_BYTES + C::STG_BYTES);
    uint64_t* empty = full + STAGES;
    uint64_t* acc_full = empty + STAGES;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_empty + 2;
    uint32_t* tmem_base_smem = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_smem + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    struct Tile {
        int g, s, m, n, slabs;
    };
    const int slabs_all = (p.depth + 63) / 64;
    // columns innermost, then row blocks: CTAs side by side share a row block's A tile and the bank's B
    auto decode = [&](int t) -> Tile {
        Tile r;
        r.n = t % p.nt;
        t /= p.nt;
        r.m = t % p.mt;
        t /= p.mt;
        r.s = t % p.splits;
        r.g = t / p.splits;
        r.slabs = min(p.split_slabs, slabs_all - r.s * p.split_slabs);
        return r;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], C::EPI_WARPS);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_base_smem, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_base_smem;

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        if (lane == 0) {
            tma_prefetch_desc(&tmA);
            tma_prefetch_desc(&tmB);
            int s = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < ntile && ok; t += gridDim.x) {
                const Tile ti = decode(t);
                for (int kb = 0; kb < ti.slabs; ++kb) {
                    if (!wait_or_abort(&empty[s], ph ^ 1, abort_flag, 0x800)) { ok = false; break; }
                    uint8_t* sa = smem + s * C::STAGE_BYTES;
                    uint8_t* sb = sa + C::A_BYTES;
                    const int k0 = (ti.s * p.split_slabs + kb) * 64;
                    mbar_arrive_expect_tx(&full[s], C::STAGE_BYTES);
                    if constexpr (A_MN) {        // [depth rows][bank][rows of D]: two blocks of 64
                        tma_load_3d(sa, &tmA, &full[s], ti.m * 128, ti.g, k0);
                        tma_load_3d(sa + 8192, &tmA, &full[s], ti.m * 128 + 64, ti.g, k0);
                    } else {                     // [rows of D][bank][depth]
                        tma_load_3d(sa, &tmA, &full[s], k0, ti.g, ti.m * 128);
                    }
                    if constexpr (B_MN) {
#pragma unroll
                        for (int i = 0; i < BN / 64; ++i) {
                            if constexpr (A_MN)  // x: [depth rows][bank][columns of D]
                                tma_load_3d(sb + i * 8192, &tmB, &full[s], ti.n * BN + i * 64, ti.g, k0);
                            else                 // W: [bank][depth rows][columns of D]
                                tma_load_3d(sb + i * 8192, &tmB, &full[s], ti.n * BN + i * 64, k0, ti.g);
                        }
                    } else {                     // W: [bank][columns of D][depth]
                        tma_load_3d(sb, &tmB, &full[s], k0, ti.n * BN, ti.g);
                    }
                    if (issued < STAGES) ++issued;
                    if (++s == STAGES) { s = 0; ph ^= 1; }
                }
            }
            // given up: the loads in flight land (a bounded wait each) before the block may end
            if (!ok || *abort_flag) {
                for (int i = 0; i < issued; ++i) {
                    if (s == 0) { s = STAGES; ph ^= 1; }
                    --s;
                    mbar_wait(&full[s], ph, 0x804);
                }
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (lane == 0) {
            constexpr uint32_t idesc = umma_idesc_bf16(128, BN) | (A_MN ? kIdescAMn : 0u) | (B_MN ? kIdescBMn : 0u);
            int s = 0, lt = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < ntile && ok; t += gridDim.x, ++lt) {
                const Tile ti = decode(t);
                const int buf = lt & 1;
                if (!wait_or_abort(&acc_empty[buf], ((lt >> 1) & 1) ^ 1, abort_flag, 0x801)) break;
                tc_fence_after();
                const uint32_t d = tmem_base + buf * BN;
                for (int kb = 0; kb < ti.slabs; ++kb) {
                    if (!wait_or_abort(&full[s], ph, abort_flag, 0x802)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sa = smem_u32(smem + s * C::STAGE_BYTES);
                    const uint32_t sb = sa + C::A_BYTES;
                    const uint64_t ad = A_MN ? umma_sdesc_mn128(sa) : umma_sdesc_sw128(sa);
                    const uint64_t bd = B_MN ? umma_sdesc_mn128(sb) : umma_sdesc_sw128(sb);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16(d, ad + (A_MN ? 128 : 2) * kk, bd + (B_MN ? 128 : 2) * kk, idesc, (kb | kk) != 0);
                    umma_commit(&empty[s]);
                    if (++s == STAGES) { s = 0; ph ^= 1; }
                }
                if (!ok) break;
                umma_commit(&acc_full[buf]);
            }
            // every MMA issued is complete before the tensor memory is released
            umma_commit(drain);
            mbar_wait(drain, 0, 0x805);
        }
    } else {
        // ---------------------------------------------------------------- epilogue
        const int q = warp & 3, half = (warp - 2) >> 2;
        constexpr int HC = BN / 2;                      // columns of this warp
        uint8_t* stg = smem + STAGES * C::STAGE_BYTES + (warp - 2) * 4096;
        int box = 0;                                    // the staging box in turn
        // lane's row of 32 columns into the free box (64-byte rows, 16-byte piece c at c ^ (row / 2 % 4)),
        // once the bulk store before the last one has read it
        auto stage = [&](const uint32_t(&pk)[16]) -> uint8_t* {
            uint8_t* bx = stg + box * 2048;
            box ^= 1;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                *reinterpret_cast<uint4*>(bx + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) =
                    make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            return bx;
        };
        auto free_box = [&]() {
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            __syncwarp();
        };
        int lt = 0;
        for (int t = blockIdx.x; t < ntile; t += gridDim.x, ++lt) {
            const Tile ti = decode(t);
            const int buf = lt & 1;
            const int row0 = ti.m * 128 + q * 32, row = row0 + lane;
            const int col0 = ti.n * BN + half * HC;
            const bool row_in = row < p.rows;
            // the addend of 32 columns, as it lies: 4 lanes a row, 8 rows an instruction; loaded a step ahead
            uint4 ad[4];
            auto load_add = [&](int c) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = row0 + 8 * i + (lane >> 2), cc = c + (lane & 3) * 8;
                    ad[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (r < p.rows && cc < p.cols)
                        ad[i] = __ldg(reinterpret_cast<const uint4*>(p.add + r * p.add_row + ti.g * p.add_group + cc));
                }
            };
            if (!F32OUT && p.add) load_add(col0);
            if (!wait_or_abort(&acc_full[buf], (lt >> 1) & 1, abort_flag, 0x803)) break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + (uint32_t(q * 32) << 16) + buf * BN + half * HC;
            // a box of 32 columns; those past the extents are not computed (uniform across the warp)
            const int ncol = row0 < p.rows ? min(HC, p.cols - col0) : 0;
            uint32_t ew = 0u;                           // exponents of up to four blocks of the row
#pragma unroll 1
            for (int c = 0; c < ncol; c += 32) {
                float v[32];
                tmem_ld32(taddr + c, v);
                const int col = col0 + c;
                if constexpr (F32OUT) {
                    // fp32 partial sums: 32 rows x 128 bytes, 128-byte swizzle, the warp's whole 4 KB
                    if (lane == 0) bulk_wait_read_all();
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<float4*>(stg + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                            make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&tmO, stg, col, row0, ti.s * p.groups + ti.g);
                        bulk_commit_group();
                    }
                } else {
                    if (p.bias) {
                        const __nv_bfloat16* bp = p.bias + (size_t)ti.g * p.cols + col;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (col + 8 * i < p.cols) {
                                const uint4 w = __ldg(reinterpret_cast<const uint4*>(bp + 8 * i));
                                const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    v[8 * i + 2 * k] += bf16_lo(a[k]);
                                    v[8 * i + 2 * k + 1] += bf16_hi(a[k]);
                                }
                            }
                        }
                    }
                    if constexpr (SAVE == LIN_KEEP_CK8) {
                        // this lane's 32 columns are one block of its row (those past the row are zero:
                        // their weights and bias were read as zero)
                        uint32_t qw[8];
                        const int e = ck8_quantize<32, 1>(v, qw);
                        ew |= (uint32_t)(e & 0xFF) << ((c & 96) >> 2);
                        if (row_in) {
                            int8_t* cp = p.codes + ((size_t)row * p.groups + ti.g) * p.cols + col;
                            if (col + 32 <= p.cols && (p.cols & 15) == 0) {
                                *reinterpret_cast<uint4*>(cp) = make_uint4(qw[0], qw[1], qw[2], qw[3]);
                                *reinterpret_cast<uint4*>(cp + 16) = make_uint4(qw[4], qw[5], qw[6], qw[7]);
                            } else {
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (col + 8 * i < p.cols)
                                        *reinterpret_cast<uint2*>(cp + 8 * i) = make_uint2(qw[2 * i], qw[2 * i + 1]);
                            }
                            // the exponents of four blocks together where they make an aligned word
                            int8_t* ep = p.exps + ((size_t)row * p.groups + ti.g) * p.nblk + (col >> 5);
                            if ((p.nblk & 3) == 0) {
                                if ((c & 96) == 96 || c + 32 >= ncol) {
                                    if ((c & 96) == 96) *reinterpret_cast<uint32_t*>(ep - 3) = ew;
                                    else
                                        for (int i = 0; i <= (c & 96) >> 5; ++i)
                                            ep[i - ((c & 96) >> 5)] = (int8_t)(ew >> (8 * i));
                                    ew = 0u;
                                }
                            } else {
                                *ep = (int8_t)e;
                            }
                        }
                    }
                    uint32_t pk[16];
                    if constexpr (SAVE == LIN_KEEP_FULL) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) pk[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
                        free_box();
                        const uint8_t* bx = stage(pk);
                        if (lane == 0) {
                            tma_store_3d(&tmZ, bx, col, ti.g, row0);
                            bulk_commit_group();
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 o = lin_act2<ACT>(make_float2(v[2 * i], v[2 * i + 1]));
                        v[2 * i] = o.x;
                        v[2 * i + 1] = o.y;
                    }
                    free_box();
                    if (p.add) {
                        // through the free box to the lane that owns the row
                        uint8_t* bx = stg + box * 2048;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = 8 * i + (lane >> 2), cc = lane & 3;
                            *reinterpret_cast<uint4*>(bx + r * 64 + ((cc ^ ((r >> 1) & 3)) << 4)) = ad[i];
                        }
                        __syncwarp();
                        if (c + 32 < ncol) load_add(col + 32);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint4 w = *reinterpret_cast<const uint4*>(bx + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4));
                            const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                v[8 * i + 2 * k] += bf16_lo(a[k]);
                                v[8 * i + 2 * k + 1] += bf16_hi(a[k]);
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) pk[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
                    const uint8_t* bx = stage(pk);
                    if (lane == 0) {
                        if constexpr (A_MN) tma_store_3d(&tmO, bx, col, row0, ti.g);   // dW: [bank][rows][columns]
                        else tma_store_3d(&tmO, bx, col, ti.g, row0);                   // [rows][bank][columns]
                        bulk_commit_group();
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[buf]);
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

}  // namespace tml
