// tm_linear.cuh -- the three contractions of the per-token linear layer on tcgen05 tensor cores:
//   forward   D[b, n] = sum_k x[b, k] W[n, k]     epilogue: + bias, activation, + residual, and the
//                                                 pre-activation saved whole or as an 8-bit checkpoint
//   dX        D[b, k] = sum_n dz[b, n] W[n, k]    epilogue: + dx_add
//   dW        D[n, k] = sum_b dz[b, n] x[b, k]    fp32 partial sums when the batch axis is split
// one problem per bank.  None of the operands is copied or transposed first: an operand whose
// contraction index is not the contiguous one (W in dX, both in dW) is loaded by TMA as it lies --
// boxes of 64 contiguous elements by 64 contraction rows -- and multiplied as an MN-major operand.
//
// Tile: 128 rows x BN columns, contraction in slabs of 64, 128-byte swizzle; edges in any direction are
// zeros from the tensor maps (loads past an extent) and predicates (stores), so sizes need only be
// multiples of 8 (16-byte strides).  Persistent CTAs, one per SM: warp 0 issues the TMA loads, warp 1
// the MMAs, the others (16 for 256 columns, 8 for 128) are the epilogue, 32 rows x 64 columns each.  Two
// accumulators in TMEM let the epilogue of a tile overlap the MMAs of the next.
//
// Pair mode (PAIR): a cluster of two CTAs on 256 rows, each holding its 128 A rows and half of the B
// rows, one tcgen05.mma.cta_group::2 for both.  A tile's operands are then 32 KB a slab and SM instead
// of the 48 of a single CTA's 128 x 256, which was bound by what the L2 delivers to the SMs (87 us against
// 73 for 8 banks of 4096 x 768 -> 1536).  Shapes with few rows, columns or tiles take 128 x 128 tiles.
//
// Epilogue: 32 columns at a time from TMEM, the box out by a bulk store.  Per 128 x 256 tile the activation
// costs one exponential per element (2048 cycles of the SM's 16 per cycle), which a contraction of depth 256
// (2048 tensor cycles) just covers; 8 epilogue warps did not keep up with it, 16 do.
//
// Measured, calls back to back: 48 banks of 8192 x 768 -> 1536, gelu 755 to 800 us as the power cap allows, 1160 to
// 1230 TFLOP/s (0.70 to 0.74 of the cuBLAS rate measured on this kind of GPU for one square bf16 product), with z kept
// 985 to 1030, with its checkpoint 995 to 1100; silu 760 to 780.  8 banks of 4096 x 768 -> 1536: gelu 72 us (1080
// TFLOP/s), silu 67, z kept or its checkpoint 84, dX 65, dW 59 (1320).  16 banks of 4096 x 256 -> 1024: gelu 48 us with the
// operands in the L2 and 47 without, where 27 would move the bytes: a tile is 4 slabs, and its 16 warps' epilogue as long
// as its loads; silu, with a second special function a value, 49, z kept 72, its checkpoint 77.
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
    FastDiv mt, nt, splits;    // tiles: rows (of 128, pair mode 256) and columns; runs of the contraction
    int ntile;                 // groups * splits * mt * nt
    int split_slabs;           // slabs of 64 of a run, at most
    const __nv_bfloat16* bias;   // [groups, cols] or NULL
    int add;                   // residual / dx_add in D's layout (its map: tmR), and
    const __nv_bfloat16* res;  // its address
    __nv_bfloat16* z;          // LIN_KEEP_FULL: [rows * groups, cols]
    int8_t* codes;             // LIN_KEEP_CK8: [rows * groups, cols], and
    int8_t* exps;              //               [rows * groups, nblk]
    int nblk;
};

template <int BN, bool PAIR>
struct LinCfg {
    static constexpr int BM = 128;                  // rows of D per CTA (a pair: 256)
    static constexpr int BC = PAIR ? BN / 2 : BN;   // B rows that this CTA loads
    static constexpr int A_BYTES = BM * 128, B_BYTES = BC * 128;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int EPI_WARPS = BN / 16;       // 4 lane quarters x BN / 64 column blocks
    static constexpr int NTHREADS = 32 * (2 + EPI_WARPS);
    // an epilogue warp's box: 32 rows x 64 bf16 of D
    static constexpr int BOX_BYTES = 4096;
    static constexpr int STG_BYTES = EPI_WARPS * BOX_BYTES;
    static constexpr int BIAS_BYTES = 2 * BN * 4;   // the tile's bias in fp32, tiles in turn
    static constexpr int BAR_BYTES = 320;
    static constexpr int STAGES_ = (232448 - BAR_BYTES - STG_BYTES - BIAS_BYTES) / STAGE_BYTES;
    static constexpr int STAGES = STAGES_ > 6 ? 6 : STAGES_;
    static constexpr int OFF_STG = STAGES * STAGE_BYTES, OFF_BIAS = OFF_STG + STG_BYTES, OFF_BAR = OFF_BIAS + BIAS_BYTES;
    static constexpr int SMEM_BYTES = OFF_BAR + BAR_BYTES;
    static constexpr int TMEM_COLS = 2 * BN;
    static_assert(SMEM_BYTES <= 232448 && STAGES >= 3 && 16 * STAGES + 48 + 8 * EPI_WARPS <= BAR_BYTES, "shared memory budget");
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

// Arrive on the leader's accumulator-free barrier.  Nothing in memory is handed over with it -- the
// tensor-memory loads are complete and fenced -- so release at CTA scope does; at cluster scope it waited
// 2000 to 4000 cycles a tile for the thread's outstanding global writes.
__device__ __forceinline__ void arrive_remote(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

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
// relative 3.7e-4, a tenth of bf16's half step.  Past 6, where Q < 1e-9, it falls on monotonically and too fast: 0.5 %
// short at 6.5, 2 % at 7, 9 % at 8, nearly all from 12 on.  (A polynomial of degree 7 holds 2.5e-3 as far as Q is a normal
// number, for two multiply-adds a pair that the epilogue of a short contraction shows: 56 -> 59 us for 16 banks of
// 4096 x 256 -> 1024.)
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
// precision in the negative tail.  silu(z) = z / (1 + e^-z), a reciprocal a value: where e^-z is
// infinite, or its reciprocal no normal number (z < -87, silu below 2^-119), silu is -0.  NaN comes out as NaN, +inf as
// +inf, -inf as -0 or 0 (relu, gelu) or NaN (silu: inf / inf).
template <int ACT>
__device__ __forceinline__ float2 lin_act2(float2 z) {
    if constexpr (ACT == LIN_RELU) return make_float2(max_nan(z.x, 0.f), max_nan(z.y, 0.f));
    if constexpr (ACT == LIN_GELU) {
        const float2 a = make_float2(fminf(fabsf(z.x), 16.f), fminf(fabsf(z.y), 16.f));
        const float2 q = gauss_tail2(a);
        return make_float2(fmaf(-a.x, q.x, max_nan(z.x, 0.f)), fmaf(-a.y, q.y, max_nan(z.y, 0.f)));
    }
    if constexpr (ACT == LIN_SILU) {
        const float2 x = mul2(z, f2(-1.4426950408889634f));       // -z log2(e)
        const float2 d = add2(make_float2(ex2_approx(x.x), ex2_approx(x.y)), f2(1.f));
        return mul2(z, make_float2(rcp_approx(d.x), rcp_approx(d.y)));
    }
    return z;
}

// D's rows are matrix rows, [bank][rows][cols], when A is MN-major (dW), else samples, [rows][bank][cols].
// Maps: tmO D (or the fp32 partial sums), tmR the addend, in boxes of 32 rows.
template <int BN, bool PAIR, bool A_MN, bool B_MN, int ACT, int SAVE, bool F32OUT>
__global__ void __launch_bounds__(LinCfg<BN, PAIR>::NTHREADS, 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmR,
                       const LinParams p) {
    using C = LinCfg<BN, PAIR>;
    constexpr int STAGES = C::STAGES;
    constexpr bool OUT_MAT = A_MN;
    const int rank = PAIR ? (int)cluster_ctarank() : 0;
    const bool leader = rank == 0;
    const int cid = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
    const int ncid = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;
    extern __shared__ __align__(1024) uint8_t lin_smem[];
    uint8_t* smem = lin_smem;
    if (smem_u32(smem) & 1023u) {            // the swizzled tiles need it; never so (checked, not assumed)
        if (threadIdx.x == 0) record_error(ERR_BOUNDS, 0x806);
        return;                              // the same in both CTAs of a pair
    }
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* empty = full + STAGES;
    uint64_t* acc_full = empty + STAGES;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_empty + 2;
    uint64_t* add_full = drain + 1;          // [EPI_WARPS] the addend of a warp's box has landed
    uint32_t* tmem_base_smem = reinterpret_cast<uint32_t*>(add_full + C::EPI_WARPS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_smem + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    struct Tile {
        int g, s, m, n, slabs;
    };
    const int slabs_all = (p.depth + 63) / 64;
    // columns innermost, then row blocks: CTAs side by side share a row block's A tile and the bank's B
    auto decode = [&](int t) -> Tile {
        Tile r;
        int u = p.nt.div(t);
        r.n = t - u * p.nt.d;
        t = u;
        u = p.mt.div(t);
        r.m = t - u * p.mt.d;
        r.g = p.splits.div(u);
        r.s = u - r.g * p.splits.d;
        r.slabs = min(p.split_slabs, slabs_all - r.s * p.split_slabs);
        if (PAIR) r.m = 2 * r.m + rank;      // this CTA's 128 rows (past the extent: loaded as zeros, not stored)
        return r;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], C::EPI_WARPS * (PAIR ? 2 : 1));
        }
        mbar_init(drain, 1);
        for (int w = 0; w < C::EPI_WARPS; ++w) mbar_init(&add_full[w], 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        if (PAIR) {
            tmem_alloc_pair(tmem_base_smem, C::TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_base_smem, C::TMEM_COLS);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    if (PAIR) cluster_sync_all();            // both CTAs' barriers exist before any remote use
    else __syncthreads();
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
            for (int t = cid; t < p.ntile && ok; t += ncid) {
                const Tile ti = decode(t);
                // pair mode: each CTA loads half of the tile's B rows
                const int n0 = ti.n * BN + (PAIR ? rank * C::BC : 0);
                for (int kb = 0; kb < ti.slabs; ++kb) {
                    if (!wait_or_abort(&empty[s], ph ^ 1, abort_flag, 0x800)) { ok = false; break; }
                    uint8_t* sa = smem + s * C::STAGE_BYTES;
                    uint8_t* sb = sa + C::A_BYTES;
                    const int k0 = (ti.s * p.split_slabs + kb) * 64;
                    if (leader) mbar_arrive_expect_tx(&full[s], (PAIR ? 2 : 1) * C::STAGE_BYTES);
                    const uint32_t lbar = PAIR ? mapa_shared(smem_u32(&full[s]), 0) : 0u;   // the leader's barrier
                    auto ld3 = [&](void* dst, const CUtensorMap* m, int c0, int c1, int c2) {
                        if (PAIR) tma_load_3d_pair(dst, m, lbar, c0, c1, c2);
                        else tma_load_3d(dst, m, &full[s], c0, c1, c2);
                    };
                    if constexpr (A_MN) {        // [depth rows][bank][rows of D]: two blocks of 64
                        ld3(sa, &tmA, ti.m * 128, ti.g, k0);
                        ld3(sa + 8192, &tmA, ti.m * 128 + 64, ti.g, k0);
                    } else {                     // [rows of D][bank][depth]
                        ld3(sa, &tmA, k0, ti.g, ti.m * 128);
                    }
                    if constexpr (B_MN) {
#pragma unroll
                        for (int i = 0; i < C::BC / 64; ++i) {
                            if constexpr (A_MN)  // x: [depth rows][bank][columns of D]
                                ld3(sb + i * 8192, &tmB, n0 + i * 64, ti.g, k0);
                            else                 // W: [bank][depth rows][columns of D]
                                ld3(sb + i * 8192, &tmB, n0 + i * 64, k0, ti.g);
                        }
                    } else {                     // W: [bank][columns of D][depth]
                        ld3(sb, &tmB, k0, n0, ti.g);
                    }
                    if (issued < STAGES) ++issued;
                    if (++s == STAGES) { s = 0; ph ^= 1; }
                }
            }
            if (!ok || *abort_flag) {
                // given up: the loads in flight land before the block may end -- a bounded wait for each,
                // or in a pair, whose loads the leader's barriers count, a millisecond
                if (PAIR) {
                    for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < 1000000;) {}
                } else {
                    for (int i = 0; i < issued; ++i) {
                        if (s == 0) { s = STAGES; ph ^= 1; }
                        --s;
                        mbar_wait(&full[s], ph, 0x804);
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer (pair: the leader's)
        if (lane == 0 && leader) {
            constexpr uint32_t idesc =
                umma_idesc_bf16(PAIR ? 256 : 128, BN) | (A_MN ? kIdescAMn : 0u) | (B_MN ? kIdescBMn : 0u);
            auto commit = [&](uint64_t* b) {
                if (PAIR) umma_commit_both(b);
                else umma_commit(b);
            };
            const uint32_t sbase = smem_u32(smem);
            int s = 0, lt = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = cid; t < p.ntile && ok; t += ncid, ++lt) {
                const int slabs = decode(t).slabs;
                const int buf = lt & 1;
                // the peer's warps arrive here too
                if (!(PAIR ? wait_or_abort_cl(&acc_empty[buf], ((lt >> 1) & 1) ^ 1, abort_flag, 0x801)
                           : wait_or_abort(&acc_empty[buf], ((lt >> 1) & 1) ^ 1, abort_flag, 0x801)))
                    break;
                tc_fence_after();
                const uint32_t d = tmem_base + buf * BN;
                for (int kb = 0; kb < slabs; ++kb) {
                    if (!wait_or_abort(&full[s], ph, abort_flag, 0x802)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sa = sbase + s * C::STAGE_BYTES, sb = sa + C::A_BYTES;
                    const uint64_t ad = A_MN ? umma_sdesc_mn128(sa) : umma_sdesc_sw128(sa);
                    const uint64_t bd = B_MN ? umma_sdesc_mn128(sb) : umma_sdesc_sw128(sb);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint64_t ak = ad + (A_MN ? 128 : 2) * kk, bk = bd + (B_MN ? 128 : 2) * kk;
                        if (PAIR) umma_bf16_pair(d, ak, bk, idesc, (kb | kk) != 0);
                        else umma_bf16(d, ak, bk, idesc, (kb | kk) != 0);
                    }
                    commit(&empty[s]);
                    if (++s == STAGES) { s = 0; ph ^= 1; }
                }
                if (!ok) break;
                commit(&acc_full[buf]);
            }
            // every MMA issued is complete before the tensor memory is released
            if (PAIR) umma_commit_pair(mapa_shared(smem_u32(drain), 0));
            else umma_commit(drain);
            mbar_wait(drain, 0, 0x805);
        }
    } else {
        // ---------------------------------------------------------------- epilogue
        // Warp: TMEM lane quarter q, 64 columns.  Its box of 32 rows x 128 bytes (128-byte swizzle) first
        // receives the addend by TMA, then each lane turns its row into D's, then a bulk store takes it.
        const int q = warp & 3, cb = ((warp - 2) >> 2) * 64;
        uint8_t* box = smem + C::OFF_STG + (warp - 2) * C::BOX_BYTES;
        uint64_t* addb = &add_full[warp - 2];
        auto at = [&](uint8_t* b, int c16) -> uint8_t* { return b + lane * 128 + ((c16 ^ (lane & 7)) << 4); };
        int lt = 0;
        uint32_t addph = 0;
        bool ok = true;
        for (int t = cid; t < p.ntile; t += ncid, ++lt) {
            const Tile ti = decode(t);
            const int buf = lt & 1;
            const int row0 = ti.m * 128 + q * 32, row = row0 + lane;
            const int col0 = ti.n * BN + cb;
            // columns of this warp inside D (none where its rows are past the extent): uniform in the warp
            const int ncol = row0 < p.rows ? min(64, p.cols - col0) : 0;
            // (where z is kept whole the box is its first, and a lane reads its row of the addend from memory)
            const bool add = !F32OUT && SAVE != LIN_KEEP_FULL && p.add && ncol > 0;
            // the box is free once the last tile's store has read it; without an addend that is waited for
            // as late as the first write
            auto free_box = [&]() {
                if (lane == 0) bulk_wait_read_all();
                __syncwarp();
            };
            if (add && lane == 0) {
                bulk_wait_read_all();
                mbar_arrive_expect_tx(addb, 4096);
                tma_load_3d(box, &tmR, addb, col0, ti.g, row0);
            }
            // two columns' bias a lane (by the columns alone: warps without rows write the shared values too)
            uint32_t bw = 0u;
            if (!F32OUT && p.bias && col0 + 2 * lane < p.cols)
                bw = __ldg(reinterpret_cast<const uint32_t*>(p.bias + (size_t)ti.g * p.cols + col0 + 2 * lane));
            if (!wait_or_abort(&acc_full[buf], (lt >> 1) & 1, abort_flag, 0x803)) ok = false;
            if (add) {                       // also on the way out: the load lands before the block ends
                ok = wait_or_abort(addb, addph, abort_flag, 0x807) && ok;
                if (!ok) mbar_wait(addb, addph, 0x808);
                addph ^= 1;
            }
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            // into shared memory, behind the wait: by then every warp has read the bias of the tile before
            // last, which lay there.  The four warps of a column block write the same values.
            float* sbias = reinterpret_cast<float*>(smem + C::OFF_BIAS) + buf * BN + cb;
            if (!F32OUT && p.bias) *reinterpret_cast<float2*>(sbias + 2 * lane) = make_float2(bf16_lo(bw), bf16_hi(bw));
            __syncwarp();
            const uint32_t taddr = tmem_base + (uint32_t(q * 32) << 16) + buf * BN + cb;
            int e2[2] = {0, 0};              // exponents of the row's two blocks
            uint32_t y[SAVE == LIN_KEEP_FULL ? 32 : 1];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[32];
                if (32 * h < ncol) {
                    tmem_ld32(taddr + 32 * h, v);
                    if (!F32OUT && p.bias) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 w = *reinterpret_cast<const float4*>(sbias + 32 * h + 4 * i);
                            const float2 lo = __fadd2_rn(make_float2(v[4 * i], v[4 * i + 1]), make_float2(w.x, w.y));
                            const float2 hi = __fadd2_rn(make_float2(v[4 * i + 2], v[4 * i + 3]), make_float2(w.z, w.w));
                            v[4 * i] = lo.x;
                            v[4 * i + 1] = lo.y;
                            v[4 * i + 2] = hi.x;
                            v[4 * i + 3] = hi.y;
                        }
                    }
                }
                if (h == 1) {
                    // the accumulator and the bias are read: the next MMAs into this buffer may start
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (PAIR) arrive_remote(mapa_shared(smem_u32(&acc_empty[buf]), 0));
                        else mbar_arrive(&acc_empty[buf]);
                    }
                }
                if (32 * h >= ncol) continue;
                if constexpr (F32OUT) {
                    free_box();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<float4*>(at(box, i)) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&tmO, box, col0 + 32 * h, row0, ti.s * p.groups + ti.g);
                        bulk_commit_group();
                    }
                } else {
                    if constexpr (SAVE == LIN_KEEP_CK8) {
                        // this lane's 32 columns are one block of its row (those past the row are zero: their
                        // weights and bias were read as zero); its codes go out from here, a whole sector
                        // (through the box, in 64-byte row pieces, the copying cost as much as it saved)
                        uint32_t qw[8];
                        e2[h] = ck8_quantize<32, 1>(reinterpret_cast<const float2(&)[16]>(v), qw);
                        if (row < p.rows) {
                            int8_t* cp = p.codes + ((size_t)row * p.groups + ti.g) * p.cols + col0 + 32 * h;
                            if ((p.cols & 15) == 0) {
                                *reinterpret_cast<uint4*>(cp) = make_uint4(qw[0], qw[1], qw[2], qw[3]);
                                if (32 * h + 16 < ncol) *reinterpret_cast<uint4*>(cp + 16) = make_uint4(qw[4], qw[5], qw[6], qw[7]);
                            } else {                                          // rows that start 8 bytes off
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (32 * h + 8 * i < ncol) *reinterpret_cast<uint2*>(cp + 8 * i) = make_uint2(qw[2 * i], qw[2 * i + 1]);
                            }
                        }
                    }
                    if constexpr (SAVE == LIN_KEEP_FULL) {
                        // z goes into the box first, y stays in registers until z is copied out
                        if (h == 0) free_box();
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *reinterpret_cast<uint4*>(at(box, 4 * h + i)) =
                                make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                                           pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 o = lin_act2<ACT>(make_float2(v[2 * i], v[2 * i + 1]));
                        v[2 * i] = o.x;
                        v[2 * i + 1] = o.y;
                    }
                    if (SAVE != LIN_KEEP_FULL && !add && h == 0) free_box();
                    if (add) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint4 w = *reinterpret_cast<const uint4*>(at(box, 4 * h + i));
                            const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float2 r = __fadd2_rn(make_float2(v[8 * i + 2 * k], v[8 * i + 2 * k + 1]),
                                                            make_float2(bf16_lo(a[k]), bf16_hi(a[k])));
                                v[8 * i + 2 * k] = r.x;
                                v[8 * i + 2 * k + 1] = r.y;
                            }
                        }
                    }
                    if constexpr (SAVE == LIN_KEEP_FULL) {
                        if (p.add && row < p.rows) {
                            const __nv_bfloat16* rp = p.res + ((size_t)row * p.groups + ti.g) * p.cols + col0 + 32 * h;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (32 * h + 8 * i < ncol) {
                                    const uint4 w = __ldg(reinterpret_cast<const uint4*>(rp + 8 * i));
                                    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        v[8 * i + 2 * k] += bf16_lo(a[k]);
                                        v[8 * i + 2 * k + 1] += bf16_hi(a[k]);
                                    }
                                }
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) y[16 * h + i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *reinterpret_cast<uint4*>(at(box, 4 * h + i)) =
                                make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                                           pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
                    }
                }
            }
            if constexpr (SAVE == LIN_KEEP_FULL) {
                if (ncol > 0) {
                    // z leaves the box in whole 128-byte row pieces, four rows a store, then y takes its place
                    // (a second box for z took the operand ring from five stages to three: 30 % of the large layer)
                    __syncwarp();
                    const int rl = lane >> 3, c16 = lane & 7;
                    const size_t rs = (size_t)p.groups * p.cols;
                    __nv_bfloat16* zp = p.z + ((size_t)(row0 + rl) * p.groups + ti.g) * p.cols + col0 + c16 * 8;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = 4 * i + rl;
                        const uint4 w = *reinterpret_cast<const uint4*>(box + r * 128 + ((c16 ^ (r & 7)) << 4));
                        if (c16 * 8 < ncol && row0 + r < p.rows) *reinterpret_cast<uint4*>(zp + 4 * i * rs) = w;
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4*>(at(box, i)) = make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                }
            }
            if constexpr (!F32OUT) {
                if (ncol > 0) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (OUT_MAT) tma_store_3d(&tmO, box, col0, row0, ti.g);
                        else tma_store_3d(&tmO, box, col0, ti.g, row0);
                        bulk_commit_group();
                    }
                    if constexpr (SAVE == LIN_KEEP_CK8) {
                        if (row < p.rows) {
                            int8_t* ep = p.exps + ((size_t)row * p.groups + ti.g) * p.nblk + (col0 >> 5);
                            if ((p.nblk & 1) == 0) {
                                *reinterpret_cast<uint16_t*>(ep) = (uint16_t)((e2[0] & 0xFF) | (e2[1] & 0xFF) << 8);
                            } else {
                                ep[0] = (int8_t)e2[0];
                                if (ncol > 32) ep[1] = (int8_t)e2[1];
                            }
                        }
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }
    tc_fence_before();
    // pair mode: neither CTA releases its tensor memory or exits while the other may still arrive on its
    // barriers or be the target of the pair's MMAs
    if (PAIR) cluster_sync_all();
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        if (PAIR) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
        else tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

}  // namespace tml
