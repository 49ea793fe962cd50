// tm_postnorm.cu -- host side of the post-norm block's calls (include/tm.h): validation, tensor maps,
// workspace and launch sequence of the layer norm, the per-token linear layer and the 8-bit
// checkpoints.  Part of the single translation unit, after tm_api.cu, whose helpers it uses.

namespace tml {
namespace {

// A tensor of a call: its bytes, to be aligned and apart from every other one that is written.
struct Span {
    const void* p;
    size_t bytes;
    bool out;
    unsigned align = 16;
};
// Every span present is aligned, and no output overlaps another span.
template <int N>
bool spans_ok(const Span (&s)[N]) {
    for (int i = 0; i < N; ++i) {
        if (!s[i].p) continue;
        if ((reinterpret_cast<uintptr_t>(s[i].p) & (s[i].align - 1)) != 0) return false;
        for (int j = 0; j < N; ++j) {
            if (i == j || !s[j].p || !s[i].out) continue;
            const uintptr_t a = (uintptr_t)s[i].p, b = (uintptr_t)s[j].p;
            if (a < b + s[j].bytes && b < a + s[i].bytes) return false;
        }
    }
    return true;
}
bool ckpt_ok(const tm_ckpt8* c) { return !c || (c->codes && c->exps); }
size_t ckpt_exps(size_t rows, int width) { return rows * (size_t)ck8_blocks(width); }

// Geometry of normalised rows: as make_geo, but the row layout takes rows of any width.
tm_status make_norm_geo(const tm_shape* s, int layout, const tm_layer_norm_w* w, Geo* g) {
    if (!w) return TM_ERR_INVALID_ARG;
    tm_status st = check_shape(s);
    if (st != TM_OK) return st;
    if (layout == TM_LAYOUT_ROWS) {
        if (w->banks <= 0 || w->width <= 0) return TM_ERR_INVALID_ARG;
        if ((long long)s->B * w->banks > (1LL << 28)) return TM_ERR_UNSUPPORTED;
        g->B = s->B;
        g->banks = w->banks;
        g->W = w->width;
        g->dtype = s->dtype;
        g->esz = s->dtype == TM_BF16 ? 2 : 4;
        g->eps = s->eps;
        g->map = RowMap{0, w->banks, w->width, s->T, s->D, s->D / s->H};
    } else if ((st = make_geo(s, layout, w->banks, w->width, g)) != TM_OK) {
        return st;
    }
    return g->W <= norm_max_width() ? TM_OK : TM_ERR_UNSUPPORTED;
}

NormParams norm_params(const Geo& g, const tm_layer_norm_w* w, const void* x, const void* res) {
    NormParams p;
    memset(&p, 0, sizeof(p));
    p.x = x;
    p.res = res;
    p.gain = w->gain;
    p.bias = w->bias;
    p.map = g.map;
    p.B = g.B;
    p.eps = g.eps;
    p.inv_w = 1.0f / (float)g.W;
    p.banks = fast_div(g.banks);
    return p;
}

// ------------------------------------------------------------------ per-token linear layer
constexpr long long kLinMostCols = INT32_MAX - 255;   // of all banks together
struct LinGeo {
    int B, banks, K, N, dtype;
    size_t esz;
};
tm_status make_lin_geo(const tm_shape* s, const tm_linear_w* w, LinGeo* g) {
    if (!w) return TM_ERR_INVALID_ARG;
    tm_status st = check_shape(s);
    if (st != TM_OK) return st;
    if (w->banks <= 0 || w->width <= 0 || w->out <= 0 || !w->w) return TM_ERR_INVALID_ARG;
    if (w->act < TM_ACT_NONE || w->act > TM_ACT_SILU) return TM_ERR_INVALID_ARG;
    if (!al16(w->w) || (w->bias && !al16(w->bias))) return TM_ERR_INVALID_ARG;
    if ((long long)s->B * w->banks > (1LL << 28)) return TM_ERR_UNSUPPORTED;
    // columns are 32-bit integers, rounded up to a tile's (and a row of x or y across the banks is a tensor-map
    // stride, below 2^40 bytes)
    if ((long long)w->banks * w->width > kLinMostCols || (long long)w->banks * w->out > kLinMostCols)
        return TM_ERR_UNSUPPORTED;
    if (s->dtype == TM_BF16) {
        if (w->width % 8 || w->out % 8) return TM_ERR_UNSUPPORTED;   // 16-byte strides of the tensor maps
        // tiles are counted in 32 bits
        auto t = [](long long v) { return (v + 127) / 128; };
        if ((long long)w->banks * t(s->B) * t(w->out) > (1 << 26) || (long long)w->banks * t(s->B) * t(w->width) > (1 << 26) ||
            (long long)w->banks * t(w->out) * t(w->width) > (1 << 26))
            return TM_ERR_UNSUPPORTED;
    } else {
        if (w->banks > 65535 || (s->B + 63) / 64 > 65535 || (w->out + 63) / 64 > 65535) return TM_ERR_UNSUPPORTED;
    }
    g->B = s->B;
    g->banks = w->banks;
    g->K = w->width;
    g->N = w->out;
    g->dtype = s->dtype;
    g->esz = s->dtype == TM_BF16 ? 2 : 4;
    return TM_OK;
}

// bf16 tensor map of [d2][d1][d0] (d0 contiguous; strides in elements) with a box of b0 x b1 x b2
bool map_3d(CUtensorMap* m, const void* base, uint64_t d0, uint64_t d1, uint64_t s1, uint64_t d2, uint64_t s2,
            uint32_t b0, uint32_t b1, uint32_t b2, CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B) {
    uint64_t dims[3] = {d0, d1, d2};
    uint64_t strides[2] = {s1 * 2, s2 * 2};
    uint32_t box[3] = {b0, b1, b2};
    return make_map(m, base, 3, dims, strides, box, swz);
}
// rows [B, banks, W] of bf16: boxes of b0 columns of one bank by b2 samples
bool map_rows(CUtensorMap* m, const void* base, int B, int banks, int W, uint32_t b0, uint32_t b2,
              CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B) {
    return map_3d(m, base, W, banks, W, B, (uint64_t)banks * W, b0, 1, b2, swz);
}
// matrices [banks, R, W] of bf16: boxes of b0 columns by b1 rows of one bank
bool map_mats(CUtensorMap* m, const void* base, int banks, int R, int W, uint32_t b0, uint32_t b1,
              CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B) {
    return map_3d(m, base, W, R, W, banks, (uint64_t)R * W, b0, b1, 1, swz);
}
bool map_mats_f32(CUtensorMap* m, const void* base, uint64_t mats, int R, int W) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)W, (cuuint64_t)R, mats};
    cuuint64_t strides[2] = {(cuuint64_t)W * 4, (cuuint64_t)R * W * 4};
    cuuint32_t box[3] = {32, 32, 1}, es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tile shape and contraction splits of one contraction.  Estimated time in units of one 64-deep slab of
// a pair's 256 x 256 tile (about 512 tensor-core cycles): full waves of tiles times slabs, plus a tile's
// fill and epilogue.  A 128 x 128 tile does a quarter of the work on half the SMs: its slab takes 0.6 of a
// pair's, bound by its loads (as many bytes per SM), or 0.95 where both operands come in 64-row boxes (dW);
// a split adds the partial sums' way out and back through memory and one more launch.  Measured (gelu, twenty kernels
// in a row in a graph, operands in the L2 where they fit), pair / tile:
// forward 16 banks of 4096 x 256 -> 1024 45 / 53 us, 8 of 4096 x 768 -> 1536 71 / 90, 4 of 1000 x 512 -> 512
// 11.2 / 8.3, 16 of 333 x 384 -> 264 11.2 / 8.2; dW of 8 x 3829 x 168 x 600 as 1 / 2 / 3 / 4 runs 40 / 26 / 21 / 28,
// of 48 x 1419 x 888 x 568 99 / 156 / 187 / 215.  Over 60 random dW the choice is 1.7 % above the best of all.
struct LinPlan {
    bool pair;
    int splits, split_slabs;
};
LinPlan plan_contraction(long long groups, int rows, int cols, int depth, bool may_split, int sms) {
    const int slabs = (depth + 63) / 64;
    LinPlan best{false, 1, slabs};
    double best_cost = 1e300;
    for (int pair = 1; pair >= 0; --pair) {
        const int bm = pair ? 256 : 128;
        const double unit = pair ? 1.0 : may_split ? 0.95 : 0.6;
        const int units = pair ? sms / 2 : sms;
        if (pair && (rows <= 128 || cols <= 128 || units < 1)) continue;
        const long long tiles = groups * ((rows + bm - 1) / bm) * ((cols + bm - 1) / bm);
        for (int s = 1; s <= (may_split ? 16 : 1); ++s) {
            const int per = (slabs + s - 1) / s;
            if (s > 1 && (per < 4 || (s - 1) * per >= slabs)) continue;
            const double waves = (double)((tiles * s + units - 1) / units);
            double cost = waves * unit * (per + 2.0);
            if (s > 1) cost += 10.0 + 8.0 * s * (double)groups * rows * cols / 6.5e12 / 2.8e-7;
            if (cost < best_cost) {
                best_cost = cost;
                best = LinPlan{pair != 0, s, per};
            }
        }
    }
    return best;
}

LinParams lin_params(int groups, int rows, int cols, int depth, const LinPlan& pl) {
    LinParams p;
    memset(&p, 0, sizeof(p));
    p.groups = groups;
    p.rows = rows;
    p.cols = cols;
    p.depth = depth;
    const int bm = pl.pair ? 256 : 128;
    p.mt = fast_div((rows + bm - 1) / bm);
    p.nt = fast_div((cols + bm - 1) / bm);
    p.splits = fast_div(pl.splits);
    p.ntile = (int)(groups * p.mt.d * p.nt.d * p.splits.d);
    p.split_slabs = pl.split_slabs;
    return p;
}

struct LinBwdWs {
    void* dz;
    float* db;
    float* dw;
    int chunks;
    LinPlan dw_plan;
};
LinBwdWs carve_lin_bwd(Carve& c, const LinGeo& g, int act) {
    LinBwdWs w;
    const size_t cols = (size_t)g.banks * g.N;
    w.dz = act == TM_ACT_NONE ? nullptr : (void*)c.take<uint8_t>((size_t)g.B * cols * g.esz);
    w.chunks = act_bwd_chunks(g.dtype, g.B, cols, g.N, num_sms());
    w.db = c.take<float>((size_t)w.chunks * cols);
    w.dw_plan = g.dtype == TM_BF16 ? plan_contraction(g.banks, g.N, g.K, g.B, true, num_sms()) : LinPlan{false, 1, 0};
    w.dw = w.dw_plan.splits > 1 ? c.take<float>((size_t)w.dw_plan.splits * cols * g.K) : nullptr;
    return w;
}

// fp32 contractions on CUDA cores
SimtLin simt_lin(const LinGeo& g, const void* a, const void* b, void* d) {
    SimtLin p;
    memset(&p, 0, sizeof(p));
    p.a = (const float*)a;
    p.b = (const float*)b;
    p.d = (float*)d;
    p.groups = g.banks;
    p.nblk = (g.N + kCk8Block - 1) / kCk8Block;
    return p;
}

}  // namespace
}  // namespace tml

using namespace tml;

extern "C" {

tm_status tm_checkpoint8_pack(const void* x, tm_dtype dtype, size_t rows, int width, const tm_ckpt8* out,
                              void* stream) {
    if ((dtype != TM_F32 && dtype != TM_BF16) || rows < 1 || width < 1 || !x || !out || !ckpt_ok(out))
        return TM_ERR_INVALID_ARG;
    if (rows > (size_t)1 << 40 || rows > ((size_t)1 << 46) / width) return TM_ERR_UNSUPPORTED;
    const size_t n = rows * width;
    const Span sp[] = {{x, n * (dtype == TM_BF16 ? 2 : 4), false},
                       {out->codes, n, true},
                       {out->exps, ckpt_exps(rows, width), true}};
    if (!spans_ok(sp)) return TM_ERR_INVALID_ARG;
    return cuda_status(launch_ckpt8(true, dtype, const_cast<void*>(x), out->codes, out->exps, (long long)rows, width,
                                    num_sms(), (cudaStream_t)stream));
}

tm_status tm_checkpoint8_unpack(const tm_ckpt8* in, tm_dtype dtype, size_t rows, int width, void* x, void* stream) {
    if ((dtype != TM_F32 && dtype != TM_BF16) || rows < 1 || width < 1 || !x || !in || !ckpt_ok(in))
        return TM_ERR_INVALID_ARG;
    if (rows > (size_t)1 << 40 || rows > ((size_t)1 << 46) / width) return TM_ERR_UNSUPPORTED;
    const size_t n = rows * width;
    const Span sp[] = {{x, n * (dtype == TM_BF16 ? 2 : 4), true},
                       {in->codes, n, false},
                       {in->exps, ckpt_exps(rows, width), false}};
    if (!spans_ok(sp)) return TM_ERR_INVALID_ARG;
    return cuda_status(launch_ckpt8(false, dtype, x, in->codes, in->exps, (long long)rows, width, num_sms(),
                                    (cudaStream_t)stream));
}

tm_status tm_layer_norm(const void* x, const void* residual, tm_layout layout, const tm_shape* shape,
                        const tm_layer_norm_w* w, void* y, float* mean_opt, float* rstd_opt, const tm_ckpt8* save_opt,
                        void* stream) {
    Geo g;
    tm_status s = make_norm_geo(shape, layout, w, &g);
    if (s != TM_OK) return s;
    if (!x || !y || !ckpt_ok(save_opt)) return TM_ERR_INVALID_ARG;
    const size_t rows = (size_t)g.B * g.banks, n = rows * g.W * g.esz;
    const Span sp[] = {{x, n, false},
                       {residual, n, false},
                       {w->gain, g.W * g.esz, false},
                       {w->bias, g.W * g.esz, false},
                       {y, n, true},
                       {mean_opt, rows * 4, true, 4},
                       {rstd_opt, rows * 4, true, 4},
                       {save_opt ? save_opt->codes : nullptr, rows * g.W, true},
                       {save_opt ? save_opt->exps : nullptr, ckpt_exps(rows, g.W), true}};
    if (!spans_ok(sp)) return TM_ERR_INVALID_ARG;
    NormParams p = norm_params(g, w, x, residual);
    p.y = y;
    p.mean = mean_opt;
    p.rstd = rstd_opt;
    p.codes = save_opt ? save_opt->codes : nullptr;
    p.exps = save_opt ? save_opt->exps : nullptr;
    return cuda_status(launch_ln_fwd(g.dtype, p, num_sms(), (cudaStream_t)stream));
}

size_t tm_layer_norm_backward_workspace_bytes(const tm_shape* shape, tm_layout layout, const tm_layer_norm_w* w) {
    Geo g;
    if (make_norm_geo(shape, layout, w, &g) != TM_OK) return 0;
    return align256(ln_part_floats((long long)g.B * g.banks, g.W, num_sms()) * sizeof(float));
}

tm_status tm_layer_norm_backward(const void* x, const void* residual, const tm_ckpt8* saved, const float* mean,
                                 const float* rstd, const void* dy, tm_layout layout, const tm_shape* shape,
                                 const tm_layer_norm_w* w, int residual_is_x, void* dx, void* dresidual_opt,
                                 const tm_layer_norm_grads* grads, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    Geo g;
    tm_status s = make_norm_geo(shape, layout, w, &g);
    if (s != TM_OK) return s;
    const bool self = residual_is_x != 0;
    if (!mean || !rstd || !dy || !dx || !ckpt_ok(saved) || (!saved && !x)) return TM_ERR_INVALID_ARG;
    if (layout == TM_LAYOUT_ROWS && (self || dresidual_opt)) return TM_ERR_INVALID_ARG;
    if (self) {
        if (shape->T != shape->H || dresidual_opt || (!saved && residual != x)) return TM_ERR_INVALID_ARG;
        if (!ln_self_supported(g.banks, g.W)) return TM_ERR_UNSUPPORTED;
    }
    void* dgain = grads ? grads->dgain : nullptr;
    void* dbias = grads ? grads->dbias : nullptr;
    const size_t rows = (size_t)g.B * g.banks, n = rows * g.W * g.esz, wb = g.W * g.esz;
    const size_t need = (dgain || dbias) ? tm_layer_norm_backward_workspace_bytes(shape, layout, w) : 0;
    if (need && (!workspace || workspace_bytes < need)) return TM_ERR_WORKSPACE;
    const Span sp[] = {{saved ? nullptr : x, n, false},
                       {saved ? nullptr : residual, n, false},
                       {saved ? saved->codes : nullptr, rows * g.W, false},
                       {saved ? saved->exps : nullptr, ckpt_exps(rows, g.W), false},
                       {mean, rows * 4, false, 4},
                       {rstd, rows * 4, false, 4},
                       {dy, n, false},
                       {w->gain, wb, false},
                       {dx, n, true},
                       {dresidual_opt, n, true},
                       {dgain, wb, true},
                       {dbias, wb, true},
                       {need ? workspace : nullptr, need, true}};
    if (!spans_ok(sp)) return TM_ERR_INVALID_ARG;
    NormParams p = norm_params(g, w, saved ? nullptr : x, saved ? nullptr : residual);
    p.mean = const_cast<float*>(mean);
    p.rstd = const_cast<float*>(rstd);
    p.codes = saved ? saved->codes : nullptr;
    p.exps = saved ? saved->exps : nullptr;
    p.dy = dy;
    p.dx = dx;
    p.dres = dresidual_opt;
    p.part = need ? (float*)workspace : nullptr;
    return cuda_status(launch_ln_bwd(g.dtype, p, self, dgain, dbias, num_sms(), (cudaStream_t)stream));
}

tm_status tm_pertoken_linear(const void* x, const void* residual, const tm_shape* shape, const tm_linear_w* w, void* y,
                             void* z_opt, const tm_ckpt8* save_opt, void* stream) {
    LinGeo g;
    tm_status s = make_lin_geo(shape, w, &g);
    if (s != TM_OK) return s;
    if (!x || !y || !ckpt_ok(save_opt) || (z_opt && save_opt) || ((z_opt || save_opt) && w->act == TM_ACT_NONE))
        return TM_ERR_INVALID_ARG;
    const size_t rows = (size_t)g.B * g.banks, nk = rows * g.K * g.esz, nn = rows * g.N * g.esz;
    const Span sp[] = {{x, nk, false},
                       {residual, nn, false},
                       {w->w, (size_t)g.banks * g.N * g.K * g.esz, false},
                       {w->bias, (size_t)g.banks * g.N * g.esz, false},
                       {y, nn, true},
                       {z_opt, nn, true},
                       {save_opt ? save_opt->codes : nullptr, rows * g.N, true},
                       {save_opt ? save_opt->exps : nullptr, ckpt_exps(rows, g.N), true}};
    if (!spans_ok(sp)) return TM_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (g.dtype == TM_F32) {
        SimtLin p = simt_lin(g, x, w->w, y);
        p.bias = (const float*)w->bias;
        p.add = (const float*)residual;
        p.z = (float*)z_opt;
        p.codes = save_opt ? save_opt->codes : nullptr;
        p.exps = save_opt ? save_opt->exps : nullptr;
        p.ag = g.K; p.am = (long long)g.banks * g.K; p.ak = 1;
        p.bg = (long long)g.N * g.K; p.bn = g.K; p.bk = 1;
        p.dg = g.N; p.dm = (long long)g.banks * g.N;
        p.M = g.B; p.N = g.N; p.K = g.K;
        p.act = w->act;
        return cuda_status(launch_linear_simt(p, st));
    }
    const int save = z_opt ? LIN_KEEP_FULL : save_opt ? LIN_KEEP_CK8 : LIN_KEEP_NOTHING;
    if (g.B == 1 && g.banks <= 65535) {          // the weights' stream alone; the grid has a bank in y
        const RowLin p{(const __nv_bfloat16*)x, (const __nv_bfloat16*)w->w, (const __nv_bfloat16*)w->bias,
                       (const __nv_bfloat16*)residual, (__nv_bfloat16*)y, (__nv_bfloat16*)z_opt,
                       save_opt ? save_opt->codes : nullptr, save_opt ? save_opt->exps : nullptr,
                       g.K, g.N, (g.N + kCk8Block - 1) / kCk8Block};
        return cuda_status(launch_linear_row(g.banks, w->act, save, p, st));
    }
    const LinPlan pl = plan_contraction(g.banks, g.B, g.N, g.K, false, num_sms());
    LinParams p = lin_params(g.banks, g.B, g.N, g.K, pl);
    p.bias = (const __nv_bfloat16*)w->bias;
    p.add = residual != nullptr;
    p.res = (const __nv_bfloat16*)residual;
    p.z = (__nv_bfloat16*)z_opt;
    p.codes = save_opt ? save_opt->codes : nullptr;
    p.exps = save_opt ? save_opt->exps : nullptr;
    p.nblk = (g.N + kCk8Block - 1) / kCk8Block;
    LinMaps m;
    if (!map_rows(&m.a, x, g.B, g.banks, g.K, 64, 128) || !map_mats(&m.b, w->w, g.banks, g.N, g.K, 64, 128) ||
        !map_rows(&m.o, y, g.B, g.banks, g.N, 64, 32))
        return TM_ERR_CUDA;
    m.r = m.o;
    if (residual && !map_rows(&m.r, residual, g.B, g.banks, g.N, 64, 32)) return TM_ERR_CUDA;
    return cuda_status(launch_linear_fwd(pl.pair, w->act, save, m, p, num_sms(), st));
}

size_t tm_pertoken_linear_backward_workspace_bytes(const tm_shape* shape, const tm_linear_w* w) {
    LinGeo g;
    if (make_lin_geo(shape, w, &g) != TM_OK) return 0;
    Carve c{nullptr};
    carve_lin_bwd(c, g, w->act);
    return align256(c.off);
}

tm_status tm_pertoken_linear_backward(const void* x, const void* dy, const void* z, const tm_ckpt8* saved,
                                      const void* dx_add, const tm_shape* shape, const tm_linear_w* w, void* dx,
                                      const tm_linear_grads* grads, void* workspace, size_t workspace_bytes,
                                      void* stream) {
    LinGeo g;
    tm_status s = make_lin_geo(shape, w, &g);
    if (s != TM_OK) return s;
    const bool act = w->act != TM_ACT_NONE;
    void* dw = grads ? grads->dw : nullptr;
    void* db = grads ? grads->db : nullptr;
    if (!dy || (dw && !x) || (dx_add && !dx) || (act && !z == !saved) || !ckpt_ok(saved)) return TM_ERR_INVALID_ARG;
    if (!act) z = nullptr, saved = nullptr;
    if (!dx && !dw && !db) return TM_OK;
    Carve c{(uint8_t*)workspace};
    const LinBwdWs ws = carve_lin_bwd(c, g, w->act);
    const size_t need = align256(c.off);
    if (!workspace || workspace_bytes < need) return TM_ERR_WORKSPACE;
    const size_t rows = (size_t)g.B * g.banks, nk = rows * g.K * g.esz, nn = rows * g.N * g.esz;
    const size_t wb = (size_t)g.banks * g.N * g.K * g.esz;
    const Span sp[] = {{dw ? x : nullptr, nk, false},
                       {dy, nn, false},
                       {z, nn, false},
                       {saved ? saved->codes : nullptr, rows * g.N, false},
                       {saved ? saved->exps : nullptr, ckpt_exps(rows, g.N), false},
                       {dx_add, nk, false},
                       {w->w, wb, false},
                       {dx, nk, true},
                       {dw, wb, true},
                       {db, (size_t)g.banks * g.N * g.esz, true},
                       {workspace, need, true}};
    if (!spans_ok(sp)) return TM_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    const long long cols = (long long)g.banks * g.N;
    const void* dz = dy;
    if (act || db) {
        dz = act ? ws.dz : dy;
        s = cuda_status(launch_act_bwd(g.dtype, dy, z, saved ? saved->codes : nullptr, saved ? saved->exps : nullptr,
                                       w->act, g.B, cols, g.N, ws.chunks, ws.dz, db ? ws.db : nullptr, st));
        if (s != TM_OK) return s;
        if (db && (s = cuda_status(launch_sum_parts(g.dtype, ws.db, ws.chunks, cols, db, st))) != TM_OK) return s;
    }
    if (g.dtype == TM_F32) {
        if (dx) {
            SimtLin p = simt_lin(g, dz, w->w, dx);
            p.add = (const float*)dx_add;
            p.ag = g.N; p.am = cols; p.ak = 1;
            p.bg = (long long)g.N * g.K; p.bn = 1; p.bk = g.K;
            p.dg = g.K; p.dm = (long long)g.banks * g.K;
            p.M = g.B; p.N = g.K; p.K = g.N;
            if ((s = cuda_status(launch_linear_simt(p, st))) != TM_OK) return s;
        }
        if (dw) {
            SimtLin p = simt_lin(g, dz, x, dw);
            p.ag = g.N; p.am = 1; p.ak = cols;
            p.bg = g.K; p.bn = 1; p.bk = (long long)g.banks * g.K;
            p.dg = (long long)g.N * g.K; p.dm = g.K;
            p.M = g.N; p.N = g.K; p.K = g.B;
            return cuda_status(launch_linear_simt(p, st));
        }
        return TM_OK;
    }
    LinMaps m;
    if (dx) {
        const LinPlan pl = plan_contraction(g.banks, g.B, g.K, g.N, false, num_sms());
        LinParams p = lin_params(g.banks, g.B, g.K, g.N, pl);
        p.add = dx_add != nullptr;
        if (!map_rows(&m.a, dz, g.B, g.banks, g.N, 64, 128) || !map_mats(&m.b, w->w, g.banks, g.N, g.K, 64, 64) ||
            !map_rows(&m.o, dx, g.B, g.banks, g.K, 64, 32))
            return TM_ERR_CUDA;
        m.r = m.o;
        if (dx_add && !map_rows(&m.r, dx_add, g.B, g.banks, g.K, 64, 32)) return TM_ERR_CUDA;
        if ((s = cuda_status(launch_linear_dx(pl.pair, m, p, num_sms(), st))) != TM_OK) return s;
    }
    if (dw) {
        const LinPlan& pl = ws.dw_plan;
        LinParams p = lin_params(g.banks, g.N, g.K, g.B, pl);
        if (!map_rows(&m.a, dz, g.B, g.banks, g.N, 64, 64) || !map_rows(&m.b, x, g.B, g.banks, g.K, 64, 64))
            return TM_ERR_CUDA;
        if (pl.splits > 1 ? !map_mats_f32(&m.o, ws.dw, (uint64_t)pl.splits * g.banks, g.N, g.K)
                          : !map_mats(&m.o, dw, g.banks, g.N, g.K, 64, 32))
            return TM_ERR_CUDA;
        m.r = m.o;
        if ((s = cuda_status(launch_linear_dw(pl.pair, m, p, num_sms(), st))) != TM_OK) return s;
        if (pl.splits > 1)
            return cuda_status(launch_sum_parts(g.dtype, ws.dw, pl.splits, cols * g.K, dw, st));
    }
    return TM_OK;
}

}  // extern "C"
