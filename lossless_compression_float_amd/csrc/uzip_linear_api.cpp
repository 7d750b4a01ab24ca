// uzip_linear_api.cpp -- the C ABI of the products with packed weights
// (include/uzip.h): argument checks, choice of kernels, workspace carving and
// launches on the caller's stream.  Nothing here allocates or synchronises.
#include <stdint.h>

#include <algorithm>

#include <hip/hip_runtime.h>

#include "uzip.h"
#include "uzip_args.hpp"
#include "uzip_linear.hpp"

using namespace uzip;

namespace {

// Token tiles of `edge` rows that a call can need: each group's last may be part of one.
uint32_t token_tiles(uint64_t tokens, uint64_t groups, bool grouped, uint64_t edge) {
    return (uint32_t)(grouped ? tokens / edge + std::min(groups, tokens) : blocks(tokens, edge));
}

// ---- forward ----------------------------------------------------------------

bool linear_ok(const uzip_weight *w, const uzip_linear_args *a, bool grouped) {
    if (!weight_ok(w) || !a || a->clear_rest > 1 || a->reserved) return false;
    if (grouped ? !a->offsets || !aligned(a->offsets, 4) || a->residual : a->offsets || w->matrices != 1) return false;
    if (!call_ok(w, a->tokens) || !type_ok(a->y_dtype) || a->act > UZIP_ACT_SWIGLU) return false;
    if ((a->act == UZIP_ACT_SWIGLU) != (w->gated == 1)) return false;
    const uint64_t out = w->rows / (w->gated + 1);
    if (!mat_ok(a->x, a->x_stride, a->tokens, w->cols, 2) || !mat_ok(a->y, a->y_stride, a->tokens, out, type_size(a->y_dtype)))
        return false;
    if (a->bias && (!type_ok(a->bias_dtype) || !aligned(a->bias, type_size(a->bias_dtype)))) return false;
    if (a->residual && !mat_ok(a->residual, a->residual_stride, a->tokens, out, type_size(a->y_dtype))) return false;
    return !a->preact || (type_ok(a->preact_dtype) && mat_ok(a->preact, a->preact_stride, a->tokens, w->rows, type_size(a->preact_dtype)));
}

LinearEpi linear_epi(const uzip_linear_args *a) {
    LinearEpi e{};
    e.bias = a->bias;
    e.residual = a->residual;
    e.y = a->y;
    e.preact = a->preact;
    e.preact_f32 = a->preact_dtype == UZIP_FP32;
    e.residual_stride = a->residual_stride;
    e.y_stride = a->y_stride;
    e.preact_stride = a->preact_stride;
    e.bias_f32 = a->bias_dtype == UZIP_FP32;
    e.y_f32 = a->y_dtype == UZIP_FP32;
    e.act = a->act;
    e.clear = a->clear_rest && a->offsets;
    return e;
}

// A tiled product's tiles and runs.
struct Cut {
    GemmTile tile;
    uint32_t r_tiles, c_tiles, splits;
    uint64_t part() const { return splits > 1 ? (uint64_t)splits * r_tiles * c_tiles * tile.r * tile.c : 0; }
    void set(GemmParams &p, float *part) const {
        p.r_tiles = r_tiles;
        p.c_tiles = c_tiles;
        p.splits = splits;
        p.part = part;
    }
};

// rows: of all parts together, padded to whole blocks in each.
Cut cut(GemmKind kind, uint64_t rows, uint64_t tokens, uint64_t groups, bool grouped, uint64_t steps) {
    Cut c{};
    c.tile = gemm_tile(kind, rows, tokens, groups);
    c.r_tiles = (uint32_t)blocks(rows, c.tile.r);
    c.c_tiles = token_tiles(tokens, groups, grouped, c.tile.c);
    c.splits = gemm_splits(kind, c.tile, c.r_tiles, c.c_tiles, steps);
    return c;
}

struct LinearPlan {
    uint16_t *x;
    float *part;
    Cut cut;
    bool skinny, stage;
};

LinearPlan plan_linear(const uzip_weight *w, const uzip_linear_args *a, Carver &c) {
    LinearPlan p{};
    const uint64_t groups = a->offsets ? w->matrices : 1;
    p.skinny = skinny_fits(a->tokens, groups, blocks(w->cols, kTileCols));
    p.stage = !tiled(a->x, a->x_stride, w->cols);
    if (p.stage) p.x = c.take<uint16_t>(a->tokens * up(w->cols, 8));
    if (!p.skinny) {
        const WeightLayout l = weight_layout(w->matrices, w->rows, w->cols, w->gated);
        p.cut = cut(kGemmForward, l.row_blocks * kTileRows, a->tokens, groups, a->offsets != nullptr, l.col_blocks);
        if (p.cut.part()) p.part = c.take<float>(p.cut.part());
    }
    return p;
}

uzip_status linear_run(const uzip_weight *w, const uzip_linear_args *a, void *ws, size_t ws_bytes, hipStream_t stream) {
    Carver c(ws);
    const LinearPlan plan = plan_linear(w, a, c);
    if (!workspace_ok(ws, ws_bytes, c.bytes())) return UZIP_ERR_INVALID_ARGUMENT;
    if (a->tokens == 0) return UZIP_OK;
    const bool grouped = a->offsets != nullptr;
    const uint32_t groups = grouped ? (uint32_t)w->matrices : 1;
    Mat x{a->x, a->x_stride};
    if (plan.stage) {
        x = Mat{plan.x, up(w->cols, 8)};
        const hipError_t e = launch_stage(static_cast<const uint16_t *>(a->x), a->x_stride, plan.x, x.stride, a->tokens,
                                          w->cols, stream);
        if (e != hipSuccess) return UZIP_ERR_DEVICE;
    }
    if (plan.skinny) {
        SkinnyParams p{};
        p.w = view(w);
        p.x = x;
        p.offsets = a->offsets;
        p.groups = groups;
        p.tokens = (uint32_t)a->tokens;
        p.rows = (uint32_t)w->rows;
        p.cols = (uint32_t)up(w->cols, 8);
        p.lin = linear_epi(a);
        return done(launch_skinny(p, stream));
    }
    GemmParams p{};
    p.w = view(w);
    p.cmat = x;
    p.offsets = a->offsets;
    p.groups = groups;
    p.tokens = (uint32_t)a->tokens;
    plan.cut.set(p, plan.part);
    p.c_limit = (uint32_t)up(w->cols, 8);
    p.steps = p.w.col_blocks;
    p.row_blocks = p.w.row_blocks;
    p.rows = (uint32_t)w->rows;
    p.cols = (uint32_t)w->cols;
    p.lin = linear_epi(a);
    return done(launch_gemm(kGemmForward, plan.cut.tile, p, stream));
}

// ---- backward ---------------------------------------------------------------

bool backward_ok(const uzip_weight *w, const uzip_linear_backward_args *a, bool grouped) {
    if (!weight_ok(w) || !a || a->clear_rest > 1 || a->reserved) return false;
    if (grouped ? !a->offsets || !aligned(a->offsets, 4) : a->offsets || w->matrices != 1) return false;
    if (!call_ok(w, a->tokens) || !type_ok(a->dy_dtype) || a->act > UZIP_ACT_SWIGLU) return false;
    if ((a->act == UZIP_ACT_SWIGLU) != (w->gated == 1)) return false;
    const uint64_t out = w->rows / (w->gated + 1);
    if (!mat_ok(a->dy, a->dy_stride, a->tokens, out, type_size(a->dy_dtype))) return false;
    if (a->act != UZIP_ACT_NONE &&
        (!type_ok(a->preact_dtype) || !mat_ok(a->preact, a->preact_stride, a->tokens, w->rows, type_size(a->preact_dtype))))
        return false;
    if (a->dx && !mat_ok(a->dx, a->dx_stride, a->tokens, w->cols, 2)) return false;
    if (a->dw && (!aligned(a->dw, 2) || !mat_ok(a->x, a->x_stride, a->tokens, w->cols, 2))) return false;
    return !a->dbias || (type_ok(a->dbias_dtype) && aligned(a->dbias, type_size(a->dbias_dtype)));
}

struct BackwardPlan {
    uint16_t *x, *dz;
    float *colsum, *part;
    Cut cut;         // of dx
    uint64_t width;  // padded columns of dz
    uint32_t chunks;
    bool stage_x, make_dz;
};

BackwardPlan plan_backward(const uzip_weight *w, const uzip_linear_backward_args *a, Carver &c) {
    const WeightLayout l = weight_layout(w->matrices, w->rows, w->cols, w->gated);
    const uint64_t groups = a->offsets ? w->matrices : 1;
    BackwardPlan p{};
    p.width = up(l.row_blocks * kTileRows, 64);
    p.make_dz = (a->dx || a->dw) &&
                (a->act != UZIP_ACT_NONE || a->dy_dtype == UZIP_FP32 || !tiled(a->dy, a->dy_stride, w->rows));
    p.stage_x = a->dw && !tiled(a->x, a->x_stride, w->cols);
    // runs of rows whose column sums are taken apart: about 2,048 workgroups (of 512 columns), of at least 8 rows
    const uint64_t wide = blocks(w->gated ? l.part_blocks * kTileRows : p.width, 512) * groups;
    p.chunks = (uint32_t)std::max<uint64_t>(1, std::min(blocks(2048, wide), blocks(a->tokens, 8)));
    if (p.make_dz) p.dz = c.take<uint16_t>(a->tokens * p.width);
    if (p.stage_x) p.x = c.take<uint16_t>(a->tokens * up(w->cols, 8));
    if (a->dbias) p.colsum = c.take<float>(groups * p.chunks * p.width);
    if (a->dx) {
        p.cut = cut(kGemmDx, w->cols, a->tokens, groups, a->offsets != nullptr, blocks(l.row_blocks, 4));
        if (p.cut.part()) p.part = c.take<float>(p.cut.part());
    }
    return p;
}

uzip_status backward_run(const uzip_weight *w, const uzip_linear_backward_args *a, void *ws, size_t ws_bytes,
                         hipStream_t stream) {
    Carver c(ws);
    const BackwardPlan plan = plan_backward(w, a, c);
    if (!workspace_ok(ws, ws_bytes, c.bytes())) return UZIP_ERR_INVALID_ARGUMENT;
    const bool grouped = a->offsets != nullptr;
    const uint32_t groups = grouped ? (uint32_t)w->matrices : 1;
    const WeightView v = view(w);
    if (plan.make_dz || a->dbias) {
        DzParams p{};
        p.dy = a->dy;
        p.dy_stride = a->dy_stride;
        p.z = a->preact;
        p.z_f32 = a->preact_dtype == UZIP_FP32;
        p.z_stride = a->preact_stride;
        p.dz = plan.dz;
        p.dz_stride = plan.width;
        p.colsum = plan.colsum;
        p.offsets = a->offsets;
        p.groups = groups;
        p.tokens = (uint32_t)a->tokens;
        p.part_rows = v.part_rows;
        p.part_pad = v.part_blocks * kTileRows;
        p.parts = v.parts;
        p.width = (uint32_t)plan.width;
        p.dy_f32 = a->dy_dtype == UZIP_FP32;
        p.act = a->act;
        p.chunks = plan.chunks;
        p.dbias = a->dbias;
        p.dbias_f32 = a->dbias_dtype == UZIP_FP32;
        if (launch_dz(p, stream) != hipSuccess) return UZIP_ERR_DEVICE;
    }
    GemmParams p{};
    p.w = v;
    p.offsets = a->offsets;
    p.groups = groups;
    p.tokens = (uint32_t)a->tokens;
    p.row_blocks = v.row_blocks;
    p.rows = (uint32_t)w->rows;
    p.cols = (uint32_t)w->cols;
    p.cmat = plan.make_dz ? Mat{plan.dz, plan.width} : Mat{a->dy, a->dy_stride};
    p.c_limit = (uint32_t)(plan.make_dz ? plan.width : w->rows);
    if (a->dx && a->tokens) {
        plan.cut.set(p, plan.part);
        p.steps = (uint32_t)blocks(v.row_blocks, 4);
        p.store = StoreEpi{};
        p.store.out = static_cast<uint16_t *>(a->dx);
        p.store.stride = a->dx_stride;
        p.store.clear = a->clear_rest && a->offsets;
        if (launch_gemm(kGemmDx, plan.cut.tile, p, stream) != hipSuccess) return UZIP_ERR_DEVICE;
    }
    if (a->dw) {
        p.rmat = Mat{a->x, a->x_stride};
        if (plan.stage_x) {
            p.rmat = Mat{plan.x, up(w->cols, 8)};
            if (launch_stage(static_cast<const uint16_t *>(a->x), a->x_stride, plan.x, p.rmat.stride, a->tokens, w->cols,
                             stream) != hipSuccess)
                return UZIP_ERR_DEVICE;
        }
        const GemmTile tile = gemm_tile(kGemmDw, w->cols, w->rows * groups, 1);
        p.r_limit = (uint32_t)up(w->cols, 8);
        p.r_tiles = (uint32_t)blocks(w->cols, tile.r);
        p.c_tiles = (uint32_t)blocks(v.row_blocks * kTileRows, tile.c);
        p.store = StoreEpi{};
        p.store.out = static_cast<uint16_t *>(a->dw);
        p.store.stride = w->cols;
        if (launch_gemm(kGemmDw, tile, p, stream) != hipSuccess) return UZIP_ERR_DEVICE;
    }
    return UZIP_OK;
}

// ---- loss -------------------------------------------------------------------

bool loss_ok(const uzip_weight *w, const uzip_loss_args *a, bool backward) {
    if (!weight_ok(w) || !a || w->matrices != 1 || w->gated || !call_ok(w, a->tokens)) return false;
    if (a->tokens == 0) return !(backward && a->dw) || aligned(a->dw, 2);
    if (!mat_ok(a->x, a->x_stride, a->tokens, w->cols, 2) || !a->target || !aligned(a->target, 8)) return false;
    if (!a->lse || !aligned(a->lse, 4)) return false;
    if (!backward) return a->loss && aligned(a->loss, 4);
    if (!a->dloss || !aligned(a->dloss, 4)) return false;
    if (a->dx && !mat_ok(a->dx, a->dx_stride, a->tokens, w->cols, 2)) return false;
    return !a->dw || aligned(a->dw, 2);
}

struct LossPlan {
    uint16_t *x;
    float2 *parts;
    float *picked, *part;
    uint16_t *dz;
    float *unit, *sum;
    uint64_t piece;  // rows of the weight in a piece
    Cut cut;         // of the forward product
    bool stage;
};

// The two products of a backward piece of `rows` weight rows that are cut.
Cut cut_dz(const uzip_weight *w, const uzip_loss_args *a, uint64_t rows) {
    return cut(kGemmLossDz, rows, a->tokens, 1, false, blocks(w->cols, kTileCols));
}
Cut cut_dx(const uzip_weight *w, const uzip_loss_args *a, uint64_t rows) {
    return cut(kGemmDx, w->cols, a->tokens, 1, false, blocks(rows, 64));
}

LossPlan plan_loss(const uzip_weight *w, const uzip_loss_args *a, bool backward, Carver &c) {
    LossPlan p{};
    p.stage = !tiled(a->x, a->x_stride, w->cols) || (backward && a->dw);  // (dw: with zeros for tokens that do not count)
    if (p.stage) p.x = c.take<uint16_t>(a->tokens * up(w->cols, 8));
    if (!backward) {
        if (a->tokens == 0) return p;
        p.cut = cut(kGemmLossStat, w->rows, a->tokens, 1, false, blocks(w->cols, kTileCols));
        p.parts = c.take<float2>(a->tokens * p.cut.r_tiles);
        p.picked = c.take<float>(a->tokens);
        if (p.cut.part()) p.part = c.take<float>(p.cut.part());
        return p;
    }
    // a piece's logit gradients take up to 128 MiB, half of what the last-level cache holds, but at least 4,096 rows
    const uint64_t fit = a->tokens ? (128ull << 20) / (2 * a->tokens) / 256 * 256 : 0;
    p.piece = std::min(up(w->rows, 256), std::max<uint64_t>(4096, fit));
    if (a->tokens == 0) return p;
    p.dz = c.take<uint16_t>(a->tokens * p.piece);
    p.unit = c.take<float>(1);
    uint64_t part = 0;
    const uint64_t all = up(w->rows, kTileRows);
    for (uint64_t r0 = 0; r0 < all; r0 += p.piece) {
        const uint64_t rows = std::min(p.piece, all - r0);
        part = std::max(part, std::max(cut_dz(w, a, rows).part(), a->dx ? cut_dx(w, a, rows).part() : 0));
    }
    if (part) p.part = c.take<float>(part);
    if (a->dx && p.piece < w->rows) p.sum = c.take<float>(a->tokens * up(w->cols, 8));
    return p;
}

// x as the products read it.
Mat loss_x(const uzip_weight *w, const uzip_loss_args *a, const LossPlan &plan) {
    return plan.stage ? Mat{plan.x, up(w->cols, 8)} : Mat{a->x, a->x_stride};
}

GemmParams loss_params(const uzip_weight *w, const uzip_loss_args *a) {
    GemmParams p{};
    p.w = view(w);
    p.groups = 1;
    p.splits = 1;
    p.tokens = (uint32_t)a->tokens;
    p.row_blocks = p.w.row_blocks;
    p.rows = (uint32_t)w->rows;
    p.cols = (uint32_t)w->cols;
    p.loss.target = a->target;
    p.loss.ignore = a->ignore_index;
    return p;
}

}  // namespace

extern "C" {

size_t uzip_weight_max_size(size_t matrices, size_t rows, size_t cols, uint32_t gated) {
    return dims_ok(matrices, rows, cols, gated) ? (size_t)weight_layout(matrices, rows, cols, gated).max_bytes : 0;
}

size_t uzip_weight_workspace_size(size_t matrices, size_t rows, size_t cols, uint32_t gated) {
    if (!dims_ok(matrices, rows, cols, gated)) return 0;
    return (size_t)(8 * blocks(weight_layout(matrices, rows, cols, gated).tiles, kScanTiles) + kAlign);
}

uzip_status uzip_weight_pack(const void *d_in, size_t matrices, size_t rows, size_t cols, size_t row_stride,
                             size_t matrix_stride, uint32_t gated, void *d_out, size_t out_capacity,
                             uint64_t *d_out_size, void *d_workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!dims_ok(matrices, rows, cols, gated) || !mat_ok(d_in, row_stride, rows, cols, 2)) return UZIP_ERR_INVALID_ARGUMENT;
    if (matrices > 1 && matrix_stride >= (1ull << 44)) return UZIP_ERR_INVALID_ARGUMENT;
    if (!d_out || !aligned(d_out, 16) || !d_out_size || !aligned(d_out_size, 8)) return UZIP_ERR_INVALID_ARGUMENT;
    if (!workspace_ok(d_workspace, workspace_bytes, uzip_weight_workspace_size(matrices, rows, cols, gated)))
        return UZIP_ERR_INVALID_ARGUMENT;
    PackParams p{};
    p.l = weight_layout(matrices, rows, cols, gated);
    if (out_capacity < p.l.max_bytes) return UZIP_ERR_CAPACITY;
    p.in = static_cast<const uint16_t *>(d_in);
    p.row_stride = row_stride;
    p.matrix_stride = matrices > 1 ? matrix_stride : 0;
    p.out = static_cast<uint8_t *>(d_out);
    p.out_size = d_out_size;
    p.sums = Carver(d_workspace).take<uint64_t>(blocks(p.l.tiles, kScanTiles));
    p.matrices = matrices;
    p.rows = rows;
    p.cols = cols;
    p.gated = gated;
    return done(launch_pack(p, stream));
}

uzip_status uzip_weight_unpack(const uzip_weight *weight, void *d_out, size_t row_stride, size_t matrix_stride,
                               hipStream_t stream) {
    if (!weight_ok(weight) || !mat_ok(d_out, row_stride, weight->rows, weight->cols, 2)) return UZIP_ERR_INVALID_ARGUMENT;
    if (weight->matrices > 1 && matrix_stride >= (1ull << 44)) return UZIP_ERR_INVALID_ARGUMENT;
    UnpackParams p{};
    p.w = view(weight);
    p.out = static_cast<uint16_t *>(d_out);
    p.row_stride = row_stride;
    p.matrix_stride = weight->matrices > 1 ? matrix_stride : 0;
    p.tiles = weight_layout(weight->matrices, weight->rows, weight->cols, weight->gated).tiles;
    p.cols = (uint32_t)weight->cols;
    return done(launch_unpack(p, stream));
}

size_t uzip_linear_workspace_size(const uzip_weight *weight, const uzip_linear_args *args) {
    if (!weight || !args || !linear_ok(weight, args, args->offsets != nullptr)) return 0;
    Carver c(nullptr);
    plan_linear(weight, args, c);
    return (size_t)c.bytes();
}

uzip_status uzip_linear(const uzip_weight *weight, const uzip_linear_args *args, void *d_workspace,
                        size_t workspace_bytes, hipStream_t stream) {
    if (!linear_ok(weight, args, false)) return UZIP_ERR_INVALID_ARGUMENT;
    return linear_run(weight, args, d_workspace, workspace_bytes, stream);
}

uzip_status uzip_grouped_linear(const uzip_weight *weight, const uzip_linear_args *args, void *d_workspace,
                                size_t workspace_bytes, hipStream_t stream) {
    if (!linear_ok(weight, args, true)) return UZIP_ERR_INVALID_ARGUMENT;
    return linear_run(weight, args, d_workspace, workspace_bytes, stream);
}

size_t uzip_linear_backward_workspace_size(const uzip_weight *weight, const uzip_linear_backward_args *args) {
    if (!weight || !args || !backward_ok(weight, args, args->offsets != nullptr)) return 0;
    Carver c(nullptr);
    plan_backward(weight, args, c);
    return (size_t)c.bytes();
}

uzip_status uzip_linear_backward(const uzip_weight *weight, const uzip_linear_backward_args *args, void *d_workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
    if (!backward_ok(weight, args, false)) return UZIP_ERR_INVALID_ARGUMENT;
    return backward_run(weight, args, d_workspace, workspace_bytes, stream);
}

uzip_status uzip_grouped_linear_backward(const uzip_weight *weight, const uzip_linear_backward_args *args,
                                         void *d_workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!backward_ok(weight, args, true)) return UZIP_ERR_INVALID_ARGUMENT;
    return backward_run(weight, args, d_workspace, workspace_bytes, stream);
}

size_t uzip_linear_cross_entropy_workspace_size(const uzip_weight *weight, const uzip_loss_args *args) {
    if (!loss_ok(weight, args, false)) return 0;
    Carver c(nullptr);
    plan_loss(weight, args, false, c);
    return (size_t)c.bytes();
}

uzip_status uzip_linear_cross_entropy(const uzip_weight *weight, const uzip_loss_args *args, void *d_workspace,
                                      size_t workspace_bytes, hipStream_t stream) {
    if (!loss_ok(weight, args, false)) return UZIP_ERR_INVALID_ARGUMENT;
    Carver c(d_workspace);
    const LossPlan plan = plan_loss(weight, args, false, c);
    if (!workspace_ok(d_workspace, workspace_bytes, c.bytes())) return UZIP_ERR_INVALID_ARGUMENT;
    if (args->tokens == 0) return UZIP_OK;
    GemmParams p = loss_params(weight, args);
    p.cmat = loss_x(weight, args, plan);
    if (plan.stage && launch_stage(static_cast<const uint16_t *>(args->x), args->x_stride, plan.x, p.cmat.stride, args->tokens,
                                   weight->cols, stream) != hipSuccess)
        return UZIP_ERR_DEVICE;
    p.c_limit = (uint32_t)up(weight->cols, 8);
    plan.cut.set(p, plan.part);
    p.steps = p.w.col_blocks;
    p.loss.parts = plan.parts;
    p.loss.picked = plan.picked;
    if (launch_gemm(kGemmLossStat, plan.cut.tile, p, stream) != hipSuccess) return UZIP_ERR_DEVICE;
    return done(launch_loss_join(p.loss, args->loss, args->lse, p.tokens, p.r_tiles, weight->rows, stream));
}

size_t uzip_linear_cross_entropy_backward_workspace_size(const uzip_weight *weight, const uzip_loss_args *args) {
    if (!loss_ok(weight, args, true)) return 0;
    Carver c(nullptr);
    plan_loss(weight, args, true, c);
    return (size_t)c.bytes();
}

uzip_status uzip_linear_cross_entropy_backward(const uzip_weight *weight, const uzip_loss_args *args,
                                               void *d_workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!loss_ok(weight, args, true)) return UZIP_ERR_INVALID_ARGUMENT;
    Carver c(d_workspace);
    const LossPlan plan = plan_loss(weight, args, true, c);
    if (!workspace_ok(d_workspace, workspace_bytes, c.bytes())) return UZIP_ERR_INVALID_ARGUMENT;
    if (!args->dx && !args->dw) return UZIP_OK;
    GemmParams p = loss_params(weight, args);
    const Mat x = loss_x(weight, args, plan);
    p.loss.lse = args->lse;
    p.loss.dloss = args->dloss;
    p.loss.dz = plan.dz;
    p.loss.dz_stride = plan.piece;
    if (args->tokens) {
        p.loss.unit = plan.unit;
        if (launch_loss_begin(p.loss, plan.unit, args->tokens, weight->rows, static_cast<const uint16_t *>(args->x),
                              args->x_stride, plan.x, x.stride, weight->cols, stream) != hipSuccess)
            return UZIP_ERR_DEVICE;
    }
    const uint32_t all = p.w.row_blocks, step = (uint32_t)(plan.piece / kTileRows);
    for (uint32_t b0 = 0; b0 < all; b0 += step) {
        p.row_block0 = b0;
        p.row_blocks = std::min(step, all - b0);
        const uint64_t rows = (uint64_t)p.row_blocks * kTileRows;
        if (args->tokens) {
            const Cut dz = cut_dz(weight, args, rows);
            dz.set(p, plan.part);
            p.cmat = x;
            p.c_limit = (uint32_t)up(weight->cols, 8);
            p.steps = p.w.col_blocks;
            if (launch_gemm(kGemmLossDz, dz.tile, p, stream) != hipSuccess) return UZIP_ERR_DEVICE;
        }
        p.cmat = Mat{plan.dz, plan.piece};
        p.c_limit = (uint32_t)up(rows, 64);  // the product above wrote zeros behind the last row
        if (args->dx && args->tokens) {
            const Cut dx = cut_dx(weight, args, rows);
            dx.set(p, plan.part);
            p.steps = (uint32_t)blocks(p.row_blocks, 4);
            p.store = StoreEpi{};
            p.store.sum = plan.sum;
            p.store.sum_stride = up(weight->cols, 8);
            p.store.unit = plan.unit;
            p.store.add = b0 > 0;
            p.store.out = b0 + step >= all ? static_cast<uint16_t *>(args->dx) : nullptr;
            p.store.stride = args->dx_stride;
            if (launch_gemm(kGemmDx, dx.tile, p, stream) != hipSuccess) return UZIP_ERR_DEVICE;
        }
        if (args->dw) {
            const GemmTile tile = gemm_tile(kGemmDw, weight->cols, rows, 1);
            p.rmat = x;
            p.r_limit = (uint32_t)up(weight->cols, 8);
            p.r_tiles = (uint32_t)blocks(weight->cols, tile.r);
            p.c_tiles = (uint32_t)blocks(rows, tile.c);
            p.store = StoreEpi{};
            p.store.out = static_cast<uint16_t *>(args->dw);
            p.store.unit = args->tokens ? plan.unit : nullptr;
            p.store.stride = weight->cols;
            if (launch_gemm(kGemmDw, tile, p, stream) != hipSuccess) return UZIP_ERR_DEVICE;
        }
    }
    return UZIP_OK;
}

}  // extern "C"
