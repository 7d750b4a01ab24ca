// uzip_moe_api.cpp -- the C ABI of the router and the expert layer
// (include/uzip.h): argument checks, workspace carving and launches on the
// caller's stream.  Nothing here allocates or synchronises.
#include <stdint.h>

#include <algorithm>

#include <hip/hip_runtime.h>

#include "uzip.h"
#include "uzip_args.hpp"
#include "uzip_moe.hpp"

using namespace uzip;

namespace {

constexpr uint64_t kMaxPairs = 1ull << 25;

// ---- the router -------------------------------------------------------------

bool route_common_ok(const uzip_moe_route_args *a) {
    if (!a || a->num_experts == 0 || a->num_experts > kMaxExperts || a->k == 0 || a->k > kMaxChosen) return false;
    return a->tokens <= kMaxPairs / a->k && a->scores <= UZIP_SCORES_SIGMOID && a->renormalize <= 1;
}

bool route_ok(const uzip_moe_route_args *a) {
    if (!route_common_ok(a)) return false;
    if (!a->offsets || !aligned(a->offsets, 4)) return false;
    if (a->bias && (a->scores != UZIP_SCORES_SIGMOID || !a->logits || !aligned(a->bias, 4))) return false;
    if (a->logits && (a->k > a->num_experts || !type_ok(a->logits_dtype) ||
                      !mat_ok(a->logits, a->logits_stride, a->tokens, a->num_experts, type_size(a->logits_dtype))))
        return false;
    if (a->tokens == 0) return true;
    return a->experts && aligned(a->experts, 4) && a->weights && aligned(a->weights, 4) && a->order && aligned(a->order, 4);
}

bool route_backward_ok(const uzip_moe_route_args *a) {
    if (!route_common_ok(a) || a->k > a->num_experts || !type_ok(a->logits_dtype)) return false;
    if (a->tokens == 0) return true;
    const uint32_t size = type_size(a->logits_dtype);
    return mat_ok(a->logits, a->logits_stride, a->tokens, a->num_experts, size) &&
           mat_ok(a->dlogits, a->dlogits_stride, a->tokens, a->num_experts, size) && a->experts &&
           aligned(a->experts, 4) && a->dweights && aligned(a->dweights, 4);
}

RouteParams plan_route(const uzip_moe_route_args *a, Carver &c) {
    RouteParams p{};
    p.logits = a->logits;
    p.stride = a->logits_stride;
    p.bias = a->bias;
    p.experts = a->experts;
    p.weights = a->weights;
    p.order = a->order;
    p.offsets = a->offsets;
    p.scale = a->scale;
    p.tokens = (uint32_t)a->tokens;
    p.num = a->num_experts;
    p.k = a->k;
    p.f32 = a->logits_dtype == UZIP_FP32;
    p.sigmoid = a->scores == UZIP_SCORES_SIGMOID;
    p.renorm = a->renormalize;
    p.chunks = route_chunks(a->tokens);
    p.chunk = (uint32_t)blocks(a->tokens, p.chunks);
    if (p.chunks > 1) p.counts = c.take<int32_t>((uint64_t)p.chunks * (p.num + 1));
    return p;
}

// ---- the layer --------------------------------------------------------------

bool moe_ok(const uzip_weight *up, const uzip_weight *down, const uzip_moe_args *a) {
    if (!weight_ok(up) || !weight_ok(down) || !a || down->gated) return false;
    if (up->matrices != down->matrices || up->matrices > kMaxExperts || down->cols != up->rows / (up->gated + 1)) return false;
    if (a->k == 0 || a->k > kMaxChosen || a->tokens > kMaxPairs / a->k) return false;
    if (a->act > UZIP_ACT_SWIGLU || (a->act == UZIP_ACT_SWIGLU) != (up->gated == 1) || !type_ok(a->y_dtype)) return false;
    if ((a->up_bias || a->down_bias) && !type_ok(a->bias_dtype)) return false;
    for (const void *b : {a->up_bias, a->down_bias})
        if (b && !aligned(b, type_size(a->bias_dtype))) return false;
    if (!call_ok(up, a->tokens * a->k) || !call_ok(down, a->tokens * a->k)) return false;
    if (a->tokens == 0) return true;
    if (!a->weights || !aligned(a->weights, 4) || !a->order || !aligned(a->order, 4) || !a->offsets || !aligned(a->offsets, 4))
        return false;
    const uint32_t size = type_size(a->y_dtype);
    if (a->residual && !mat_ok(a->residual, a->residual_stride, a->tokens, down->rows, size)) return false;
    return mat_ok(a->x, a->x_stride, a->tokens, up->cols, 2) && mat_ok(a->y, a->y_stride, a->tokens, down->rows, size);
}

// Few tokens: two kernels.  As for the products alone, up to 16 pairs an expert on average.
bool few(const uzip_weight *up, const uzip_weight *down, const uzip_moe_args *a) {
    const uint64_t pairs = a->tokens * a->k;
    // (the pairs' activations, two bf16 values each, are addressed with 31 bits)
    return a->tokens <= kFewTokens && pairs <= kFewPairs && pairs <= 16 * up->matrices &&
           pairs * 4 * uzip::up(down->cols, 64) < 1ull << 31;
}

MoeParams plan_few(const uzip_weight *up, const uzip_weight *down, const uzip_moe_args *a, Carver &c) {
    MoeParams p{};
    p.up = view(up);
    p.down = view(down);
    p.x = Mat{a->x, a->x_stride};
    p.x_any = !tiled(a->x, a->x_stride, up->cols);
    p.order = a->order;
    p.offsets = a->offsets;
    p.weights = a->weights;
    p.up_bias = a->up_bias;
    p.down_bias = a->down_bias;
    p.residual = a->residual;
    p.residual_stride = a->residual_stride;
    p.y = a->y;
    p.y_stride = a->y_stride;
    p.tokens = (uint32_t)a->tokens;
    p.k = a->k;
    p.num = (uint32_t)up->matrices;
    p.up_rows = (uint32_t)up->rows;
    p.up_cols = (uint32_t)up->cols;
    p.down_rows = (uint32_t)down->rows;
    p.h_cols = (uint32_t)down->cols;
    p.h_stride = (uint32_t)uzip::up(down->cols, 64);
    p.bias_f32 = a->bias_dtype == UZIP_FP32;
    p.y_f32 = a->y_dtype == UZIP_FP32;
    p.act = a->act;
    const uint64_t pairs = a->tokens * a->k;
    const MoeShape m = moe_shape(a->tokens, pairs, up->matrices, p.down.row_blocks, p.down.col_blocks);
    p.splits = m.splits;
    p.h = c.take<uint16_t>(pairs * 2 * p.h_stride);
    if (p.splits > 1) {
        p.part = c.take<float>((uint64_t)p.splits * uzip::up(p.down.row_blocks, m.rows) * a->tokens * 16);
        p.arrived = c.take<uint32_t>(p.down.row_blocks);
    }
    return p;
}

// Many: rows gathered by expert, the two grouped products, the results joined.
// The activations between them are rounded to bf16 once: as two values they would
// double the second product, which is a third of the work, and their memory.  The
// layer's error is then 0.0023 of the whole with a bf16 result (two values 0.0017,
// the result's own rounding), 0.0017 with an fp32 one (2e-6).
struct ManyPlan {
    uint16_t *x, *h;
    float *o;
    uint32_t *place;
    uzip_linear_args first, second;
    size_t ws_bytes;
    uint8_t *ws;
};

ManyPlan plan_many(const uzip_weight *up, const uzip_weight *down, const uzip_moe_args *a, Carver &c) {
    ManyPlan p{};
    const uint64_t pairs = a->tokens * a->k;
    uzip_linear_args f{};
    f.tokens = pairs;
    f.offsets = a->offsets;
    f.bias_dtype = a->bias_dtype;
    p.first = p.second = f;
    p.first.x_stride = uzip::up(up->cols, 8);
    p.first.bias = a->up_bias;
    p.first.y_stride = p.second.x_stride = uzip::up(down->cols, 8);
    p.first.y_dtype = UZIP_BF16;
    p.first.act = a->act;
    p.second.bias = a->down_bias;
    p.second.y_stride = down->rows;
    p.second.y_dtype = UZIP_FP32;
    p.x = c.take<uint16_t>(pairs * p.first.x_stride);
    p.h = c.take<uint16_t>(pairs * p.first.y_stride);
    p.o = c.take<float>(pairs * p.second.y_stride);
    p.place = c.take<uint32_t>(pairs);
    p.first.x = p.x;
    p.first.y = p.h;
    p.second.x = p.h;
    p.second.y = p.o;
    // the products' workspace: it does not depend on where the buffers are, which are all aligned
    uzip_linear_args one = p.first, two = p.second;
    void *const some = reinterpret_cast<void *>(kAlign);
    one.x = two.x = some;
    one.y = two.y = some;
    p.ws_bytes = std::max(uzip_linear_workspace_size(up, &one), uzip_linear_workspace_size(down, &two));
    if (p.ws_bytes) p.ws = c.take<uint8_t>(p.ws_bytes);
    return p;
}

uzip_status run_many(const uzip_weight *up, const uzip_weight *down, const uzip_moe_args *a, const ManyPlan &plan,
                     hipStream_t stream) {
    GatherParams g{};
    g.x = Mat{a->x, a->x_stride};
    g.out = plan.x;
    g.out_stride = plan.first.x_stride;
    g.cols = (uint32_t)up->cols;
    g.tokens = (uint32_t)a->tokens;
    g.k = a->k;
    g.num = (uint32_t)up->matrices;
    g.order = a->order;
    g.offsets = a->offsets;
    g.place = plan.place;
    if (launch_gather(g, stream) != hipSuccess) return UZIP_ERR_DEVICE;
    uzip_status st = uzip_grouped_linear(up, &plan.first, plan.ws, plan.ws_bytes, stream);
    if (st != UZIP_OK) return st;
    st = uzip_grouped_linear(down, &plan.second, plan.ws, plan.ws_bytes, stream);
    if (st != UZIP_OK) return st;
    CombineParams p{};
    p.o = plan.o;
    p.stride = plan.second.y_stride;
    p.place = plan.place;
    p.order = a->order;
    p.weights = a->weights;
    p.residual = a->residual;
    p.residual_stride = a->residual_stride;
    p.y = a->y;
    p.y_stride = a->y_stride;
    p.y_f32 = a->y_dtype == UZIP_FP32;
    p.tokens = g.tokens;
    p.k = a->k;
    p.cols = (uint32_t)down->rows;
    return done(launch_combine(p, stream));
}

}  // namespace

extern "C" {

size_t uzip_moe_route_workspace_size(const uzip_moe_route_args *args) {
    if (!route_ok(args) || args->tokens == 0) return 0;
    Carver c(nullptr);
    plan_route(args, c);
    return (size_t)c.bytes();
}

uzip_status uzip_moe_route(const uzip_moe_route_args *args, void *d_workspace, size_t workspace_bytes,
                           hipStream_t stream) {
    if (!route_ok(args)) return UZIP_ERR_INVALID_ARGUMENT;
    Carver c(d_workspace);
    const RouteParams p = plan_route(args, c);
    if (!workspace_ok(d_workspace, workspace_bytes, c.bytes())) return UZIP_ERR_INVALID_ARGUMENT;
    return done(launch_route(p, stream));
}

uzip_status uzip_moe_route_backward(const uzip_moe_route_args *args, hipStream_t stream) {
    if (!route_backward_ok(args)) return UZIP_ERR_INVALID_ARGUMENT;
    RouteBackwardParams p{};
    p.logits = args->logits;
    p.stride = args->logits_stride;
    p.experts = args->experts;
    p.dweights = args->dweights;
    p.dlogits = args->dlogits;
    p.d_stride = args->dlogits_stride;
    p.scale = args->scale;
    p.tokens = (uint32_t)args->tokens;
    p.num = args->num_experts;
    p.k = args->k;
    p.f32 = args->logits_dtype == UZIP_FP32;
    p.sigmoid = args->scores == UZIP_SCORES_SIGMOID;
    p.renorm = args->renormalize;
    return done(launch_route_backward(p, stream));
}

size_t uzip_moe_workspace_size(const uzip_weight *up, const uzip_weight *down, const uzip_moe_args *args) {
    if (!moe_ok(up, down, args) || args->tokens == 0) return 0;
    Carver c(nullptr);
    if (few(up, down, args)) plan_few(up, down, args, c);
    else plan_many(up, down, args, c);
    return (size_t)c.bytes();
}

uzip_status uzip_moe(const uzip_weight *up, const uzip_weight *down, const uzip_moe_args *args, void *d_workspace,
                     size_t workspace_bytes, hipStream_t stream) {
    if (!moe_ok(up, down, args)) return UZIP_ERR_INVALID_ARGUMENT;
    if (args->tokens == 0) return UZIP_OK;
    Carver c(d_workspace);
    if (!few(up, down, args)) {
        const ManyPlan plan = plan_many(up, down, args, c);
        if (!workspace_ok(d_workspace, workspace_bytes, c.bytes())) return UZIP_ERR_INVALID_ARGUMENT;
        return run_many(up, down, args, plan, stream);
    }
    const MoeParams p = plan_few(up, down, args, c);
    if (!workspace_ok(d_workspace, workspace_bytes, c.bytes())) return UZIP_ERR_INVALID_ARGUMENT;
    return done(launch_moe_few(p, stream));
}

}  // extern "C"
