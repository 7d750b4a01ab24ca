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
    p.chunks = route_chunks(a->tokens, a->k);
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

// Rows gathered by expert, the two grouped products, the results joined.
struct MoePlan {
    uint16_t *x, *h;
    float *o;
    uint32_t *place;
    uzip_linear_args first, second;
    size_t ws_bytes;
    uint8_t *ws;
};

MoePlan plan_moe(const uzip_weight *up, const uzip_weight *down, const uzip_moe_args *a, Carver &c) {
    MoePlan p{};
    const uint64_t pairs = a->tokens * a->k, xs = uzip::up(up->cols, 8), hs = uzip::up(down->cols, 8);
    p.x = c.take<uint16_t>(pairs * xs);
    p.h = c.take<uint16_t>(pairs * hs);
    p.o = c.take<float>(pairs * down->rows);
    p.place = c.take<uint32_t>(pairs);
    uzip_linear_args f{};
    f.tokens = pairs;
    f.offsets = a->offsets;
    f.bias_dtype = a->bias_dtype;
    f.x = p.x;
    f.x_stride = xs;
    f.bias = a->up_bias;
    f.y = p.h;
    f.y_stride = hs;
    f.y_dtype = UZIP_BF16;
    f.act = a->act;
    p.first = f;
    f.x = p.h;
    f.x_stride = hs;
    f.bias = a->down_bias;
    f.y = p.o;
    f.y_stride = down->rows;
    f.y_dtype = UZIP_FP32;
    f.act = UZIP_ACT_NONE;
    p.second = f;
    // (sizes do not depend on where the buffers are, only on their alignment)
    uint8_t *const some = reinterpret_cast<uint8_t *>(kAlign);
    for (uzip_linear_args *l : {&f, &p.first}) {
        uzip_linear_args probe = *l;
        if (!probe.x) probe.x = some;
        if (!probe.y) probe.y = some;
        p.ws_bytes = std::max(p.ws_bytes, uzip_linear_workspace_size(l == &f ? down : up, &probe));
    }
    if (p.ws_bytes) p.ws = c.take<uint8_t>(p.ws_bytes);
    return p;
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
    plan_moe(up, down, args, c);
    return (size_t)c.bytes();
}

uzip_status uzip_moe(const uzip_weight *up, const uzip_weight *down, const uzip_moe_args *args, void *d_workspace,
                     size_t workspace_bytes, hipStream_t stream) {
    if (!moe_ok(up, down, args)) return UZIP_ERR_INVALID_ARGUMENT;
    if (args->tokens == 0) return UZIP_OK;
    Carver c(d_workspace);
    const MoePlan plan = plan_moe(up, down, args, c);
    if (!workspace_ok(d_workspace, workspace_bytes, c.bytes())) return UZIP_ERR_INVALID_ARGUMENT;
    GatherParams g{};
    g.x = Mat{args->x, args->x_stride};
    g.out = plan.x;
    g.out_stride = plan.first.x_stride;
    g.cols = (uint32_t)up->cols;
    g.tokens = (uint32_t)args->tokens;
    g.k = args->k;
    g.order = args->order;
    g.ends = args->offsets + up->matrices;
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
    p.ends = g.ends;
    p.weights = args->weights;
    p.residual = args->residual;
    p.residual_stride = args->residual_stride;
    p.y = args->y;
    p.y_stride = args->y_stride;
    p.y_f32 = args->y_dtype == UZIP_FP32;
    p.tokens = g.tokens;
    p.k = args->k;
    p.cols = (uint32_t)down->rows;
    return done(launch_combine(p, stream));
}

}  // extern "C"
