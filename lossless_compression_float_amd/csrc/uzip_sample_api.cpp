// uzip_sample_api.cpp -- the C ABI of the sampler (include/uzip.h): argument
// checks and launches on the caller's stream.  Nothing here allocates or
// synchronises.
#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "uzip.h"
#include "uzip_args.hpp"
#include "uzip_sample.hpp"

using namespace uzip;

namespace {

constexpr uint64_t kMaxRows = 1ull << 21;
constexpr uint64_t kMaxSegments = 1ull << 24;  // of a call

bool sample_ok(const uzip_sample_args *a) {
    if (!a || a->rows > kMaxRows || a->vocab == 0 || a->vocab > kMaxVocab || !type_ok(a->logits_dtype) || a->u_double > 1)
        return false;
    if (a->rows * blocks(a->vocab, kSegment) > kMaxSegments) return false;
    if (!a->temperature && !(a->temperature_all >= 0 && a->temperature_all < INFINITY)) return false;
    if ((!a->top_p && a->top_p_all != a->top_p_all) || (!a->min_p && a->min_p_all != a->min_p_all)) return false;
    for (const void *p : {(const void *)a->temperature, (const void *)a->top_k, (const void *)a->top_p, (const void *)a->min_p,
                          (const void *)a->logprob})
        if (p && !aligned(p, 4)) return false;
    if (a->rows == 0) return true;
    return mat_ok(a->logits, a->logits_stride, a->rows, a->vocab, type_size(a->logits_dtype)) && a->u &&
           aligned(a->u, a->u_double ? 8 : 4) && a->token && aligned(a->token, 8);
}

SampleParams plan(const uzip_sample_args *a, Carver &c) {
    SampleParams p{};
    p.logits = a->logits;
    p.stride = a->logits_stride;
    p.u = a->u;
    p.temperature = a->temperature;
    p.top_k = a->top_k;
    p.top_p = a->top_p;
    p.min_p = a->min_p;
    p.temperature_all = a->temperature_all;
    p.top_k_all = a->top_k_all;
    p.top_p_all = a->top_p_all;
    p.min_p_all = a->min_p_all;
    p.token = a->token;
    p.logprob = a->logprob;
    p.rows = (uint32_t)a->rows;
    p.vocab = (uint32_t)a->vocab;
    p.f32 = a->logits_dtype == UZIP_FP32;
    p.u_f64 = a->u_double;
    p.segments = (uint32_t)blocks(a->vocab, kSegment);
    p.segment = c.take<Segment>(a->rows * p.segments);
    p.groups = c.take<float>(a->rows * p.segments * (kSegment / kGroup));
    return p;
}

}  // namespace

extern "C" {

size_t uzip_sample_workspace_size(const uzip_sample_args *args) {
    if (!sample_ok(args) || args->rows == 0) return 0;
    Carver c(nullptr);
    plan(args, c);
    return (size_t)c.bytes();
}

uzip_status uzip_sample(const uzip_sample_args *args, void *d_workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!sample_ok(args)) return UZIP_ERR_INVALID_ARGUMENT;
    if (args->rows == 0) return UZIP_OK;
    Carver c(d_workspace);
    const SampleParams p = plan(args, c);
    if (!workspace_ok(d_workspace, workspace_bytes, c.bytes())) return UZIP_ERR_INVALID_ARGUMENT;
    return done(launch_sample(p, stream));
}

}  // extern "C"
