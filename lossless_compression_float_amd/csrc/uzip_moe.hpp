// uzip_moe.hpp -- kernel parameter blocks and launchers of the router and the
// expert layer (internal).
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

#include "uzip_linear.hpp"

namespace uzip {

constexpr uint32_t kMaxExperts = 1024;  // a wave holds a token's scores, 16 a lane
constexpr uint32_t kMaxChosen = 64;     // and its choice, one a lane
constexpr uint32_t kRouteChunks = 256;
constexpr uint32_t kRouteOnce = 32;  // tokens that one workgroup routes

struct RouteParams {
    const void *logits;  // null: experts and weights are given, and only grouped
    uint64_t stride;
    const float *bias;
    int32_t *experts;
    float *weights;
    int32_t *order, *offsets;
    int32_t *counts;  // [chunks][num + 1]: pairs of each expert, then those of none
    float scale;
    uint32_t tokens, num, k, f32, sigmoid, renorm;
    uint32_t chunk, chunks;  // tokens of a workgroup
};

struct RouteBackwardParams {
    const void *logits;
    uint64_t stride;
    const int32_t *experts;
    const float *dweights;
    void *dlogits;
    uint64_t d_stride;
    float scale;
    uint32_t tokens, num, k, f32, sigmoid, renorm;
};

// The layer with rows gathered by expert.
struct GatherParams {
    Mat x;
    uint16_t *out;         // [pairs][out_stride]
    uint64_t out_stride;
    uint32_t cols, tokens, k, num;
    const int32_t *order, *offsets;
    uint32_t *place;       // of each pair that the order names
};

struct CombineParams {
    const float *o;        // [pairs][stride]
    uint64_t stride;
    const uint32_t *place;
    const int32_t *order;
    const float *weights;
    const void *residual;
    uint64_t residual_stride;
    void *y;
    uint64_t y_stride;
    uint32_t y_f32, tokens, k, cols;
};

// The layer for few tokens, in two kernels.
struct MoeParams {
    WeightView up, down;
    Mat x;
    const int32_t *order, *offsets;
    const float *weights;
    const void *up_bias, *down_bias, *residual;
    uint64_t residual_stride;
    uint16_t *h;          // [pairs][2][h_stride]: activation times weight as the sum of two bf16 values
    float *part;          // [splits][row blocks of down][tokens][16], with more than one split
    uint32_t *arrived;    // [row blocks of down]
    void *y;
    uint64_t y_stride;
    uint32_t tokens, k, num;
    uint32_t up_rows, up_cols, down_rows, h_cols, h_stride;
    uint32_t bias_f32, y_f32, act, splits;
    uint32_t x_any;       // x's rows are not 16 bytes apart, or too far for 32 bits
};
constexpr uint32_t kFewTokens = 256, kFewPairs = 4096;

hipError_t launch_moe_few(const MoeParams &p, hipStream_t s);
struct MoeShape {
    uint32_t rows, waves, splits;  // row blocks and waves of a workgroup, workgroups that share them
};
MoeShape moe_shape(uint64_t tokens, uint64_t pairs, uint64_t experts, uint64_t row_blocks, uint64_t col_blocks);
hipError_t launch_route(const RouteParams &p, hipStream_t s);
uint32_t route_chunks(uint64_t tokens);
hipError_t launch_route_backward(const RouteBackwardParams &p, hipStream_t s);
hipError_t launch_gather(const GatherParams &p, hipStream_t s);
hipError_t launch_combine(const CombineParams &p, hipStream_t s);

}  // namespace uzip
