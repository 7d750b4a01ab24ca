// uzip_sample.hpp -- kernel parameters and launchers of the sampler (internal).
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

namespace uzip {

constexpr uint64_t kMaxVocab = 1ull << 22;
constexpr uint32_t kSegment = 2048;  // tokens that a wave surveys
constexpr uint32_t kGroup = 16;      // tokens of a lane in half a segment

// Of a segment: the sum of its weights relative to its largest value (NaN if
// it holds one), that value, and its smallest.
struct Segment {
    double sum;
    float top, low;
};

struct SampleParams {
    const void *logits;
    uint64_t stride;
    const void *u;
    const float *temperature, *top_p, *min_p;  // of each row, or null: the value below
    const int32_t *top_k;
    float temperature_all, top_p_all, min_p_all;
    int32_t top_k_all;
    int64_t *token;
    float *logprob;  // or null
    Segment *segment;    // workspace: [rows][segments]
    float *groups;       // workspace: the largest value of each group, [rows][segments][2][64]
    uint32_t rows, vocab, segments, f32, u_f64;
};

hipError_t launch_sample(const SampleParams &p, hipStream_t s);

}  // namespace uzip
