// uzip_sample.hpp -- kernel parameters and launchers of the sampler (internal).
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

namespace uzip {

constexpr uint64_t kMaxVocab = 1ull << 22;

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
    uint32_t rows, vocab, f32, u_f64;
};

hipError_t launch_sample(const SampleParams &p, hipStream_t s);

}  // namespace uzip
