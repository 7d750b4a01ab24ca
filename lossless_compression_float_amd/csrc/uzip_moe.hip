// uzip_moe.hip -- gfx950 kernels of the router (the experts of each token,
// their weights, and the pairs of token and expert grouped by expert) with its
// gradient, and of the expert layer around the grouped products.
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "uzip_moe.hpp"
#include "uzip_tiles.hpp"

namespace uzip {
namespace {

// ---- the router -------------------------------------------------------------------

__device__ inline float logit(const void *p, uint64_t at, bool f32) {
    return f32 ? static_cast<const float *>(p)[at] : from_bf16(static_cast<const uint16_t *>(p)[at]);
}

// Unsigned keys in the order of the values.
__device__ inline uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ inline float unordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }
__device__ inline uint64_t ordered(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    return u >> 63 ? ~u : u | 1ull << 63;
}

__device__ inline uint64_t wave_max(uint64_t v) {
    for (int d = 1; d < 64; d <<= 1) {
        const uint64_t o = __shfl_xor((unsigned long long)v, d);
        v = o > v ? o : v;
    }
    return v;
}
__device__ inline uint32_t wave_min(uint32_t v) {
    for (int d = 1; d < 64; d <<= 1) v = min(v, (uint32_t)__shfl_xor((int)v, d));
    return v;
}
template <class T>
__device__ inline T wave_sum(T v) {
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

// The limit where the maximum is infinite: all of it shares alike.
__device__ inline float exp_below(float z, float top) { return z == top ? 1.0f : expf(z - top); }
__device__ inline double sigmoid64(double z) { return 1.0 / (1.0 + exp(-z)); }

// A token's choice by one wave: lane j < k gets the j-th best expert and its
// weight.  Lane l holds the scores of experts 64 i + l.  Keys are the logits,
// since softmax and sigmoid keep their order; with a bias the biased scores,
// in 64 bits, since there neighbours could change places.
template <int V, bool BIAS>
__device__ inline void choose(const RouteParams &p, uint32_t t, uint32_t lane, int32_t &expert, float &weight) {
    float z[V];
    bool nan = false;
    uint64_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t e = i * 64 + lane;
        z[i] = e < p.num ? logit(p.logits, (uint64_t)t * p.stride + e, p.f32) : -INFINITY;
        nan |= z[i] != z[i];
        const bool out = !(z[i] > -INFINITY);
        if constexpr (BIAS) {
            const double s = out ? -INFINITY : sigmoid64(z[i]) + (double)p.bias[e];
            key[i] = s > -INFINITY ? ordered(s) : 0;
        } else {
            key[i] = out ? 0 : (uint64_t)ordered(z[i]) << 32 | (0xFFFFFFFFu - e);
        }
    }
    nan = __any(nan);
    expert = -1;
    float mine = 0;
    for (uint32_t j = 0; j < p.k; ++j) {
        uint64_t best = 0;
        uint32_t at = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i] > best) best = key[i], at = i * 64 + lane;
        const uint64_t top = wave_max(best);
        if (top == 0) break;
        uint32_t e;
        if constexpr (BIAS)
            e = wave_min(best == top ? at : 0xFFFFFFFFu);
        else
            e = 0xFFFFFFFFu - (uint32_t)top;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e == i * 64 + lane) key[i] = 0;
        if (lane == j) {
            expert = (int32_t)e;
            if constexpr (BIAS)
                mine = logit(p.logits, (uint64_t)t * p.stride + e, p.f32);
            else
                mine = unordered((uint32_t)(top >> 32));
        }
    }
    const bool on = expert >= 0;
    if (p.sigmoid) {
        // (64 bits: scores of very negative logits keep their ratio)
        const double s = on ? sigmoid64(mine) : 0.0;
        const double all = p.renorm ? wave_sum(s) : 1.0;
        weight = on ? (float)(s / all * p.scale) : 0.0f;
    } else {
        float top = z[0];
#pragma unroll
        for (int i = 1; i < V; ++i) top = fmaxf(top, z[i]);
        for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
        const float s = on ? exp_below(mine, top) : 0.0f;
        float all = s;
        if (!p.renorm) {
            all = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) all += z[i] > -INFINITY ? exp_below(z[i], top) : 0.0f;
        }
        all = wave_sum(all);
        weight = on ? s / all * p.scale : 0.0f;
    }
    if (nan && on) weight = __builtin_nanf("");
}

// The same for a choice that is given: an expert that does not exist is none,
// one that is named again adds its weight to the first.
__device__ inline void given(const RouteParams &p, uint32_t t, uint32_t lane, int32_t &expert, float &weight) {
    expert = lane < p.k ? p.experts[(uint64_t)t * p.k + lane] : -1;
    weight = lane < p.k ? p.weights[(uint64_t)t * p.k + lane] : 0.0f;
    if (expert < 0 || expert >= (int32_t)p.num) expert = -1;
    bool again = false;
    const int32_t was = expert;
    const float w = weight;
    for (uint32_t j = 0; j < p.k; ++j) {
        const int32_t e = __shfl(was, j);
        const float x = __shfl(w, j);
        if (e != was || was < 0 || j == lane) continue;
        if (j < lane) again = true;
        else weight += x;
    }
    if (again) expert = -1;
    if (expert < 0) weight = 0;
}

template <int V>
__device__ inline void choose_any(const RouteParams &p, uint32_t t, uint32_t lane, int32_t &expert, float &weight) {
    if (!p.logits) given(p, t, lane, expert, weight);
    else if (p.bias) choose<V, true>(p, t, lane, expert, weight);
    else choose<V, false>(p, t, lane, expert, weight);
}

// Exclusive prefix of a workgroup's 1,024 values.
__device__ inline uint32_t scan1024(uint32_t v, uint32_t *lds) {
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t x = v;
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t y = __shfl_up(x, d);
        if (lane >= (uint32_t)d) x += y;
    }
    if (lane == 63) lds[wave] = x;
    __syncthreads();
    uint32_t before = 0;
    for (uint32_t i = 0; i < wave; ++i) before += lds[i];
    return before + x - v;
}

// Pairs [p0, p1) to their places: base[e] is the next one of expert e.  Waves
// take turns, 64 pairs each, so that an expert's pairs keep their order.
template <class E>
__device__ inline void place(const RouteParams &p, E expert_of, uint32_t p0, uint32_t p1, uint32_t *base) {
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t bits = 1;
    while (p.num >> bits) ++bits;
    for (uint32_t r = p0; r < p1; r += 1024) {
        const uint32_t pair = r + wave * 64 + lane;
        const bool on = pair < p1;
        const int32_t x = on ? expert_of(pair) : -1;
        const uint32_t e = x < 0 ? p.num : (uint32_t)x;
        uint64_t same = __ballot(on);
        for (uint32_t b = 0; b < bits; ++b) {
            const uint64_t m = __ballot(e >> b & 1);
            same &= e >> b & 1 ? m : ~m;
        }
        const uint32_t before = __popcll(same & ((1ull << lane) - 1));
        const uint32_t turns = min((p1 - r + 63) / 64, 16u);
        for (uint32_t turn = 0; turn < turns; ++turn) {
            if (turn == wave && on) {
                const uint32_t at = base[e];
                p.order[at + before] = (int32_t)pair;
                if (before == 0) base[e] = at + __popcll(same);
            }
            __syncthreads();
        }
    }
}

// Few pairs, or one chunk of many: choice and counts (CHOOSE), then the places
// (PLACE), which need the counts of the chunks before.
template <int V, bool CHOOSE, bool PLACE>
__global__ __launch_bounds__(1024) void k_route(RouteParams p) {
    __shared__ uint32_t count[kMaxExperts + 1], base[kMaxExperts + 1], lds[16];
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t t0 = min(blockIdx.x * p.chunk, p.tokens), t1 = min(t0 + p.chunk, p.tokens);
    for (uint32_t e = threadIdx.x; e <= p.num; e += 1024) count[e] = base[e] = 0;
    __syncthreads();
    if constexpr (CHOOSE) {
        for (uint32_t t = t0 + wave; t < t1; t += 16) {
            int32_t e;
            float w;
            choose_any<V>(p, t, lane, e, w);
            if (lane < p.k) {
                p.experts[(uint64_t)t * p.k + lane] = e;
                p.weights[(uint64_t)t * p.k + lane] = w;
                atomicAdd(&count[e < 0 ? p.num : (uint32_t)e], 1u);
            }
        }
        __syncthreads();
        if constexpr (!PLACE)
            for (uint32_t e = threadIdx.x; e <= p.num; e += 1024) p.counts[(uint64_t)blockIdx.x * (p.num + 1) + e] = (int32_t)count[e];
    } else {
        // count: pairs of all chunks, base: of those before this one
        uint32_t wide = 1;
        while (wide < p.num + 1) wide *= 2;
        const uint32_t runs = wide < 1024 ? 1024 / wide : 1;
        for (uint32_t e = threadIdx.x & (wide - 1); e <= p.num; e += 1024) {
            uint32_t all = 0, before = 0;
            for (uint32_t c = wide < 1024 ? threadIdx.x / wide : 0; c < p.chunks; c += runs) {
                const uint32_t n = (uint32_t)p.counts[(uint64_t)c * (p.num + 1) + e];
                all += n;
                before += c < blockIdx.x ? n : 0;
            }
            atomicAdd(&count[e], all);
            atomicAdd(&base[e], before);
        }
        __syncthreads();
    }
    if constexpr (PLACE) {
        const uint32_t start = scan1024(threadIdx.x < p.num ? count[threadIdx.x] : 0, lds);
        if (threadIdx.x < p.num) {
            base[threadIdx.x] += start;
            if (blockIdx.x == 0) p.offsets[threadIdx.x] = (int32_t)start;
        }
        const uint32_t none = p.tokens * p.k - count[p.num];
        if (threadIdx.x == 0) {
            base[p.num] += none;
            if (blockIdx.x == 0) p.offsets[p.num] = (int32_t)none;
        }
        __syncthreads();
        const int32_t *experts = p.experts;
        place(p, [=](uint32_t pair) { return experts[pair]; }, t0 * p.k, t1 * p.k, base);
    }
}

// The gradient of the logits, a wave a token: dp of the chosen experts, then
// through the scores.  The choice itself has none.
template <int V>
__global__ __launch_bounds__(256) void k_route_backward(RouteBackwardParams p) {
    const uint32_t lane = threadIdx.x & 63, t = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= p.tokens) return;
    float z[V];
    float top = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t e = i * 64 + lane;
        z[i] = e < p.num ? logit(p.logits, (uint64_t)t * p.stride + e, p.f32) : -INFINITY;
        nan |= z[i] != z[i];
        top = fmaxf(top, z[i]);
    }
    nan = __any(nan);
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    int32_t expert = lane < p.k ? p.experts[(uint64_t)t * p.k + lane] : -1;
    if (expert >= (int32_t)p.num) expert = -1;
    const bool on = expert >= 0;
    const float g = on ? p.dweights[(uint64_t)t * p.k + lane] * p.scale : 0.0f;
    const float zj = on ? logit(p.logits, (uint64_t)t * p.stride + expert, p.f32) : -INFINITY;
    float out[V], dz;  // of the experts that are not chosen, of this lane's chosen one
    if (p.sigmoid) {
        const double s = on ? sigmoid64(zj) : 0.0, rest = on ? sigmoid64(-zj) : 0.0;
        double d = g;
        if (p.renorm) {
            const double all = wave_sum(s);
            d = (d - wave_sum(d * s) / all) / all;
        }
        dz = (float)(d * s * rest);
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = 0;
    } else {
        const float s = on ? exp_below(zj, top) : 0.0f;
        float all = s;
        if (!p.renorm) {
            all = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) all += z[i] > -INFINITY ? exp_below(z[i], top) : 0.0f;
        }
        all = wave_sum(all);
        const float dot = wave_sum(g * s) / all;
        dz = s / all * (g - dot);
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = p.renorm || !(z[i] > -INFINITY) ? 0.0f : -exp_below(z[i], top) / all * dot;
    }
    if (!__any(on)) {
        dz = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = 0;
    }
    for (uint32_t j = 0; j < p.k; ++j) {
        const int32_t e = __shfl(expert, j);
        const float d = __shfl(dz, j);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e == (int32_t)(i * 64 + lane)) out[i] = d;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t e = i * 64 + lane;
        if (e >= p.num) continue;
        const float v = nan ? __builtin_nanf("") : out[i];
        if (p.f32) static_cast<float *>(p.dlogits)[(uint64_t)t * p.d_stride + e] = v;
        else static_cast<uint16_t *>(p.dlogits)[(uint64_t)t * p.d_stride + e] = to_bf16(v);
    }
}

// ---- the layer around grouped products ----------------------------------------------

// Rows of x in the order of their experts, zeros behind the last column, and the place of each pair.
__global__ __launch_bounds__(256) void k_gather(GatherParams p) {
    const uint32_t pairs = p.tokens * p.k, units = (uint32_t)(p.out_stride / 8);
    const uint32_t end = (uint32_t)min(max(*p.ends, 0), (int32_t)pairs);
    const uint64_t n = (uint64_t)pairs * units;
    const uint16_t *x = static_cast<const uint16_t *>(p.x.p);
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (uint64_t)gridDim.x * 256) {
        const uint32_t s = (uint32_t)(i / units), u = (uint32_t)(i % units);
        const uint32_t pair = (uint32_t)p.order[s];
        if (pair >= pairs) continue;
        if (u == 0) p.place[pair] = s;
        if (s >= end) continue;
        const uint16_t *row = x + (uint64_t)(pair / p.k) * p.x.stride;
        u32x4 v;
        if ((u + 1) * 8 <= p.cols) {
            v = *reinterpret_cast<const u32x4_any *>(row + u * 8);
        } else {
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (uint32_t c = 0; c < 8; ++c)
                if (u * 8 + c < p.cols) w[c / 2] |= (uint32_t)row[u * 8 + c] << (16 * (c & 1));
            v = u32x4{w[0], w[1], w[2], w[3]};
        }
        *reinterpret_cast<u32x4 *>(p.out + (uint64_t)s * p.out_stride + u * 8) = v;
    }
}

// y of a token: its experts' results by their weights, in the order of the choice, and the residual.
__global__ __launch_bounds__(256) void k_combine(CombineParams p) {
    const uint32_t pairs = p.tokens * p.k, units = (p.cols + 7) / 8;
    const uint32_t end = (uint32_t)min(max(*p.ends, 0), (int32_t)pairs);
    const uint64_t n = (uint64_t)p.tokens * units;
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (uint64_t)gridDim.x * 256) {
        const uint32_t t = (uint32_t)(i / units), c = (uint32_t)(i % units) * 8;
        const uint32_t count = min(8u, p.cols - c);
        float y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (uint32_t j = 0; j < p.k; ++j) {
            const uint32_t s = p.place[(uint64_t)t * p.k + j];
            if (s >= end) continue;
            const float w = p.weights[(uint64_t)t * p.k + j];
            float o[8];
            load<8>(p.o, (uint64_t)s * p.stride + c, true, count, o);
#pragma unroll
            for (int d = 0; d < 8; ++d) y[d] += w * o[d];
        }
        if (p.residual) {
            float r[8];
            load<8>(p.residual, (uint64_t)t * p.residual_stride + c, p.y_f32, count, r);
#pragma unroll
            for (int d = 0; d < 8; ++d) y[d] += r[d];
        }
        store<8>(p.y, (uint64_t)t * p.y_stride + c, p.y_f32, count, y);
    }
}

template <int V>
hipError_t route(const RouteParams &p, hipStream_t s) {
    if (p.chunks == 1) {
        k_route<V, true, true><<<1, 1024, 0, s>>>(p);
        return hipGetLastError();
    }
    k_route<V, true, false><<<p.chunks, 1024, 0, s>>>(p);
    k_route<V, false, true><<<p.chunks, 1024, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace

uint32_t route_chunks(uint64_t tokens, uint64_t k) {
    (void)k;
    if (tokens <= 64) return 1;
    const uint64_t n = (tokens + 15) / 16;  // a token a wave
    return (uint32_t)(n < kRouteChunks ? n : kRouteChunks);
}

hipError_t launch_route(const RouteParams &p, hipStream_t s) {
    if (!p.logits || p.num <= 64) return route<1>(p, s);
    if (p.num <= 128) return route<2>(p, s);
    if (p.num <= 256) return route<4>(p, s);
    return route<16>(p, s);
}

hipError_t launch_route_backward(const RouteBackwardParams &p, hipStream_t s) {
    const uint32_t wgs = (p.tokens + 3) / 4;
    if (wgs == 0) return hipSuccess;
    if (p.num <= 64) k_route_backward<1><<<wgs, 256, 0, s>>>(p);
    else if (p.num <= 128) k_route_backward<2><<<wgs, 256, 0, s>>>(p);
    else if (p.num <= 256) k_route_backward<4><<<wgs, 256, 0, s>>>(p);
    else k_route_backward<16><<<wgs, 256, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_gather(const GatherParams &p, hipStream_t s) {
    const uint64_t wgs = ((uint64_t)p.tokens * p.k * (p.out_stride / 8) + 255) / 256;
    k_gather<<<(uint32_t)(wgs < 8192 ? wgs : 8192), 256, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_combine(const CombineParams &p, hipStream_t s) {
    const uint64_t wgs = ((uint64_t)p.tokens * ((p.cols + 7) / 8) + 255) / 256;
    k_combine<<<(uint32_t)(wgs < 8192 ? wgs : 8192), 256, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace uzip
