// uzip_moe.hip -- gfx950 kernels of the router (the experts of each token,
// their weights, and the pairs of token and expert grouped by expert) with its
// gradient, and of the expert layer around the grouped products.
#include <stdint.h>

#include <type_traits>

#include <hip/hip_runtime.h>

#include "uzip_lanes.hpp"
#include "uzip_moe.hpp"
#include "uzip_tiles.hpp"

namespace uzip {
namespace {

// ---- the router -------------------------------------------------------------------

__device__ inline float logit(const void *p, uint64_t at, bool f32) {
    return f32 ? static_cast<const float *>(p)[at] : from_bf16(static_cast<const uint16_t *>(p)[at]);
}

// Unsigned keys in the order of the values; both zeros are one value.
__device__ inline uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ inline float unordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }
__device__ inline uint64_t ordered(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    return u >> 63 ? ~u : u | 1ull << 63;
}

// The limit where the maximum is infinite: all of it shares alike.
__device__ inline float exp_below(float z, float top) { return z == top ? 1.0f : expf(z - top); }
__device__ inline double sigmoid64(double z) { return 1.0 / (1.0 + exp(-z)); }

// Scores that are all below this are exp(z) in 64 bits, or less than that can
// tell; relative to the largest they are whatever the logits are (masked by
// their type's lowest value, say).
constexpr double kFaint = 1e-290;
__device__ inline double faint(bool on, float z) {
    const float top = unordered(wave_max(on ? ordered(z) : 0u));
    return on ? exp((double)z - (double)top) : 0.0;
}

// A token's choice by one wave: lane j < k gets the j-th best expert and its
// weight.  Lane l holds the scores of experts 64 i + l.  Keys are the logits,
// since softmax and sigmoid keep their order; with a bias the biased scores,
// in 64 bits, since there neighbours could change places.
template <int V, bool BIAS, class B>
__device__ inline void choose(const RouteParams &p, uint32_t t, uint32_t lane, const float (&z)[V], B bias, int32_t &expert,
                              float &weight) {
    typedef std::conditional_t<BIAS, uint64_t, uint32_t> Key;
    bool nan = false;
    Key key[V];
    double score[BIAS ? V : 1];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        nan |= z[i] != z[i];
        key[i] = 0;
        if constexpr (BIAS) {
            score[i] = sigmoid64(z[i]);
            if (z[i] > -INFINITY) {
                const double s = score[i] + (double)bias(i);
                key[i] = s > -INFINITY ? ordered(s) : 0;
            }
        } else if (z[i] > -INFINITY) {
            key[i] = ordered(z[i]);
        }
    }
    nan = __any(nan);
    expert = -1;
    float mine = 0;         // the chosen logit
    double mine_score = 0;  // its score, where it is known
    for (uint32_t j = 0; j < p.k; ++j) {
        Key best = key[0];
#pragma unroll
        for (int i = 1; i < V; ++i) best = key[i] > best ? key[i] : best;
        Key top;
        if constexpr (BIAS) {  // the upper halves, and the lower ones where more than one lane has it
            const uint32_t hi = wave_max((uint32_t)(best >> 32));
            const uint64_t m = __ballot((uint32_t)(best >> 32) == hi);
            const uint32_t lo = m & (m - 1) ? wave_max((uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u)
                                            : lane_of((uint32_t)best, (uint32_t)__ffsll((unsigned long long)m) - 1);
            top = (uint64_t)hi << 32 | lo;
        } else {
            top = wave_max(best);
        }
        if (top == 0) break;
        uint32_t e = 0xFFFFFFFFu;  // the first that has it
        double its = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint64_t m = __ballot(key[i] == top);
            if (m && e == 0xFFFFFFFFu) {
                const uint32_t l = (uint32_t)__ffsll((unsigned long long)m) - 1;
                e = i * 64 + l;
                if constexpr (BIAS) its = lane_of(score[i], l);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e == i * 64 + lane) key[i] = 0;
        if (lane == j) {
            expert = (int32_t)e;
            if constexpr (BIAS) mine_score = its;
            else mine = unordered(top);
        }
    }
    const bool on = expert >= 0;
    if (p.sigmoid) {
        // (64 bits: scores of very negative logits keep their ratio)
        double s = BIAS ? mine_score : on ? sigmoid64(mine) : 0.0;
        double all = p.renorm ? wave_sum(s) : 1.0;
        if (all < kFaint) {
            if (BIAS && on) mine = logit(p.logits, (uint64_t)t * p.stride + (uint32_t)expert, p.f32);
            s = faint(on, mine);
            all = wave_sum(s);
        }
        weight = on ? (float)(s / all * p.scale) : 0.0f;
    } else {
        float top = z[0];
#pragma unroll
        for (int i = 1; i < V; ++i) top = fmaxf(top, z[i]);
        top = unordered(wave_max(ordered(top)));
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
        const int32_t e = lane_of(was, j);
        const float x = lane_of(w, j);
        if (e != was || was < 0 || j == lane) continue;
        if (j < lane) again = true;
        else weight += x;
    }
    if (again) expert = -1;
    if (expert < 0) weight = 0;
}

// The tokens t0, t0 + step, .. before t1, the next one's logits on their way
// (up to 256 experts: more have no registers left for it).
template <int V, class F>
__device__ inline void choose_all(const RouteParams &p, uint32_t t0, uint32_t t1, uint32_t step, uint32_t lane, F keep) {
    int32_t expert;
    float weight;
    if (!p.logits) {
        for (uint32_t t = t0; t < t1; t += step) {
            given(p, t, lane, expert, weight);
            keep(t, expert, weight);
        }
        return;
    }
    constexpr bool AHEAD = V <= 4;
    float first[V], next[V];
    auto bias = [&](int i) { return AHEAD ? first[i] : p.bias[i * 64 + lane]; };  // of one that has a logit
    auto load = [&](uint32_t t) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t e = i * 64 + lane;
            next[i] = e < p.num ? logit(p.logits, (uint64_t)t * p.stride + e, p.f32) : -INFINITY;
        }
    };
#pragma unroll
    for (int i = 0; i < V; ++i) first[i] = AHEAD && p.bias && i * 64 + lane < p.num ? p.bias[i * 64 + lane] : 0.0f;
    if (AHEAD && t0 < t1) load(t0);
    for (uint32_t t = t0; t < t1; t += step) {
        float z[V];
        if (!AHEAD) load(t);
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = next[i];
        if (AHEAD && t + step < t1) load(t + step);
        if (p.bias) choose<V, true>(p, t, lane, z, bias, expert, weight);
        else choose<V, false>(p, t, lane, z, bias, expert, weight);
        keep(t, expert, weight);
    }
}

// Pairs [p0, p1) to their places: base[e] is the next one of expert e.  Waves
// take turns, 64 pairs each, so that an expert's pairs keep their order.
template <uint32_t NT>
__device__ inline void place(const RouteParams &p, uint32_t p0, uint32_t p1, uint32_t *base) {
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t bits = 1;
    while (p.num >> bits) ++bits;
    for (uint32_t r = p0; r < p1; r += NT) {
        const uint32_t pair = r + wave * 64 + lane;
        const bool on = pair < p1;
        const int32_t x = on ? p.experts[pair] : -1;
        const uint32_t e = x < 0 ? p.num : (uint32_t)x;
        uint64_t same = __ballot(on);
        for (uint32_t b = 0; b < bits; ++b) {
            const uint64_t m = __ballot(e >> b & 1);
            same &= e >> b & 1 ? m : ~m;
        }
        const uint32_t before = __popcll(same & ((1ull << lane) - 1));
        const uint32_t turns = min((p1 - r + 63) / 64, NT / 64);
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
// (PLACE), which need the counts of the chunks before.  The same pairs have the
// same places whatever the order of the workgroups.  Bound by latency where
// tokens are few (4 of 128 experts, 8 each: 5 us, a launch 2.5 of them; 777 of
// 60, 4 each: 4.5 and 4.5), by the steps of a search where they are many (16384
// of 64, 6 each, biased: 14 and 7 us, a third of the issue slots; 4.2 MB of logits).
// More than 256 experts take all 128 registers of a lane and 14 to 16 more in scratch.
template <int V, bool CHOOSE, bool PLACE, uint32_t NT>
__global__ __launch_bounds__(NT) void k_route(RouteParams p) {
    __shared__ uint32_t count[kMaxExperts + 1], base[kMaxExperts + 1], waves[NT / 64];
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t t0 = min(blockIdx.x * p.chunk, p.tokens), t1 = min(t0 + p.chunk, p.tokens);
    for (uint32_t e = threadIdx.x; e <= p.num; e += NT) count[e] = base[e] = 0;
    __syncthreads();
    if constexpr (CHOOSE) {
        choose_all<V>(p, t0 + wave, t1, NT / 64, lane, [&](uint32_t t, int32_t e, float w) {
            if (lane < p.k) {
                p.experts[(uint64_t)t * p.k + lane] = e;
                p.weights[(uint64_t)t * p.k + lane] = w;
                atomicAdd(&count[e < 0 ? p.num : (uint32_t)e], 1u);
            }
        });
        __syncthreads();
        if constexpr (!PLACE)
            for (uint32_t e = threadIdx.x; e <= p.num; e += NT) p.counts[(uint64_t)blockIdx.x * (p.num + 1) + e] = (int32_t)count[e];
    } else {
        // count: pairs of all chunks, base: of those before this one
        uint32_t wide = 1;
        while (wide < p.num + 1) wide *= 2;
        const uint32_t runs = wide < NT ? NT / wide : 1;
        for (uint32_t e = threadIdx.x & (wide - 1); e <= p.num; e += NT) {
            uint32_t all = 0, before = 0;
            for (uint32_t c0 = wide < NT ? threadIdx.x / wide : 0; c0 < p.chunks; c0 += 8 * runs) {
                uint32_t n[8];  // on their way at once
#pragma unroll
                for (uint32_t u = 0; u < 8; ++u) {
                    const uint32_t c = c0 + u * runs;
                    n[u] = c < p.chunks ? (uint32_t)p.counts[(uint64_t)c * (p.num + 1) + e] : 0;
                }
#pragma unroll
                for (uint32_t u = 0; u < 8; ++u) {
                    all += n[u];
                    before += c0 + u * runs < blockIdx.x ? n[u] : 0;
                }
            }
            atomicAdd(&count[e], all);
            atomicAdd(&base[e], before);
        }
        __syncthreads();
    }
    if constexpr (PLACE) {
        // (a thread an expert: a small workgroup has no more)
        uint32_t with;
        const uint32_t start = scan_before<NT / 64>(threadIdx.x < p.num ? count[threadIdx.x] : 0u, waves, with);
        if (threadIdx.x < p.num) {
            base[threadIdx.x] += start;
            if (blockIdx.x == 0) p.offsets[threadIdx.x] = (int32_t)start;
        }
        if (threadIdx.x == 0) {
            base[p.num] += with;
            if (blockIdx.x == 0) p.offsets[p.num] = (int32_t)with;
        }
        __syncthreads();
        place<NT>(p, t0 * p.k, t1 * p.k, base);
    }
}

// The gradient of the logits, a wave a token: dp of the chosen experts, then
// through the scores.  The choice itself has none.  Half of the issue slots are
// busy: all lanes take the exponentials and divisions of at most k experts, for
// sigmoid scores in 64 bits (16384 tokens of 64, 6 each: 10 us, softmax 8; 8.4 MB).
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
    top = unordered(wave_max(ordered(top)));
    int32_t expert = lane < p.k ? p.experts[(uint64_t)t * p.k + lane] : -1;
    if (expert >= (int32_t)p.num) expert = -1;
    const bool on = expert >= 0;
    const float g = on ? p.dweights[(uint64_t)t * p.k + lane] : 0.0f;
    float zj = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float x = __shfl(z[i], expert & 63);
        if (on && expert / 64 == i) zj = x;
    }
    // The share p_j times (g_j - the sum of p_i g_i).  Where p_j is nearly 1 that cancels; for the largest, the leading one, it
    // is p_j (g_j Q - R) with Q and R the sums of p_i and p_i g_i over the others.
    float out[V], dz;  // of the experts that are not chosen, of this lane's chosen one
    if (p.sigmoid) {
        const double t = exp(fmin(-(double)zj, 700.0));
        double s = on ? 1.0 / (1.0 + t) : 0.0, rest = t * s, d = g;  // rest: 1 - s
        if (p.renorm) {
            const uint32_t key = on ? ordered(zj) : 0;
            const uint32_t lead = (uint32_t)__ffsll((unsigned long long)__ballot(key == wave_max(key))) - 1;
            const bool leads = lane == lead;
            double q = wave_sum(leads ? 0.0 : s), all = q + lane_of(s, lead);
            if (all < kFaint) {
                s = faint(on, zj), rest = 1.0;
                q = wave_sum(leads ? 0.0 : s), all = q + lane_of(s, lead);
            }
            const double r = wave_sum(leads ? 0.0 : d * s), dot = r + lane_of(d * s, lead), inv = 1.0 / all;
            d = (leads ? (d * q - r) * inv : d - dot * inv) * inv;
        }
        dz = (float)(d * s * rest * p.scale);
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = 0;
    } else {
        const float s = on ? exp_below(zj, top) : 0.0f;
        // (of a routing of moe_route's there is one; of another perhaps none, and nothing to lead)
        const uint64_t tops = __ballot(on && zj == top);
        const uint32_t lead = tops ? (uint32_t)__ffsll((unsigned long long)tops) - 1 : 64;
        const bool leads = lane == lead;
        const uint32_t first = tops ? (uint32_t)lane_of(expert, lead) : 0xFFFFFFFFu;
        const float its = tops ? 1.0f : 0.0f, g0 = tops ? lane_of(g, lead) : 0.0f;
        float q = leads ? 0.0f : s;
        if (!p.renorm) {
            q = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) q += z[i] > -INFINITY && i * 64 + lane != first ? exp_below(z[i], top) : 0.0f;
        }
        q = wave_sum(q);
        const float inv = 1.0f / (q + its), r = wave_sum(leads ? 0.0f : g * s), dot = (r + its * g0) * inv;
        dz = (leads ? (g0 * q - r) * inv : s * (g - dot)) * inv * p.scale;
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = p.renorm || !(z[i] > -INFINITY) ? 0.0f : -exp_below(z[i], top) * inv * dot * p.scale;
    }
    if (!__any(on)) {
        dz = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = 0;
    }
    for (uint32_t j = 0; j < p.k; ++j) {
        const int32_t e = lane_of(expert, j);
        const float d = lane_of(dz, j);
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

// Pairs [begin, end) of an expert; offsets are clamped to the pairs that exist.
__device__ inline uint32_t clamped(int32_t v, uint32_t pairs) { return v < 0 ? 0u : min((uint32_t)v, pairs); }

// Whether a group holds row s, by a thread: where the offsets ascend (a wave
// finds out at once) the first and the last tell.
struct Held {
    const int32_t *offsets;
    uint32_t num, pairs, first, last;
    bool down;
};
__device__ inline Held held_rows(const int32_t *offsets, uint32_t num, uint32_t pairs) {
    Held h{offsets, num, pairs, clamped(offsets[0], pairs), clamped(offsets[num], pairs), false};
    for (uint32_t e = threadIdx.x & 63; e < num; e += 64) h.down |= clamped(offsets[e + 1], pairs) < clamped(offsets[e], pairs);
    h.down = __any(h.down);
    return h;
}
__device__ inline bool is_held(const Held &h, uint32_t s) {
    if (!h.down) return s >= h.first && s < h.last;
    bool in = false;
#pragma unroll 1
    for (uint32_t e = 0; e < h.num; ++e) in |= clamped(h.offsets[e], h.pairs) <= s && s < clamped(h.offsets[e + 1], h.pairs);
    return in;
}

// Rows of x in the order of their experts, zeros behind the last column, and the place of each pair that the order names (one
// that lies in no group has none).  Bound by the writes
// (4096 tokens of 2048, 6 of 64 experts each: 101 MB, 31 us, where the two products take 740).
__global__ __launch_bounds__(256) void k_gather(GatherParams p) {
    const uint32_t pairs = p.tokens * p.k, units = (uint32_t)(p.out_stride / 8);
    const Held held = held_rows(p.offsets, p.num, pairs);
    const uint64_t n = (uint64_t)pairs * units;
    const uint16_t *x = static_cast<const uint16_t *>(p.x.p);
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (uint64_t)gridDim.x * 256) {
        const uint32_t s = (uint32_t)(i / units), u = (uint32_t)(i % units);
        const uint32_t pair = (uint32_t)p.order[s];
        if (pair >= pairs) continue;
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
        if (is_held(held, s)) *reinterpret_cast<u32x4 *>(p.out + (uint64_t)s * p.out_stride + u * 8) = v;
        if (u == 0) p.place[pair] = is_held(held, s) ? s : pairs;
    }
}

// y of a token: its experts' results by their weights, in the order of the choice, and the residual.  For a pair that the
// order does not name nothing was written: whatever stands there, the order has another pair at that place.  Bound by the
// reads (of the above 201 MB of fp32, 36 us, 6.0 TB/s).
__global__ __launch_bounds__(256) void k_combine(CombineParams p) {
    const uint32_t pairs = p.tokens * p.k, units = (p.cols + 7) / 8;
    const uint64_t n = (uint64_t)p.tokens * units;
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (uint64_t)gridDim.x * 256) {
        const uint32_t t = (uint32_t)(i / units), c = (uint32_t)(i % units) * 8;
        const uint32_t count = min(8u, p.cols - c);
        float y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (uint32_t j = 0; j < p.k; ++j) {
            const uint32_t pair = t * p.k + j, s = p.place[pair];
            if (s >= pairs) continue;
            const bool its = (uint32_t)p.order[s] == pair;  // (on its way beside o)
            const float w = p.weights[pair];
            float o[8];
            load<8>(p.o, (uint64_t)s * p.stride + c, true, count, o);
#pragma unroll
            for (int d = 0; d < 8; ++d) y[d] += its ? w * o[d] : 0.0f;
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

// ---- the layer for few tokens ---------------------------------------------------------

// The n-th expert that has pairs, and those; none: no pairs.
struct Found {
    uint32_t expert, begin, end;
};
__device__ inline Found find_expert(const MoeParams &p, uint32_t n) {
    constexpr uint32_t AHEAD = 4;
    const uint32_t lane = threadIdx.x & 63, pairs = p.tokens * p.k;
    Found f{0, 0, 0};
    uint32_t seen = 0;
    for (uint32_t e0 = 0; e0 < p.num; e0 += 64 * AHEAD) {
        uint32_t b[AHEAD], t[AHEAD];
#pragma unroll
        for (uint32_t i = 0; i < AHEAD; ++i) {
            const uint32_t e = e0 + i * 64 + lane;
            b[i] = e < p.num ? clamped(p.offsets[e], pairs) : 0;
            t[i] = e < p.num ? clamped(p.offsets[e + 1], pairs) : 0;
        }
#pragma unroll
        for (uint32_t i = 0; i < AHEAD; ++i) {
            const uint64_t m = __ballot(t[i] > b[i]);
            const uint32_t c = __popcll(m);
            if (n >= seen && n < seen + c) {
                const uint64_t at = __ballot((m >> lane & 1) && __popcll(m & ((1ull << lane) - 1)) == n - seen);
                const uint32_t l = (uint32_t)__ffsll((unsigned long long)at) - 1;
                f.expert = e0 + i * 64 + l;
                f.begin = __builtin_amdgcn_readlane(b[i], l);
                f.end = __builtin_amdgcn_readlane(t[i], l);
                return f;
            }
            seen += c;
        }
    }
    return f;
}

// Reads at a lane's offset plus a uniform one, which costs no vector operation.
// Lanes that are to read zeros have an offset behind every buffer used here.
constexpr uint32_t kBehind = 1u << 31;
__device__ inline uint4 read16(rsrc_t r, uint32_t lane_off, uint32_t off) {
    const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, (int)lane_off, (int)off, 0);
    return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ inline uint2 read8(rsrc_t r, uint32_t lane_off, uint32_t off) {
    const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(r, (int)lane_off, (int)off, 0);
    return make_uint2(v[0], v[1]);
}

// 8 values of which `left` exist, zeros for the others.
__device__ inline uint4 read_tail(const uint16_t *from, int left) {
    if (left >= 8) return __builtin_bit_cast(uint4, *reinterpret_cast<const u32x4_any *>(from));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < 8; ++c)
        if (c < left) w[c / 2] |= (uint32_t)from[c] << (16 * (c & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A wave's tiles of one row block, kb = first, first + step, ..: from memory
// through the decoder into the matrix instructions with `columns`, one block on
// its way.  `load` reads the second operand's values of a block, `multiply`
// takes the weights'.
template <int RB>
struct TileRows {
    rsrc_t rows[RB];
    uint64_t tile0[RB];
};
template <int RB, class L, class M>
__device__ inline void stream_tiles(const WeightView &w, const TileRows<RB> &t, uint32_t first, uint32_t step, uint32_t count,
                                    uint32_t lane, L load_columns, M multiply) {
    if (count == 0) return;
    const uint32_t KB = w.col_blocks;
    Tile tile[RB];
    uint4 heads[RB];
    auto load = [&](uint32_t i) __attribute__((always_inline)) {
        const uint32_t kb = first + min(i, count - 1) * step;  // (behind the last block: that again, for nothing)
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            tile[b].sm = read16(t.rows[b], lane * 16, kb * kTileBytes);
            tile[b].code = read8(t.rows[b], kTileSm + lane * 8, kb * kTileBytes);
        }
        load_columns(kb);
    };
    for (uint32_t i0 = 0; i0 < count; i0 += 64) {
#pragma unroll
        for (int b = 0; b < RB; ++b) heads[b] = w.head[t.tile0[b] + min(first + (i0 + lane) * step, KB - 1)];
        if (i0 == 0) load(0);
#pragma unroll
        for (int b = 0; b < RB; ++b) heads[b] = head_checked(w, heads[b]);
        for (uint32_t i = i0; i < min(count, i0 + 64); ++i) {
#pragma unroll
            for (int b = 0; b < RB; ++b) {
                uint32_t v[8];
                tile[b].h.x = __builtin_amdgcn_readlane(heads[b].x, i & 63);
                tile_decode_plain(tile[b], v);
                if (tile[b].h.x & (0xFF00u | kTileZero)) {
                    tile[b].h.y = __builtin_amdgcn_readlane(heads[b].y, i & 63);
                    tile[b].h.z = __builtin_amdgcn_readlane(heads[b].z, i & 63);
                    tile[b].h.w = __builtin_amdgcn_readlane(heads[b].w, i & 63);
                    tile_decode(tile[b], w, lane, v);
                }
                multiply(b, v);
            }
            load(i + 1);
        }
    }
}

// h = weight * act(U x + bias) for the pairs of one expert: RB row blocks of U
// (gated: RB / 2, each with its up rows), NW waves that split its columns, 16 CT
// pairs at a time, whose rows of x are read where they are.  Bound by the reads
// of U (8 experts of 28672 x 4096, 16 tokens: 234 us, 6.1 TB/s of packed bytes, part of
// them from the last-level cache; 64 of 2048 x 2048: 75 us, 5.5), for a token by the
// chain from offsets to pairs to a wave's four blocks, one on its way at a time
// (8 of 1536 x 2048: 12.5 us, 3.1 TB/s).  ANY: rows of x that are not 16 bytes
// apart, or too far for 32 bits, by 64-bit addresses (13 tokens, 7 experts of 1333 x
// 1027: 12.3 us, where a copy of x before took 4.1 and the kernel 9.8).
template <int CT, int RB, bool GATED, int NW, bool ANY>
__global__ __launch_bounds__(NW * 64) void k_moe_up(MoeParams p) {
    __shared__ f32x4 part[NW][RB * CT * 64];
    const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const uint32_t q = lane >> 4, r = lane & 15, pairs = p.tokens * p.k;
    if (blockIdx.x == 0 && blockIdx.y == 0 && p.splits > 1)
        for (uint32_t i = threadIdx.x; i < p.down.row_blocks; i += NW * 64) p.arrived[i] = 0;
    const Found f = find_expert(p, blockIdx.y);
    if (f.begin == f.end) return;
    const uint32_t KB = p.up.col_blocks, n = KB > wave ? (KB + NW - 1 - wave) / NW : 0;
    TileRows<RB> t;
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        uint32_t b = GATED ? blockIdx.x * (RB / 2) + i / 2 : blockIdx.x * RB + i;
        if (b >= p.up.part_blocks) b = p.up.part_blocks - 1;  // computed and dropped
        if (GATED && (i & 1)) b += p.up.part_blocks;
        t.tile0[i] = ((uint64_t)f.expert * p.up.row_blocks + b) * KB;
        t.rows[i] = buffer(p.up.tiles + t.tile0[i] * kTileBytes, KB * kTileBytes);
    }
    const rsrc_t xb = buffer(static_cast<const uint8_t *>(p.x.p), ((p.tokens - 1) * (uint32_t)p.x.stride + p.up_cols) * 2);
    const uint32_t part_block = p.up_cols % kTileCols ? KB - 1 : KB;  // the block whose last columns x does not have
    for (uint32_t s0 = f.begin; s0 < f.end; s0 += 16 * CT) {
        const uint32_t here = min(f.end - s0, 16u * CT);
        uint32_t row[CT];
        const uint16_t *from[CT];
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const uint32_t pair = j * 16 + r < here ? (uint32_t)p.order[s0 + j * 16 + r] : pairs;
            row[j] = pair < pairs ? pair / p.k * (uint32_t)p.x.stride * 2 + q * 16 : kBehind;
            // (the first row where there is no pair: its column is computed and dropped)
            from[j] = static_cast<const uint16_t *>(p.x.p) + (pair < pairs ? pair / p.k * p.x.stride : 0) + q * 8;
        }
        f32x4 acc[RB][CT];
#pragma unroll
        for (int i = 0; i < RB; ++i)
            for (int j = 0; j < CT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
        uint4 x[CT][2];
        stream_tiles<RB>(
            p.up, t, wave, NW, n, lane,
            [&](uint32_t kb) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < CT; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if constexpr (ANY) {
                            if (j && (uint32_t)j * 16 >= here) continue;
                            const uint32_t c = kb * kTileCols + h * 32;
                            if (kb != part_block) x[j][h] = __builtin_bit_cast(uint4, *reinterpret_cast<const u32x4_any *>(from[j] + c));
                            else x[j][h] = read_tail(from[j] + c, (int)p.up_cols - (int)(c + q * 8));
                            continue;
                        }
                        const bool in = kb != part_block || part_block * kTileCols + h * 32 + q * 8 < p.up_cols;
                        if (j == 0 || (uint32_t)j * 16 < here) x[j][h] = read16(xb, in ? row[j] : kBehind, (kb * kTileCols + h * 32) * 2);
                    }
            },
            [&](int i, const uint32_t (&v)[8]) __attribute__((always_inline)) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bf16x8 a = __builtin_bit_cast(bf16x8, u32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]});
#pragma unroll
                    for (int j = 0; j < CT; ++j)
                        if (j == 0 || (uint32_t)j * 16 < here)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, x[j][h]), acc[i][j], 0, 0, 0);
                }
            });
#pragma unroll
        for (int i = 0; i < RB; ++i)
            for (int j = 0; j < CT; ++j) part[wave][(i * CT + j) * 64 + lane] = acc[i][j];
        __syncthreads();
        constexpr int STEP = GATED ? 2 : 1;
        for (uint32_t u = threadIdx.x; u < RB / STEP * CT * 64; u += NW * 64) {
            const uint32_t l = u & 63, j = (u >> 6) % CT, i = (u >> 6) / CT * STEP;
            const uint32_t slot = j * 16 + (l & 15);
            const uint32_t b = GATED ? blockIdx.x * (RB / 2) + i / 2 : blockIdx.x * RB + i;
            if (slot >= here || b >= p.up.part_blocks) continue;
            const uint32_t m = b * 16 + (l >> 4) * 4, count = m < p.h_cols ? min(p.h_cols - m, 4u) : 0;
            const uint32_t pair = (uint32_t)p.order[s0 + slot];
            const float w = pair < pairs ? p.weights[pair] : 0.0f;
            float z[STEP][4];
#pragma unroll
            for (int h = 0; h < STEP; ++h) {
                f32x4 s = part[0][((i + h) * CT + j) * 64 + l];
                for (int g = 1; g < NW; ++g) s += part[g][((i + h) * CT + j) * 64 + l];
                float bias[4] = {0, 0, 0, 0};
                if (p.up_bias && count) load<4>(p.up_bias, (uint64_t)f.expert * p.up_rows + h * p.up.part_rows + m, p.bias_f32, count, bias);
                for (int d = 0; d < 4; ++d) z[h][d] = s[d] + bias[d];
            }
            // weight times activation as the sum of two bf16 values, off by 2^-17 of it: the second product then adds
            // less than its own result's rounding (with one value the layer's error is 1.4 times that)
            float hi[4], lo[4];
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const float a = GATED ? z[0][d] * sigmoid(z[0][d]) * z[GATED ? 1 : 0][d] : activate(z[0][d], p.act);
                const float y = d < (int)count && pair < pairs ? w * a : 0.0f;
                hi[d] = from_bf16(to_bf16(y));
                lo[d] = isfinite(hi[d]) ? y - hi[d] : 0.0f;
            }
            uint16_t *out = p.h + (uint64_t)(s0 + slot) * 2 * p.h_stride + m;
            *reinterpret_cast<u32x2 *>(out) = u32x2{pack_bf16(hi[0], hi[1]), pack_bf16(hi[2], hi[3])};
            *reinterpret_cast<u32x2 *>(out + p.h_stride) = u32x2{pack_bf16(lo[0], lo[1]), pack_bf16(lo[2], lo[3])};
            if (b + 1 == p.up.part_blocks)  // zeros up to a whole block of columns
                for (uint32_t c = 16; b * 16 + c < p.h_stride; c += 16)
                    *reinterpret_cast<u32x2 *>(out + c) = *reinterpret_cast<u32x2 *>(out + p.h_stride + c) = u32x2{0, 0};
        }
        __syncthreads();
    }
}

// y = the sum over the experts of D_e h_e, as one long contraction: the blocks
// of all experts that have pairs, in a row, are dealt out in runs to the waves
// of the workgroups that share RB row blocks.  Columns 2 i and 2 i + 1 of the
// matrix instruction are the two values of pair i; an expert with more than 8 CT
// pairs comes several times.  A wave's blocks follow one another without a
// pause over the experts, DEPTH on their way (two with 8 waves, where they gain
// 2 to 5%; with 16 the registers cost as much); when it leaves an expert, it adds
// its results to its own sums of the pairs' tokens in LDS.  The waves' sums are
// added in a fixed order, and the splits' by the workgroup that comes last.
// Bound by the reads of D where experts are large (8 of 4096 x 14336, 16 tokens:
// 128 us, 5.6 TB/s of packed bytes), by the turns of the waves where they are small (64 of
// 2048 x 1024, 64 tokens: 53 us, 3.9 TB/s), for a token by a chain as above on half of the
// CUs (8 of 2048 x 768: 128 workgroups, 10.5 us).
constexpr uint32_t kMaxVisits = kMaxExperts + kFewPairs / 8;
template <int CT, int RB, int NW, int DEPTH>
__global__ __launch_bounds__(NW * 64) void k_moe_down(MoeParams p) {
    static_assert(64 % DEPTH == 0, "stages keep their turns over batches of headers");
    extern __shared__ float sums[];                 // [NW][RB][tokens][16]
    __shared__ uint32_t visits[kMaxVisits];         // expert, first pair << 10, pairs - 1 << 23
    __shared__ uint16_t token_of[kFewPairs];
    __shared__ uint32_t before[NW], last;
    constexpr uint32_t PAIRS = 8 * CT, EXPERTS = (kMaxExperts + NW * 64 - 1) / (NW * 64);
    const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const uint32_t q = lane >> 4, r = lane & 15, pairs = p.tokens * p.k, block = blockIdx.x * RB;
    const uint32_t KB = p.down.col_blocks, rows4 = RB * p.tokens * 4;
    f32x4 *const all = reinterpret_cast<f32x4 *>(sums), *const mine = all + wave * rows4;
    uint32_t first[EXPERTS], count[EXPERTS], own = 0, entries;
#pragma unroll
    for (uint32_t i = 0; i < EXPERTS; ++i) {
        const uint32_t e = threadIdx.x * EXPERTS + i;
        first[i] = e < p.num ? clamped(p.offsets[e], pairs) : 0;
        const uint32_t end = e < p.num ? clamped(p.offsets[e + 1], pairs) : 0;
        count[i] = end > first[i] ? end - first[i] : 0;
        own += (count[i] + PAIRS - 1) / PAIRS;
    }
    for (uint32_t s = threadIdx.x; s < pairs; s += NW * 64) {
        const uint32_t pair = (uint32_t)p.order[s];
        token_of[s] = (uint16_t)(pair < pairs ? pair / p.k : 0xFFFF);
    }
    for (uint32_t i = lane; i < rows4; i += 64) mine[i] = f32x4{0, 0, 0, 0};
    uint32_t at = scan_before<NW>(own, before, entries);
#pragma unroll
    for (uint32_t i = 0; i < EXPERTS; ++i)
        for (uint32_t c = 0; c < count[i]; c += PAIRS, ++at)  // (groups that overlap could be more than there is room for)
            if (at < kMaxVisits) visits[at] = (threadIdx.x * EXPERTS + i) | (first[i] + c) << 10 | (min(count[i] - c, PAIRS) - 1) << 23;
    entries = min(entries, kMaxVisits);
    __syncthreads();
    const uint32_t waves = NW * p.splits, w = blockIdx.y * NW + wave;
    const uint64_t items = (uint64_t)entries * KB;
    const uint32_t begin = uniform((uint32_t)(items * w / waves)), n = uniform((uint32_t)(items * (w + 1) / waves)) - begin;
    const rsrc_t hb = buffer(reinterpret_cast<const uint8_t *>(p.h), pairs * 4 * p.h_stride);
    uint64_t row_tile[RB];  // of expert 0 (a block behind the last: the last, computed and dropped)
#pragma unroll
    for (int i = 0; i < RB; ++i) row_tile[i] = (uint64_t)min(block + i, p.down.row_blocks - 1) * KB;
    const uint64_t expert_tiles = (uint64_t)p.down.row_blocks * KB;
    // what is loaded: an entry and its next block
    uint32_t visit = begin / KB, kb = begin % KB, coming = 0, row[CT];
    rsrc_t rows[RB];
    auto enter = [&]() __attribute__((always_inline)) {
        const uint32_t v = uniform(visits[min(visit, entries - 1)]), s0 = v >> 10 & 0x1FFF;
        coming = (v >> 23) + 1;
#pragma unroll
        for (int i = 0; i < RB; ++i)
            rows[i] = buffer(p.down.tiles + ((v & 1023) * expert_tiles + row_tile[i]) * kTileBytes, KB * kTileBytes);
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const uint32_t slot = j * 8 + r / 2;
            row[j] = slot < coming ? ((s0 + slot) * 2 + (r & 1)) * p.h_stride * 2 + q * 16 : kBehind;
        }
    };
    struct Stage {
        Tile tile[RB];
        uint4 x[CT][2];
    } stage[DEPTH];
    auto load = [&](Stage &s, uint32_t i) __attribute__((always_inline)) {
        if (kb == KB) {
            kb = 0;
            ++visit;
            enter();
        }
#pragma unroll
        for (int d = 0; d < RB; ++d) {
            s.tile[d].sm = read16(rows[d], lane * 16, kb * kTileBytes);
            s.tile[d].code = read8(rows[d], kTileSm + lane * 8, kb * kTileBytes);
        }
#pragma unroll
        for (int j = 0; j < CT; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (j == 0 || (uint32_t)j * 8 < coming) s.x[j][h] = read16(hb, row[j], (kb * kTileCols + h * 32) * 2);
        kb += i + 1 < n;  // (behind the last block: that again, for nothing)
    };
    // what is multiplied
    uint32_t done_visit = visit, done_kb = kb, have = 0, s0 = 0;
    f32x4 acc[RB][CT];
    auto start = [&]() __attribute__((always_inline)) {
        const uint32_t v = uniform(visits[min(done_visit, entries - 1)]);
        s0 = v >> 10 & 0x1FFF, have = (v >> 23) + 1;
#pragma unroll
        for (int i = 0; i < RB; ++i)
            for (int j = 0; j < CT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    };
    auto leave = [&]() __attribute__((always_inline)) {  // both values together, to the tokens' sums
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            if (j && (uint32_t)j * 8 >= have) continue;
            const uint32_t slot = j * 8 + r / 2, token = slot < have ? token_of[s0 + slot] : 0xFFFF;
            // Where the tokens ascend no two lanes add to one sum; in a program's own order, which may name an expert twice for
            // a token, pair after pair.
            const uint32_t after = moved<kRowBack + 2>(token);
            const bool ascend = __all(r >= 14 || after > min(token, 0xFFFEu));
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                f32x4 s = acc[i][j];
#pragma unroll
                for (int d = 0; d < 4; ++d) s[d] += moved<kNeighbour>(s[d]);
                const bool on = token < p.tokens && !(r & 1);
                f32x4 *to = mine + (i * p.tokens + (on ? token : 0)) * 4 + q;
                if (ascend) {
                    if (on) *to = *to + s;
                    continue;
                }
#pragma unroll 1
                for (uint32_t c = 0; c < 16; c += 2) {
                    if (on && r == c) *to = *to + s;
                    asm volatile("" ::: "memory");
                }
            }
            asm volatile("" ::: "memory");  // (what one lane has added here another may add to next)
        }
    };
    uint4 heads[RB];
    auto multiply = [&](Stage &s, uint32_t i) __attribute__((always_inline)) {
        if (done_kb == KB) {
            leave();
            done_kb = 0;
            ++done_visit;
            start();
        }
        ++done_kb;
#pragma unroll
        for (int d = 0; d < RB; ++d) {
            uint32_t v[8];
            Tile &t = s.tile[d];
            t.h.x = __builtin_amdgcn_readlane(heads[d].x, i & 63);
            tile_decode_plain(t, v);
            if (t.h.x & (0xFF00u | kTileZero)) {
                t.h.y = __builtin_amdgcn_readlane(heads[d].y, i & 63);
                t.h.z = __builtin_amdgcn_readlane(heads[d].z, i & 63);
                t.h.w = __builtin_amdgcn_readlane(heads[d].w, i & 63);
                tile_decode(t, p.down, lane, v);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bf16x8 a = __builtin_bit_cast(bf16x8, u32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]});
#pragma unroll
                for (int j = 0; j < CT; ++j)
                    if (j == 0 || (uint32_t)j * 8 < have)
                        acc[d][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, s.x[j][h]), acc[d][j], 0, 0, 0);
            }
        }
    };
    auto load_heads = [&](uint32_t i0) __attribute__((always_inline)) {
        const uint32_t item = begin + min(i0 + lane, n - 1), v = visits[item / KB];
#pragma unroll
        for (int d = 0; d < RB; ++d) heads[d] = p.down.head[(v & 1023) * expert_tiles + row_tile[d] + item % KB];
    };
    if (n) {
        start();
        enter();
        load_heads(0);  // (first: loads come back in order)
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) load(stage[u], u);
        for (uint32_t i0 = 0; i0 < n; i0 += 64) {
            if (i0) load_heads(i0);
#pragma unroll
            for (int d = 0; d < RB; ++d) heads[d] = head_checked(p.down, heads[d]);
            const uint32_t end = min(n, i0 + 64);
            for (uint32_t i = i0; i < end; i += DEPTH) {
#pragma unroll
                for (int u = 0; u < DEPTH; ++u) {
                    if (u == 0 || i + u < end) multiply(stage[u], i + u);
                    load(stage[u], i + u + DEPTH);
                }
            }
        }
        leave();
    }
    if (p.down_bias && blockIdx.y == 0) {  // each pair's by its weight
        for (uint32_t v = wave; v < entries; v += NW) {
            const uint32_t x = visits[v], first_pair = x >> 10 & 0x1FFF, pairs_here = (x >> 23) + 1;
            for (uint32_t c = 0; c < pairs_here; ++c) {
                const uint32_t token = token_of[first_pair + c];
                if (token >= p.tokens) continue;
                const float g = p.weights[p.order[first_pair + c]];
                for (uint32_t u = lane; u < RB * 16; u += 64) {
                    const uint32_t m = block * 16 + u;
                    if (m >= p.down_rows) continue;
                    const uint64_t from = (uint64_t)(x & 1023) * p.down_rows + m;
                    const float b = p.bias_f32 ? static_cast<const float *>(p.down_bias)[from] : from_bf16(static_cast<const uint16_t *>(p.down_bias)[from]);
                    reinterpret_cast<float *>(mine)[((u / 16) * p.tokens + token) * 16 + u % 16] += g * b;
                }
            }
        }
    }
    __syncthreads();
    auto finish = [&](uint32_t u, f32x4 s) {
        const uint32_t t = u / 4 % p.tokens, m = (block + u / 4 / p.tokens) * 16 + u % 4 * 4;
        if (m >= p.down_rows) return;
        const uint32_t count = min(p.down_rows - m, 4u);
        float y[4] = {s[0], s[1], s[2], s[3]};
        if (p.residual) {
            float res[4];
            uzip::load<4>(p.residual, (uint64_t)t * p.residual_stride + m, p.y_f32, count, res);
#pragma unroll
            for (int d = 0; d < 4; ++d) y[d] += res[d];
        }
        store<4>(p.y, (uint64_t)t * p.y_stride + m, p.y_f32, count, y);
    };
    float *const part = p.part + (uint64_t)blockIdx.x * rows4 * 4;  // this block's of the first split
    const uint64_t split = (uint64_t)gridDim.x * rows4 * 4;
    for (uint32_t u = threadIdx.x; u < rows4; u += NW * 64) {
        f32x4 s = all[u];
        for (uint32_t g = 1; g < NW; ++g) s += all[g * rows4 + u];
        if (p.splits == 1) {
            finish(u, s);
            continue;
        }
        // Past the L2, which the other workgroup's XCD does not share.  (With fences around plain stores, which write that
        // cache back from every wave, the kernel took 90 us more.)
        float *to = part + blockIdx.y * split + u * 4;
#pragma unroll
        for (int d = 0; d < 4; ++d) __hip_atomic_store(to + d, s[d], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (p.splits == 1) return;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // they are there
    __syncthreads();
    if (threadIdx.x == 0)
        last = __hip_atomic_fetch_add(&p.arrived[blockIdx.x], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == p.splits - 1;
    __syncthreads();
    if (!last) return;
    for (uint32_t u = threadIdx.x; u < rows4; u += NW * 64) {
        f32x4 s = f32x4{0, 0, 0, 0};
        for (uint32_t g = 0; g < p.splits; ++g)
#pragma unroll
            for (int d = 0; d < 4; ++d)
                s[d] += __hip_atomic_load(part + g * split + u * 4 + d, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        finish(u, s);
    }
}

template <int CT, int RB, int NW, int DEPTH = 1>
hipError_t moe_down(const MoeParams &p, hipStream_t s) {
    const dim3 grid((p.down.row_blocks + RB - 1) / RB, p.splits);
    k_moe_down<CT, RB, NW, DEPTH><<<grid, NW * 64, NW * RB * p.tokens * 64, s>>>(p);
    return hipGetLastError();
}

template <int CT, int RB, bool GATED, int NW>
hipError_t moe_up(const MoeParams &p, hipStream_t s) {
    const uint32_t per = GATED ? RB / 2 : RB, experts = p.num < p.tokens * p.k ? p.num : p.tokens * p.k;
    const dim3 grid((p.up.part_blocks + per - 1) / per, experts);
    if (p.x_any) k_moe_up<CT, RB, GATED, NW, true><<<grid, NW * 64, 0, s>>>(p);
    else k_moe_up<CT, RB, GATED, NW, false><<<grid, NW * 64, 0, s>>>(p);
    return hipGetLastError();
}

template <int V>
hipError_t route(const RouteParams &p, hipStream_t s) {
    if (p.chunks > 1) {
        k_route<V, true, false, 1024><<<p.chunks, 1024, 0, s>>>(p);
        k_route<V, false, true, 1024><<<p.chunks, 1024, 0, s>>>(p);
        return hipGetLastError();
    }
    if constexpr (V <= 4) {
        if (p.tokens <= 4 && p.num <= 256) {  // (any number may be grouped by V = 1)
            k_route<V, true, true, 256><<<1, 256, 0, s>>>(p);
            return hipGetLastError();
        }
    }
    k_route<V, true, true, 1024><<<1, 1024, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace

uint32_t route_chunks(uint64_t tokens) {
    if (tokens <= kRouteOnce) return 1;
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

// How many workgroups, of how many waves and row blocks, the second product
// takes.  Row blocks: one with 16 waves; two with 8, which read h once for both,
// where an expert has many pairs (in us, one and two: 64 tokens, 64 experts of 2048 x
// 1024, 8 pairs each, 58 and 53; 128 tokens, 16 of 4096 x 4096, 16 each, 159 and 116; but
// 64 of 1024 x 512, 3 each, 16.5 and 19; 8 of 4096 x 14336, 4 each, 128 and 134); 8 waves
// too where the tokens' sums fill LDS.  Splits: until there are 16 waves a CU (8
// of the others), each with 4 blocks or more (the layer with 8, 4 and 2 blocks or
// more: 64 row blocks of 192 blocks 25.7, 23.1 and 23.3 us, of 147 27.7, 25.1 and 24.0; 128
// of 192 35.7, 33.3 and 33.2, of 147 33.8, 31.4 and 31.4; 64 of 64 12.5, 12.5 and 13.3; 256 row
// blocks need none).
MoeShape moe_shape(uint64_t tokens, uint64_t pairs, uint64_t experts, uint64_t row_blocks, uint64_t col_blocks) {
    MoeShape m;
    experts = experts < pairs ? experts : pairs;
    m.rows = tokens <= 128 && pairs >= 6 * experts ? 2 : 1;
    m.waves = m.rows == 2 || tokens > 64 ? 8 : 16;
    const uint64_t n = (m.waves == 8 ? 2048 : 4096) / (m.waves * ((row_blocks + m.rows - 1) / m.rows)), most = experts * col_blocks / (4 * m.waves);
    m.splits = (uint32_t)(n < most ? n : most);
    if (m.splits == 0) m.splits = 1;
    return m;
}

// The first product.  Two row blocks a workgroup and eight waves where such
// workgroups about fill the chip, which holds two on each of 256 CUs; else four and
// four, so that x is read once for more of them.  Experts without a pair are counted
// too, and odd numbers of blocks leave a part of four idle.  The layer in us, two and
// four, every expert with pairs: gated, one token, 384 workgroups of two 20.0 and 22.7,
// 512 23.1 and 25.4, 768 32.7 and 30.9, 1024 39.7 and 37.2; 64 tokens, 512 31.9 and 33.1,
// 768 40.5 and 38.3, 2048 82.7 and 77.8; plain, one token, 512 26.1 and 28.2, 640 33.4 and 32.5.
// Sizes drawn over the whole range, some experts without: gated, 18 of 512 to 768, two
// from 7% slower to 22% faster; plain, 24 of 384 to 640, from 3% slower to 12% faster, 12
// of 640 to 768 from 7% slower to 10% faster.  With more than 16 pairs of an expert in
// sight two columns of tiles (16 each: 58 us against 72).
template <bool GATED>
hipError_t moe_up_any(const MoeParams &p, hipStream_t s) {
    const uint64_t pairs = (uint64_t)p.tokens * p.k, experts = p.num < pairs ? p.num : pairs;
    const bool wide = p.tokens > 16 && pairs > 4 * experts;
    if (GATED ? p.up.part_blocks * experts <= 768 : (p.up.part_blocks + 1) / 2 * experts <= 640)
        return wide ? moe_up<2, 2, GATED, 8>(p, s) : moe_up<1, 2, GATED, 8>(p, s);
    return wide ? moe_up<2, 4, GATED, 4>(p, s) : moe_up<1, 4, GATED, 4>(p, s);
}

hipError_t launch_moe_few(const MoeParams &p, hipStream_t s) {
    const hipError_t e = p.act == kActSwiglu ? moe_up_any<true>(p, s) : moe_up_any<false>(p, s);
    if (e != hipSuccess) return e;
    const MoeShape m = moe_shape(p.tokens, (uint64_t)p.tokens * p.k, p.num, p.down.row_blocks, p.down.col_blocks);
    if (m.rows == 2) return moe_down<2, 2, 8, 2>(p, s);
    if (m.waves == 8) return moe_down<2, 1, 8, 2>(p, s);
    return p.tokens <= 8 ? moe_down<1, 1, 16>(p, s) : moe_down<2, 1, 16>(p, s);
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
