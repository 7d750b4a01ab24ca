// uzip_sample.hip -- gfx950 kernels of the sampler: a token a row from logits,
// with temperature, top-k, top-p and min-p, from given random numbers.
//
// With e_i = exp((z_i - max) / temperature) and the tokens in the order of
// (z descending, index ascending), each filter keeps a prefix: the first k; the
// shortest whose sum reaches p of the sum left by top-k; those with e >= min_p.
// The kept set is the shortest of them, so it is told by one key: all tokens
// above it, and the first few (by index) of those equal to it.  The draw is the
// first kept token, by index, whose running sum exceeds u times the kept sum.
//
// e is computed in 64 bits, since every neighbour in a running sum is a border
// that fp32's error moves (128,256 even tokens, off by 1e-7 of the whole each,
// would change one draw in a hundred); histograms are summed in fixed point, so
// that the order of their atomics is no matter.
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "uzip_sample.hpp"

namespace uzip {
namespace {

constexpr uint32_t kThreads = 1024, kWaves = kThreads / 64;

// Unsigned keys in the order of the values; both zeros are one value.
__device__ inline uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ inline float unordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }
constexpr uint32_t kKeyMinusInf = 0x007FFFFFu;  // of -inf; NaNs have keys below it or above that of +inf

__device__ inline float value(const void *p, uint64_t at, bool f32) {
    return f32 ? static_cast<const float *>(p)[at] : __uint_as_float((uint32_t) static_cast<const uint16_t *>(p)[at] << 16);
}

// 2^x for x <= 0, off by 3e-13 of itself: x = n + f, |f| <= 1/2, Taylor's
// series of 2^f up to f^10.
__device__ inline double exp2_below(double x) {
    if (!(x > -1000.0)) return 0.0;
    const double n = rint(x), f = x - n;
    double p = 7.054911620801121e-9;
    p = p * f + 1.01780860092396960e-7;
    p = p * f + 1.32154867901443094e-6;
    p = p * f + 1.52527338040598402e-5;
    p = p * f + 1.54035303933816099e-4;
    p = p * f + 1.33335581464284434e-3;
    p = p * f + 9.61812910762847716e-3;
    p = p * f + 5.55041086648215800e-2;
    p = p * f + 2.40226506959100712e-1;
    p = p * f + 6.93147180559945309e-1;
    p = p * f + 1.0;
    return ldexp(p, (int)n);
}

// What a row asks for, read once.
struct Row {
    double scale;   // log2(e) / temperature
    double top_p, min_p;
    double heat;
    uint32_t k;     // 0: all
    bool bad;
};

__device__ inline Row row_of(const SampleParams &p, uint32_t r) {
    Row o;
    const float t = p.temperature ? p.temperature[r] : p.temperature_all;
    const float tp = p.top_p ? p.top_p[r] : p.top_p_all, mp = p.min_p ? p.min_p[r] : p.min_p_all;
    const int32_t k = p.top_k ? p.top_k[r] : p.top_k_all;
    o.bad = !(t >= 0) || tp != tp || mp != mp;
    o.heat = t > 0 ? (double)t : 1.0;
    o.scale = 1.4426950408889634 / o.heat;
    o.top_p = tp;
    o.min_p = fmin((double)mp, 1.0);
    o.k = t > 0 ? (k <= 0 || (uint32_t)k >= p.vocab ? 0 : (uint32_t)k) : 1;  // temperature 0: the largest
    return o;
}

// e of a value; the limit where the largest is infinite.
__device__ inline double weight(float z, float top, double scale) {
    return z == top ? 1.0 : exp2_below(((double)z - (double)top) * scale);
}

template <class T>
__device__ inline T wave_sum(T v) {
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    return v;
}
__device__ inline uint32_t wave_max(uint32_t v) {
    for (int d = 1; d < 64; d <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d));
    return v;
}

struct Shared {
    double mass[kWaves];
    uint32_t count[kWaves];
    uint64_t bin_mass[256];
    uint32_t bin_count[256];
    uint32_t pick, pick_count;
    double pick_mass;
    uint64_t found;
};

// The sum of a value over the workgroup, the same for all, in a fixed order.
__device__ inline double block_sum(double v, double *lds) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0;
    for (uint32_t i = 0; i < kWaves; ++i) s += lds[i];
    return s;
}

// Where a prefix of the order ends: all keys above `key`, and the first `equal`
// of those equal to it.
struct Border {
    uint32_t key, equal;
};
__device__ inline bool shorter(Border a, Border b) { return a.key > b.key || (a.key == b.key && a.equal < b.equal); }

// The border of the shortest prefix with at least `count` tokens (by_count), or
// with a sum of at least `mass`, among the keys that `in` admits; 8 bits of the
// key at a time.  above: the sum above the border's key.
__device__ inline Border find_border(const SampleParams &p, uint64_t at, float top, double scale, Border in, bool by_count,
                                     uint32_t count, double mass, double unit, Shared &s, double &above) {
    uint32_t prefix = 0;
    uint32_t have_count = 0;
    uint64_t have_mass = 0;
    uint32_t equal = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (uint32_t i = threadIdx.x; i < 256; i += kThreads) s.bin_mass[i] = 0, s.bin_count[i] = 0;
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < p.vocab; i += kThreads) {
            const float z = value(p.logits, at + i, p.f32);
            const uint32_t k = ordered(z);
            if (k < in.key || k <= kKeyMinusInf) continue;
            if (shift < 24 && (k >> (shift + 8)) != (prefix >> (shift + 8))) continue;
            const uint32_t b = k >> shift & 255;
            atomicAdd(&s.bin_count[b], 1u);
            atomicAdd((unsigned long long *)&s.bin_mass[b], (unsigned long long)(weight(z, top, scale) * unit + 0.5));
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            // (keys equal to `in`'s count as often as it admits)
            int b = 255;
            uint32_t c = have_count;
            uint64_t m = have_mass;
            for (; b > 0; --b) {
                if (by_count ? c + s.bin_count[b] >= count : (double)(m + s.bin_mass[b]) >= mass * unit) {
                    if (s.bin_count[b]) break;
                }
                c += s.bin_count[b];
                m += s.bin_mass[b];
            }
            s.pick = prefix | (uint32_t)b << shift;
            s.pick_count = c;
            s.found = m;
        }
        __syncthreads();
        prefix = s.pick;
        have_count = s.pick_count;
        have_mass = s.found;
        equal = s.bin_count[prefix >> shift & 255];
        __syncthreads();
    }
    above = (double)have_mass / unit;
    Border out{prefix, equal};
    if (by_count) {
        out.equal = min(equal, count - min(count, have_count));
    } else {
        const double each = weight(unordered(prefix), top, scale), left = mass - above;
        const double n = each > 0 ? ceil(left / each) : (double)equal;
        out.equal = n < 1 ? 1 : n < (double)equal ? (uint32_t)n : equal;
    }
    return out;
}

// A row by one workgroup, any filters.
__global__ __launch_bounds__(kThreads) void k_sample(SampleParams p) {
    __shared__ Shared s;
    const uint32_t r = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t at = (uint64_t)r * p.stride;
    const Row row = row_of(p, r);
    // the largest, and whether there is a NaN
    uint32_t best = 0, nan = 0;
    for (uint32_t i = threadIdx.x; i < p.vocab; i += kThreads) {
        const float z = value(p.logits, at + i, p.f32);
        nan |= z != z;
        if (z == z) best = max(best, ordered(z));
    }
    best = wave_max(best);
    nan = __any(nan);
    if (lane == 0) s.count[wave] = best, s.bin_count[wave] = nan;
    __syncthreads();
    for (uint32_t i = 0; i < kWaves; ++i) best = max(best, s.count[i]), nan |= s.bin_count[i];
    __syncthreads();
    if (nan || best <= kKeyMinusInf || row.bad) {
        if (threadIdx.x == 0) {
            p.token[r] = -1;
            if (p.logprob) p.logprob[r] = __builtin_nanf("");
        }
        return;
    }
    const float top = unordered(best);
    double all = 0;
    for (uint32_t i = threadIdx.x; i < p.vocab; i += kThreads) all += weight(value(p.logits, at + i, p.f32), top, row.scale);
    all = block_sum(all, s.mass);
    // fixed point: sums of `vocab` values of at most 1 stay below 2^63
    uint32_t bits = 1;
    while (p.vocab >> bits) ++bits;
    const double unit = ldexp(1.0, 62 - (int)bits);
    Border border{kKeyMinusInf + 1, p.vocab};
    double left = all, above;
    if (row.k) {
        border = find_border(p, at, top, row.scale, border, true, row.k, 0, unit, s, above);
        left = above + border.equal * weight(unordered(border.key), top, row.scale);
    }
    if (row.top_p < 1) {
        const Border b = find_border(p, at, top, row.scale, border, false, 0, row.top_p * left, unit, s, above);
        if (shorter(b, border)) border = b;
    }
    const double each = weight(unordered(border.key), top, row.scale);
    // sums and equals of each wave's run of tokens
    const uint32_t run = ((p.vocab + kThreads - 1) / kThreads) * 64;
    const uint32_t begin = min(wave * run, p.vocab), end = min(begin + run, p.vocab);
    double mine = 0;
    uint32_t equals = 0;
    for (uint32_t i = begin + lane; i < end; i += 64) {
        const float z = value(p.logits, at + i, p.f32);
        const uint32_t k = ordered(z);
        if (k > border.key) {
            const double e = weight(z, top, row.scale);
            mine += e >= row.min_p || z == top ? e : 0.0;
        }
        equals += k == border.key;
    }
    mine = wave_sum(mine);
    equals = wave_sum(equals);
    if (lane == 0) s.mass[wave] = mine, s.count[wave] = equals;
    __syncthreads();
    const bool keep_equal = each >= row.min_p || border.key == best;
    double sums[kWaves], total = 0;
    uint32_t rest = border.equal;
    uint32_t before_mine = 0;
    for (uint32_t i = 0; i < kWaves; ++i) {
        const uint32_t n = min(rest, s.count[i]);
        if (i == wave) before_mine = border.equal - rest;
        rest -= n;
        sums[i] = s.mass[i] + (keep_equal ? n * each : 0.0);
        total += sums[i];
    }
    const double want = (p.u_f64 ? static_cast<const double *>(p.u)[r] : (double)static_cast<const float *>(p.u)[r]) * total;
    // the run that holds the draw: the first whose running sum exceeds it; the last with any, if rounding leaves none
    double before = 0, base = 0;
    uint32_t hit = kWaves;
    for (uint32_t i = 0; i < kWaves; ++i) {
        if (sums[i] > 0 && (hit == kWaves || !(base + sums[hit] > want))) hit = i, base = before;
        before += sums[i];
    }
    if (wave != hit) return;
    uint32_t token = 0;
    double running = base;
    uint32_t seen = before_mine;
    bool done = false;
    for (uint32_t i0 = begin; i0 < end && !done; i0 += 64) {
        const uint32_t i = i0 + lane;
        const float z = i < end ? value(p.logits, at + i, p.f32) : -INFINITY;
        const uint32_t k = ordered(z);
        const bool same = i < end && k == border.key;
        const uint64_t m = __ballot(same);
        double e = 0;
        if (i < end && k > border.key) {
            e = weight(z, top, row.scale);
            if (!(e >= row.min_p || z == top)) e = 0;
        } else if (same && keep_equal && seen + __popcll(m & ((1ull << lane) - 1)) < border.equal) {
            e = each;
        }
        seen += __popcll(m);
        double x = e;
        for (int d = 1; d < 64; d <<= 1) {
            const double y = __shfl_up(x, d);
            if (lane >= (uint32_t)d) x += y;
        }
        const uint64_t some = __ballot(e > 0), over = __ballot(e > 0 && running + x > want);
        if (over) {
            token = i0 + (uint32_t)__ffsll((unsigned long long)over) - 1;
            done = true;
        } else if (some) {
            token = i0 + 63 - (uint32_t)__clzll((long long)some);  // the last so far
        }
        running += __shfl(x, 63);
    }
    if (lane == 0) {
        p.token[r] = token;
        if (p.logprob) {
            const float z = value(p.logits, at + token, p.f32);
            p.logprob[r] = (float)((z == top ? 0.0 : ((double)z - (double)top) / row.heat) - log(all));
        }
    }
}

}  // namespace

hipError_t launch_sample(const SampleParams &p, hipStream_t s) {
    k_sample<<<p.rows, kThreads, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace uzip
