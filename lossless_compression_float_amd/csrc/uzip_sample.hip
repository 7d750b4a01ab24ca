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
#include <float.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "uzip_lanes.hpp"
#include "uzip_sample.hpp"

namespace uzip {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

constexpr uint32_t kThreads = 1024, kWaves = kThreads / 64;

// Unsigned keys in the order of the values; both zeros are one value.
__device__ inline uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ inline float unordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }
constexpr uint32_t kKeyMinusInf = 0x007FFFFFu, kKeyInf = 0xFF800000u;  // NaNs have keys beyond them

__device__ inline float value(const void *p, uint64_t at, bool f32) {
    return f32 ? static_cast<const float *>(p)[at] : __uint_as_float((uint32_t) static_cast<const uint16_t *>(p)[at] << 16);
}

// 2^x for x <= 0, off by 1.5e-14 of itself and exact at 0: x = n + f, |f| <= 1/2,
// and 1 + f q(f) with q the polynomial of degree 8 whose largest relative error
// is smallest there (least squares, weighted until it stops falling).  Below -1000 anything tiny.
__device__ inline double exp2_low(double x) {
    constexpr double ROUND = 6755399441055744.0;  // 1.5 2^52: added, it leaves n in the low bits
    x = fmax(x, -1000.0);
    const double n = x + ROUND, f = x - (n - ROUND);
    double p = 1.01483365409060702e-07;
    p = p * f + 1.32583358083804669e-06;
    p = p * f + 1.52529900401267599e-05;
    p = p * f + 1.54034408823874327e-04;
    p = p * f + 1.33335576254202024e-03;
    p = p * f + 9.61812918116721968e-03;
    p = p * f + 5.55041086684161314e-02;
    p = p * f + 2.40226506957228025e-01;
    p = p * f + 6.93147180559885112e-01;
    p = p * f + 1.0;
    return __longlong_as_double(__double_as_longlong(p) + (int64_t)((uint64_t)__double_as_longlong(n) << 52));
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
    o.bad = !(t >= 0 && t < INFINITY) || tp != tp || mp != mp;
    o.heat = t > 0 ? (double)t : 1.0;
    o.scale = 1.4426950408889634 / o.heat;
    o.top_p = tp;
    o.min_p = fmin((double)mp, 1.0);
    o.k = t > 0 ? (k <= 0 || (uint32_t)k >= p.vocab ? 0 : (uint32_t)k) : 1;  // temperature 0: the largest
    return o;
}

// e of a value; the limit where the largest is infinite.
__device__ inline double weight(float z, float top, double scale) {
    const double x = ((double)z - (double)top) * scale;
    return z == top ? 1.0 : x > -1000.0 ? exp2_low(x) : 0.0;
}

// The same where the largest is finite and z not below 2^-1000 of it (there not 0).
__device__ inline double weight_near(float z, float top, double scale) { return exp2_low(((double)z - (double)top) * scale); }

constexpr uint32_t kMaxHot = 2048;         // groups that are read again apart from the others
constexpr uint32_t kMaxCandidates = 4096;  // tokens that are sorted
constexpr uint32_t kReads = 4, kCell = 64 * kReads;  // of a lane at a time, of a wave: a run
constexpr uint32_t kMaxCells = kThreads;             // runs
constexpr uint32_t kBins = 1024, kCoarse = kBins / 4;

struct Shared {
    double mass[kWaves], total;
    uint64_t large[kWaves];
    uint32_t count[kWaves], other[kWaves];
    uint32_t pick, pick_count;
    uint64_t pick_mass;
    uint32_t bin_count[kBins];
    uint64_t bin_mass[kBins];
    union {
        uint64_t hot[2 * kMaxVocab / kSegment];          // the hot lanes of each half segment
        uint32_t reads[kMaxHot * (kGroup / 4)];          // first tokens of the hot groups' reads, by index
    };
    double cell[kMaxCells];
    uint64_t tokens[kMaxCandidates];                     // key << 32 | ~index
    uint64_t sorted[kMaxCandidates];
};

template <class T>
__device__ inline T block_scan(T v, T *lds, T &total) { return scan_before<kWaves>(v, lds, total); }
__device__ inline uint32_t block_max(uint32_t v, uint32_t *lds) {
    v = wave_max(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return lane_of(row_scan<Max>(lds[threadIdx.x & (kWaves - 1)]), kWaves - 1);
}

// Fixed point for sums of at most `all`: 61 to 62 bits of it.
__device__ inline double unit_of(double all) { return ldexp(1.0, 61 - ilogb(all)); }

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
        if (threadIdx.x < 256) s.bin_mass[threadIdx.x] = 0, s.bin_count[threadIdx.x] = 0;
        __syncthreads();
        for (uint32_t i0 = 0; i0 < p.vocab; i0 += kThreads) {
            const uint32_t i = i0 + threadIdx.x;
            const float z = i < p.vocab ? value(p.logits, at + i, p.f32) : -INFINITY;
            const uint32_t k = ordered(z), b = k >> shift & 255;
            const bool on = k >= in.key && k > kKeyMinusInf && (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)));
            const uint64_t some = __ballot(on);
            if (!some) continue;
            const uint64_t w = on ? (uint64_t)(weight(z, top, scale) * unit + 0.5) : 0;
            const uint32_t lane = (uint32_t)__ffsll((unsigned long long)some) - 1, b0 = lane_of(b, lane);
            if (__ballot(on && b == b0) == some) {  // (a wave's equal ones together: 64 at one address take 64 turns)
                const uint64_t sum = wave_sum(w);
                if ((threadIdx.x & 63) == lane) {
                    atomicAdd(&s.bin_count[b], (uint32_t)__popcll(some));
                    atomicAdd((unsigned long long *)&s.bin_mass[b], (unsigned long long)sum);
                }
            } else if (on) {
                atomicAdd(&s.bin_count[b], 1u);
                atomicAdd((unsigned long long *)&s.bin_mass[b], (unsigned long long)w);
            }
        }
        __syncthreads();
        // from the highest bin down: the first at which the prefix is long enough; else the lowest
        const uint32_t b = 255 - min(threadIdx.x, 255u);
        const uint32_t c = threadIdx.x < 256 ? s.bin_count[b] : 0;
        const uint64_t m = threadIdx.x < 256 ? s.bin_mass[b] : 0;
        uint32_t counts;
        uint64_t masses;
        const uint32_t c0 = have_count + block_scan(c, s.count, counts);
        const uint64_t m0 = have_mass + block_scan(m, s.large, masses);
        const bool enough = c && (by_count ? c0 + c >= count : (double)(m0 + m) >= mass * unit);
        const uint32_t first = ~0u - block_max(enough ? 0xFFFFFFFFu - threadIdx.x : 0, s.other);
        if (threadIdx.x == min(first, 255u)) s.pick = prefix | b << shift, s.pick_count = c0, s.pick_mass = m0;
        __syncthreads();
        prefix = s.pick;
        have_count = s.pick_count;
        have_mass = s.pick_mass;
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

__device__ inline void finish(const SampleParams &p, uint32_t r, uint32_t token, float z, float top, double heat, double all) {
    p.token[r] = token;
    if (p.logprob) p.logprob[r] = (float)((z == top ? 0.0 : ((double)z - (double)top) / heat) - log(all));
}
__device__ inline double uniform_of(const SampleParams &p, uint32_t r) {
    return p.u_f64 ? static_cast<const double *>(p.u)[r] : (double)static_cast<const float *>(p.u)[r];
}

// Any row by passes over all of it, four for each border and two for the draw:
// where more than 4,096 tokens would have to be ordered, for many tokens alike in
// weight or a larger k.  One workgroup, by its operations and the turns of its
// atomics: 128,256 tokens, top-k 20,000 370 us, equal logits with top-p 420 to 500.
__device__ inline void by_histograms(const SampleParams &p, uint32_t r, const Row &row, float top, double all,
                                           Shared &s) {
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t at = (uint64_t)r * p.stride;
    const double unit = unit_of(all);
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
    const bool keep_equal = each >= row.min_p || unordered(border.key) == top;
    if (threadIdx.x == 0) {
        double total = 0;
        uint32_t rest = border.equal;
        for (uint32_t i = 0; i < kWaves; ++i) {
            const uint32_t n = min(rest, s.count[i]);
            s.other[i] = border.equal - rest;  // equals before this run
            rest -= n;
            s.mass[i] += keep_equal ? n * each : 0.0;
            total += s.mass[i];
        }
        s.total = uniform_of(p, r) * total;
        // the run that holds the draw: the first whose running sum exceeds it; the last with any, if rounding leaves none
        double before = 0, base = 0;
        uint32_t hit = kWaves;
        for (uint32_t i = 0; i < kWaves; ++i) {
            if (s.mass[i] > 0 && (hit == kWaves || !(base + s.mass[hit] > s.total))) hit = i, base = before;
            before += s.mass[i];
        }
        s.pick = hit;
        s.mass[0] = base;
    }
    __syncthreads();
    if (wave != s.pick) return;
    const double want = s.total;
    uint32_t token = 0, seen = s.other[wave];
    double running = s.mass[0];
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
        const double x = wave_scan<Sum>(e);
        const uint64_t some = __ballot(e > 0), over = __ballot(e > 0 && running + x > want);
        if (over) {
            token = i0 + (uint32_t)__ffsll((unsigned long long)over) - 1;
            done = true;
        } else if (some) {
            token = i0 + 63 - (uint32_t)__clzll((long long)some);  // the last so far
        }
        running += lane_of(x, 63);
    }
    if (lane == 0) finish(p, r, token, value(p.logits, at + token, p.f32), top, row.heat, all);
}

// ---- the survey ---------------------------------------------------------------------

// 16 bytes of values from token i on, -inf behind the last.
template <bool F32>
__device__ inline u32x4 read_raw(const SampleParams &p, uint64_t at, uint32_t i) {
    constexpr uint32_t W = F32 ? 4 : 8;
    if (i + W <= p.vocab)
        return F32 ? __builtin_bit_cast(u32x4, *reinterpret_cast<const f32x4_any *>(static_cast<const float *>(p.logits) + at + i))
                   : (u32x4) * reinterpret_cast<const u32x4_any *>(static_cast<const uint16_t *>(p.logits) + at + i);
    u32x4 x;
#pragma unroll
    for (uint32_t c = 0; c < 4; ++c) {
        if constexpr (F32) {
            x[c] = i + c < p.vocab ? static_cast<const uint32_t *>(p.logits)[at + i + c] : 0xFF800000u;
        } else {
            const uint16_t *s = static_cast<const uint16_t *>(p.logits) + at + i + 2 * c;
            const uint32_t lo = i + 2 * c < p.vocab ? s[0] : 0xFF80u, hi = i + 2 * c + 1 < p.vocab ? s[1] : 0xFF80u;
            x[c] = lo | hi << 16;
        }
    }
    return x;
}
template <bool F32, int W = F32 ? 4 : 8>
__device__ inline void unpack(u32x4 x, float v[W]) {
#pragma unroll
    for (int c = 0; c < W; ++c)
        v[c] = F32 ? __uint_as_float(x[c & 3]) : __uint_as_float(c & 1 ? x[c / 2 & 3] & 0xFFFF0000u : x[c / 2 & 3] << 16);
}
template <bool F32, int W = F32 ? 4 : 8>
__device__ inline void read_values(const SampleParams &p, uint64_t at, uint32_t i, float v[W]) {
    unpack<F32>(read_raw<F32>(p, at, i), v);
}

// A wave a segment of 2,048 tokens: its largest value, the sum of its weights
// relative to that, its smallest value, and the largest of each group of 16
// tokens (a lane's reads of half a segment), so that the second kernel reads
// little of the row again.  About 24 operations a token: 256 rows of 128,256 in
// fp32 36 us, 3.7 TB/s, half of the issue slots; 64 in bf16 12 us.
template <bool F32>
__global__ __launch_bounds__(256) void k_survey(SampleParams p) {
    constexpr int W = F32 ? 4 : 8, READS = kSegment / 64 / W, HALF = READS / 2;
    const uint32_t lane = threadIdx.x & 63;
    const uint64_t n = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (n >= (uint64_t)p.rows * p.segments) return;
    const uint32_t r = (uint32_t)(n / p.segments), seg = (uint32_t)(n % p.segments);
    const uint64_t at = (uint64_t)r * p.stride;
    float v[READS][W];
#pragma unroll
    for (int i = 0; i < READS; ++i) read_values<F32>(p, at, seg * kSegment + (i * 64 + lane) * W, v[i]);
    bool nan = false;
    float group[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        group[h] = -INFINITY;
#pragma unroll
        for (int i = h * HALF; i < (h + 1) * HALF; ++i)
#pragma unroll
            for (int c = 0; c < W; c += 2) {
                nan |= __builtin_isunordered(v[i][c], v[i][c + 1]);
                group[h] = fmaxf(group[h], fmaxf(v[i][c], v[i][c + 1]));
            }
        p.groups[(n * 2 + h) * 64 + lane] = group[h];
    }
    float top = fmaxf(group[0], group[1]), low = INFINITY;
#pragma unroll
    for (int i = 0; i < READS; ++i)
#pragma unroll
        for (int c = 0; c < W; ++c) low = fminf(low, v[i][c]);
    top = unordered(wave_max(ordered(top)));
    low = unordered(~wave_max(~ordered(low)));
    if (low == -INFINITY) {  // (masked tokens, and what is behind the last one, do not count)
        low = INFINITY;
#pragma unroll
        for (int i = 0; i < READS; ++i)
#pragma unroll
            for (int c = 0; c < W; ++c) low = fminf(low, v[i][c] > -INFINITY ? v[i][c] : INFINITY);
        low = unordered(~wave_max(~ordered(low)));
    }
    const double scale = row_of(p, r).scale;
    double sum = 0;
    if (top > -INFINITY) {
        double part[W];
#pragma unroll
        for (int c = 0; c < W; ++c) part[c] = 0;
#pragma unroll
        for (int i = 0; i < READS; ++i)
#pragma unroll
            for (int c = 0; c < W; ++c) part[c] += exp2_low(((double)v[i][c] - (double)top) * scale);
#pragma unroll
        for (int c = 0; c < W; ++c) sum += part[c];
        sum = wave_sum(sum);
    }
    if (top == INFINITY) sum = 1;
    if (__any(nan)) sum = __builtin_nan("");
    if (lane == 0) p.segment[n] = Segment{sum, top, low};
}

// ---- the draw -----------------------------------------------------------------------

// Bins of the values from the largest (0) to `floor` in even steps; beyond that
// kBins.  Four make a coarse bin.
struct Bins {
    float top, floor, inv;
};
__device__ inline uint32_t bin_of(const Bins &b, float z) {
    return z >= b.floor ? min((uint32_t)((b.top - z) * b.inv), kBins - 1) : kBins;
}

// The least value whose bin is at most `bin` (above infinity: none has it), by a
// wave that tries 64 keys at a time.
__device__ inline float least_of_bin(const Bins &b, uint32_t bin) {
    const uint32_t lane = threadIdx.x & 63;
    uint64_t lo = kKeyMinusInf;  // too low
    for (int shift = 26; shift > -6; shift -= 6) {
        const uint64_t step = shift > 0 ? 1ull << shift : 1;
        const uint64_t k = lo + (lane + 1) * step;
        const float z = k <= kKeyInf ? unordered((uint32_t)k) : INFINITY;
        const uint64_t low = __ballot(k < kKeyInf && !(z <= b.top && bin_of(b, z) <= bin) && z < b.top);
        lo += (uint64_t)__popcll(low) * step;
    }
    return lo + 1 >= kKeyInf ? INFINITY : unordered((uint32_t)(lo + 1));
}

// The reads that hold every token of the first `last` + 1 coarse bins, by
// index: of the hot groups, or all of the row's.
struct Reads {
    uint32_t count;
    bool all;
};
template <bool F32>
__device__ inline uint32_t read_at(const Shared &s, const Reads &q, uint32_t j) {
    return q.all ? j * (F32 ? 4 : 8) : s.reads[j];
}

// The first bins whose groups (by their largest values) hold k tokens, or
// weigh enough for top-p, none beyond `least`, and the reads of those groups.
constexpr uint32_t kAhead = 8;  // loads on their way
struct Groups {  // this lane's of the first 128 half segments: of kAhead times a wave each
    float z[kAhead];
};
__device__ inline void load_groups(Groups &g, const float *groups, uint32_t halves, uint32_t h0) {
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (uint32_t c = 0; c < kAhead; ++c) {
        const uint32_t h = h0 + c * kWaves + wave;
        g.z[c] = h < halves ? groups[h * 64 + lane] : -INFINITY;
    }
}
template <bool F32>
__device__ inline Reads choose_reads(const SampleParams &p, uint32_t r, const Row &row, const Bins &bins, double all,
                                     uint32_t least, Groups &g, uint32_t &last, Shared &s) {
    constexpr uint32_t W = F32 ? 4 : 8, READS = kGroup / W;
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float *groups = p.groups + (uint64_t)r * p.segments * 128;
    const uint32_t halves = p.segments * 2;
    const bool by_mass = !row.k && row.top_p < 1;
    const double unit = unit_of(all);
    s.bin_count[threadIdx.x] = 0;
    s.bin_mass[threadIdx.x] = 0;
    __syncthreads();
    for (uint32_t h0 = 0; h0 < halves; h0 += kAhead * kWaves) {
        if (h0) load_groups(g, groups, halves, h0);
#pragma unroll
        for (uint32_t c = 0; c < kAhead; ++c) {
            const uint32_t b = bin_of(bins, g.z[c]) / 4;
            if (b >= kCoarse) continue;
            atomicAdd(&s.bin_count[b], 1u);
            if (by_mass)  // (a lower bound of what the bins hold: fp32 will do, a little less of it)
                atomicAdd((unsigned long long *)&s.bin_mass[b],
                          (unsigned long long)(exp2f((float)(((double)g.z[c] - (double)bins.top) * row.scale)) * (float)(unit * 0.9999)));
        }
    }
    __syncthreads();
    // the first bin with groups for k, or weights for p, but none beyond `least`
    const uint32_t c = threadIdx.x < kCoarse ? s.bin_count[threadIdx.x] : 0;
    const uint64_t m = threadIdx.x < kCoarse ? s.bin_mass[threadIdx.x] : 0;
    uint32_t counts;
    uint64_t masses;
    const uint32_t c0 = block_scan(c, s.count, counts);
    const uint64_t m0 = by_mass ? block_scan(m, s.large, masses) : 0;
    const bool enough = threadIdx.x >= least || (row.k ? c0 + c >= row.k : by_mass && (double)(m0 + m) >= row.top_p * all * unit);
    last = min(0xFFFFFFFFu - block_max(enough ? 0xFFFFFFFFu - threadIdx.x : 0, s.other), kCoarse - 1);
    if (threadIdx.x == last) s.pick_count = c0 + c;
    __syncthreads();
    const uint32_t hot = s.pick_count;
    if (hot > kMaxHot) {
        __syncthreads();  // (all have read the count before sum_runs counts there anew)
        return Reads{(p.vocab + W - 1) / W, true};
    }
    for (uint32_t h0 = 0; h0 < halves; h0 += kAhead * kWaves) {
        if (halves > kAhead * kWaves) load_groups(g, groups, halves, h0);
#pragma unroll
        for (uint32_t c = 0; c < kAhead; ++c) {
            const uint64_t on = __ballot(bin_of(bins, g.z[c]) / 4 <= last);
            const uint32_t h = h0 + c * kWaves + wave;
            if (lane == 0 && h < halves) s.hot[h] = on;
        }
    }
    __syncthreads();
    constexpr uint32_t EACH = 2 * kMaxVocab / kSegment / kThreads;
    uint64_t mine[EACH];
    uint32_t sum = 0, total;
    // (a half a thread where there are no more, so that they share the work)
    auto half_of = [&](uint32_t i) { return halves > kThreads ? threadIdx.x * EACH + i : threadIdx.x + i * kThreads; };
#pragma unroll
    for (uint32_t i = 0; i < EACH; ++i) {
        const uint32_t h = half_of(i);
        mine[i] = h < halves ? s.hot[h] : 0;
        sum += __popcll(mine[i]);
    }
    uint32_t at = block_scan(sum, s.count, total);
    __syncthreads();  // (s.reads takes the place of s.hot)
#pragma unroll
    for (uint32_t i = 0; i < EACH; ++i) {
        const uint32_t h = half_of(i), n = __popcll(mine[i]);
        uint32_t rank = 0;
        for (uint64_t m64 = mine[i]; m64; m64 &= m64 - 1, ++rank) {
            const uint32_t l = (uint32_t)__ffsll((unsigned long long)m64) - 1;
#pragma unroll
            for (uint32_t q = 0; q < READS; ++q) s.reads[at * READS + q * n + rank] = h * (kSegment / 2) + (q * 64 + l) * W;
        }
        at += n;
    }
    __syncthreads();
    return Reads{total * READS, false};
}

// Tokens of the bins [from, to] into s.tokens, by index; false if there are too many.
template <bool F32>
__device__ inline bool collect(const SampleParams &p, uint64_t at, const Bins &bins, const Reads &q, uint32_t from, uint32_t to,
                               uint32_t &n, Shared &s) {
    constexpr uint32_t W = F32 ? 4 : 8;
    n = 0;
    for (uint32_t j0 = 0; j0 < q.count; j0 += kThreads) {
        const uint32_t j = j0 + threadIdx.x, i = j < q.count ? read_at<F32>(s, q, j) : p.vocab;
        float v[W];
        read_values<F32>(p, at, i, v);
        uint32_t have = 0;
#pragma unroll
        for (uint32_t c = 0; c < W; ++c) {
            const uint32_t b = bin_of(bins, v[c]);
            have += v[c] > -INFINITY && b >= from && b <= to;
        }
        uint32_t found, place = n + block_scan(have, s.count, found);
        n += found;
        if (n > kMaxCandidates) return false;
        if (have)
#pragma unroll
            for (uint32_t c = 0; c < W; ++c) {
                const uint32_t b = bin_of(bins, v[c]);
                if (v[c] > -INFINITY && b >= from && b <= to)
                    s.tokens[place++] = (uint64_t)ordered(v[c]) << 32 | (0xFFFFFFFFu - (i + c));
            }
    }
    __syncthreads();
    return true;
}

// s.tokens into s.sorted, the order of the filters.  Few are ranked by counting.
__device__ inline void sort_tokens(uint32_t n, Shared &s) {
    if (n <= 256) {
        uint32_t wide = 64;
        while (wide < n) wide *= 2;
        s.bin_count[threadIdx.x] = 0;
        __syncthreads();
        const uint32_t i = threadIdx.x & (wide - 1), parts = kThreads / wide;
        const uint64_t mine = i < n ? s.tokens[i] : 0;
        uint32_t above = 0;
        for (uint32_t j = threadIdx.x / wide; j < n; j += parts) above += s.tokens[j] > mine;
        if (i < n) atomicAdd(&s.bin_count[i], above);
        __syncthreads();
        if (threadIdx.x < n) s.sorted[s.bin_count[threadIdx.x]] = mine;
        __syncthreads();
        return;
    }
    uint32_t n2 = 512;
    while (n2 < n) n2 *= 2;
    for (uint32_t i = threadIdx.x; i < n2; i += kThreads) s.sorted[i] = i < n ? s.tokens[i] : 0;
    __syncthreads();
    for (uint32_t k = 2; k <= n2; k *= 2)
        for (uint32_t j = k / 2; j; j /= 2) {
            for (uint32_t t = threadIdx.x; t < n2 / 2; t += kThreads) {
                const uint32_t i = 2 * t - (t & (j - 1));
                const uint64_t a = s.sorted[i], b = s.sorted[i + j];
                if ((a < b) == ((i & k) == 0)) s.sorted[i] = b, s.sorted[i + j] = a;
            }
            __syncthreads();
        }
}
__device__ inline double sorted_weight(uint64_t x, float top, double scale) {
    return weight(unordered((uint32_t)(x >> 32)), top, scale);
}

constexpr uint32_t kOwn = kMaxCandidates / kThreads;  // tokens of a thread, one after another

// The first place, by index, at which the running sum of e[] over threads and
// their N values exceeds the draw; of the last with any, if rounding leaves
// none.  s.pick: set to kNone before the scan that gave `run`.
constexpr uint32_t kNone = 0xFFFFFFFFu;
template <uint32_t N>
__device__ inline uint32_t first_over(const double (&e)[N], double run, double want, Shared &s) {
    double sum = run;
#pragma unroll
    for (uint32_t c = 0; c < N; ++c) {
        const double before = sum;
        sum += e[c];
        if (sum > want && before <= want) atomicMin(&s.pick, threadIdx.x * N + c);
    }
    __syncthreads();
    const uint32_t first = s.pick;
    if (first != kNone) return first;
    // (the sums of neighbouring threads need not meet exactly)
    uint32_t over = 0, any = 0;
    sum = run;
#pragma unroll
    for (uint32_t c = 0; c < N; ++c) {
        const uint32_t i = threadIdx.x * N + c;
        sum += e[c];
        if (e[c] > 0) any = i + 1;
        if (e[c] > 0 && sum > want && !over) over = kNone - i;
    }
    over = block_max(over, s.count);
    any = block_max(any, s.other);
    return over ? kNone - over : any - 1;
}

// A lane's reads of its wave's run, all on their way at once.
template <bool F32>
__device__ inline void run_reads(const SampleParams &p, uint64_t at, const Shared &s, const Reads &q, uint32_t run, u32x4 (&x)[kReads]) {
#pragma unroll
    for (uint32_t u = 0; u < kReads; ++u) {
        const uint32_t j = run * kCell + u * 64 + (threadIdx.x & 63);
        x[u] = read_raw<F32>(p, at, j < q.count ? read_at<F32>(s, q, j) : p.vocab);
    }
}

// The first bin up to which all reads hold k tokens.
template <bool F32>
__device__ inline uint32_t bin_of_count(const SampleParams &p, uint64_t at, const Bins &bins, const Reads &q, uint32_t k, Shared &s) {
    constexpr uint32_t W = F32 ? 4 : 8;
    s.bin_count[threadIdx.x] = 0;
    __syncthreads();
    uint32_t tops = 0;
    for (uint32_t i = threadIdx.x >> 6; i * kCell < q.count; i += kWaves) {
        u32x4 x[kReads];
        run_reads<F32>(p, at, s, q, i, x);
#pragma unroll
        for (uint32_t u = 0; u < kReads; ++u) {
            float v[W];
            unpack<F32>(x[u], v);
#pragma unroll
            for (uint32_t c = 0; c < W; ++c) {
                const uint32_t b = bin_of(bins, v[c]);
                tops += v[c] == bins.top;
                if (v[c] != bins.top && v[c] > -INFINITY && b < kBins) atomicAdd(&s.bin_count[b], 1u);
            }
        }
    }
    uint32_t all_tops, all;
    block_scan(tops, s.count, all_tops);
    const uint32_t c = s.bin_count[threadIdx.x] + (threadIdx.x == 0 ? all_tops : 0), c0 = block_scan(c, s.count, all);
    return min(kNone - block_max(c0 + c >= k ? kNone - threadIdx.x : 0, s.other), kBins - 1);
}

// Rows with top-k: the tokens of the first bins that hold k, sorted.  Where the
// row has fewer groups than k, or too many of them are hot, the tokens
// themselves are counted.
template <bool F32>
__device__ inline bool by_sorting(const SampleParams &p, uint32_t r, const Row &row, const Bins &bins, double all,
                                  uint32_t least, Groups &g, Shared &s) {
    uint32_t last, n;
    const float top = bins.top;
    const uint64_t at = (uint64_t)r * p.stride;
    Reads q = choose_reads<F32>(p, r, row, bins, all, least, g, last, s);
    uint32_t to = last * 4 + 3;
    if (q.all || (last == least && s.pick_count < row.k)) {
        q = Reads{(p.vocab + (F32 ? 3 : 7)) / (F32 ? 4 : 8), true};
        to = min(bin_of_count<F32>(p, at, bins, q, row.k, s), least * 4 + 3);
    }
    if (!collect<F32>(p, at, bins, q, 0, to, n, s)) return false;
    sort_tokens(n, s);
    // the sums before each, and how many are kept
    double e[kOwn], part = 0, whole;
#pragma unroll
    for (uint32_t c = 0; c < kOwn; ++c) {
        const uint32_t i = threadIdx.x * kOwn + c;
        e[c] = i < n ? sorted_weight(s.sorted[i], top, row.scale) : 0.0;
        part += e[c];
    }
    double run = block_scan(part, s.mass, whole);
    const uint32_t limit = min(row.k, n);
    double x = run;
#pragma unroll
    for (uint32_t c = 0; c < kOwn; ++c) {
        x += e[c];
        if (threadIdx.x * kOwn + c == limit - 1) s.total = x;
    }
    __syncthreads();
    const double reach = row.top_p * s.total;
    uint32_t kept = 0, keep;
#pragma unroll
    for (uint32_t c = 0; c < kOwn; ++c) {
        const uint32_t i = threadIdx.x * kOwn + c;
        kept += i < limit && (i == 0 || ((row.top_p >= 1 || run < reach) && e[c] >= row.min_p));
        run += e[c];
    }
    block_scan(kept, s.count, keep);
    const uint64_t border = s.sorted[keep - 1];
    part = 0;
#pragma unroll
    for (uint32_t c = 0; c < kOwn; ++c) {
        const uint32_t i = threadIdx.x * kOwn + c;
        const uint64_t t = i < n ? s.tokens[i] : 0;
        e[c] = t >= border ? sorted_weight(t, top, row.scale) : 0.0;
        part += e[c];
    }
    if (threadIdx.x == 0) s.pick = kNone;
    run = block_scan(part, s.mass, whole);
    const uint32_t i = first_over(e, run, uniform_of(p, r) * whole, s);
    if (threadIdx.x == 0)
        finish(p, r, kNone - (uint32_t)s.tokens[i], unordered((uint32_t)(s.tokens[i] >> 32)), top, row.heat, all);
    return true;
}

// The sums of the tokens from z1 on by runs of reads (of those that min_p
// keeps), this thread's part of all of them, and the tokens from z0 to below z1
// as a list.
template <bool F32, bool MIN_P>
__device__ inline double sum_runs(const SampleParams &p, uint64_t at, const Reads &q, float top, const Row &row, float z0, float z1,
                                  Shared &s) {
    constexpr uint32_t W = F32 ? 4 : 8;
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (threadIdx.x == 0) s.pick_count = 0;
    __syncthreads();
    double above = 0;
    for (uint32_t run = wave; run * kCell < q.count; run += kWaves) {
        u32x4 x[kReads];
        run_reads<F32>(p, at, s, q, run, x);
        double sum = 0;
#pragma unroll
        for (uint32_t u = 0; u < kReads; ++u) {
            float v[W];
            unpack<F32>(x[u], v);
            float most = v[0];
#pragma unroll
            for (uint32_t c = 1; c < W; ++c) most = fmaxf(most, v[c]);
            if (__any(most >= z1)) {
#pragma unroll
                for (uint32_t c = 0; c < W; ++c) {
                    const double w = weight_near(v[c], top, row.scale), e = v[c] >= z1 ? w : 0.0;
                    if constexpr (MIN_P) {
                        above += e;
                        sum += e >= row.min_p ? e : 0.0;
                    } else {
                        sum += e;
                    }
                }
            }
            if (__any(most >= z0)) {
#pragma unroll
                for (uint32_t c = 0; c < W; ++c)
                    if (v[c] >= z0 && v[c] < z1) {
                        const uint32_t place = atomicAdd(&s.pick_count, 1u), first = read_at<F32>(s, q, run * kCell + u * 64 + lane);
                        if (place < kMaxCandidates) s.tokens[place] = (uint64_t)ordered(v[c]) << 32 | (kNone - (first + c));
                    }
            }
        }
        if constexpr (!MIN_P) above += sum;
        sum = wave_sum(sum);
        if (lane == 0) s.cell[run] = sum;
    }
    __syncthreads();
    return above;
}

// The first bin, up to `end`, up to which all reads weigh `reach`, in 64 bits;
// beyond the last if they do not.
template <bool F32>
__device__ inline uint32_t bin_of_mass(const SampleParams &p, uint64_t at, const Bins &bins, const Reads &q, uint32_t end, double scale,
                                       uint32_t tops, double unit, double reach, Shared &s) {
    constexpr uint32_t W = F32 ? 4 : 8;
    s.bin_mass[threadIdx.x] = 0;
    __syncthreads();
    for (uint32_t j = threadIdx.x; j < q.count; j += kThreads) {
        float v[W];
        read_values<F32>(p, at, read_at<F32>(s, q, j), v);
#pragma unroll
        for (uint32_t c = 0; c < W; ++c) {
            const uint32_t b = bin_of(bins, v[c]);
            if (v[c] != bins.top && b <= end)
                atomicAdd((unsigned long long *)&s.bin_mass[b], (unsigned long long)(weight_near(v[c], bins.top, scale) * unit + 0.5));
        }
    }
    __syncthreads();
    const uint64_t m = s.bin_mass[threadIdx.x] + (threadIdx.x == 0 ? (uint64_t)(tops * unit) : 0);
    uint64_t all;
    const uint64_t m0 = block_scan(m, s.large, all);
    return kNone - block_max(m && (double)(m0 + m) >= reach * unit ? kNone - threadIdx.x : 0, s.other);
}

// Rows with top-p or min-p alone.  A histogram of the weights, in fp32, tells
// the bin in which top-p ends, unless it ends among tokens too faint for it;
// then the sums before that bin in 64 bits, by runs of reads, beside the list of
// the bin's tokens, whose order gives the border.  Should the histogram's
// rounding have missed the bin, it is the next one.  False if that holds too
// many tokens.
template <bool F32>
__device__ inline bool by_sums(const SampleParams &p, uint32_t r, const Row &row, const Bins &bins, double all, uint32_t least,
                               Groups &g, Shared &s) {
    constexpr uint32_t W = F32 ? 4 : 8;
    const uint32_t wave = threadIdx.x >> 6;
    const uint64_t at = (uint64_t)r * p.stride;
    const float top = bins.top;
    uint32_t last;
    const Reads q = choose_reads<F32>(p, r, row, bins, all, least, g, last, s);
    const uint32_t runs = (q.count + kCell - 1) / kCell;
    if (runs > kMaxCells) return false;
    const uint32_t end = (q.all ? least : last) * 4 + 3;  // bins that the reads hold whole
    const double unit = unit_of(all), reach = fmax(row.top_p * all, 1e-300);
    uint32_t bin = kBins;
    if (row.top_p < 1) {
        // fixed point with 30 to 31 bits for all
        s.bin_count[threadIdx.x] = 0;
        __syncthreads();
        const float scale = (float)row.scale, unit31 = (float)(unit * 0x1p-31);
        uint32_t tops = 0;
        for (uint32_t i = wave; i * kCell < q.count; i += kWaves) {
            u32x4 x[kReads];
            run_reads<F32>(p, at, s, q, i, x);
#pragma unroll
            for (uint32_t u = 0; u < kReads; ++u) {
                float v[W];
                unpack<F32>(x[u], v);
#pragma unroll
                for (uint32_t c = 0; c < W; ++c) {
                    const uint32_t b = bin_of(bins, v[c]);
                    const uint32_t e = (uint32_t)(__builtin_amdgcn_exp2f((v[c] - top) * scale) * unit31 + 0.5f);
                    tops += v[c] == top;
                    if (v[c] != top && b <= end) atomicAdd(&s.bin_count[b], e);  // (equal ones would meet at one address)
                }
            }
        }
        uint32_t all_tops;
        block_scan(tops, s.count, all_tops);
        const uint64_t m = s.bin_count[threadIdx.x] + (threadIdx.x == 0 ? (uint64_t)(all_tops * unit * 0x1p-31) : 0);
        uint64_t masses;
        const uint64_t m0 = block_scan(m, s.large, masses);
        bin = kNone - block_max(m && (double)(m0 + m) >= reach * unit * 0x1p-31 ? kNone - threadIdx.x : 0, s.other);
        // Below the reach in all bins: min_p ends all if they are below it by more than the histogram's error (half a unit a token;
        // 80 2^-22 of a weight's logarithm; anything where differences of logits overflow), else 64 bits tell.
        const double most = (double)masses + 0.5 * W * q.count + 0x1p-12 * all * unit * 0x1p-31;
        if (bin >= kBins && !(bins.inv > 0 && most < reach * unit * 0x1p-31))
            bin = bin_of_mass<F32>(p, at, bins, q, end, row.scale, all_tops, unit, reach, s);
        if (bin >= kBins) {
            if (!q.all && last < least) return false;
            bin = kBins;
        }
    }
    uint64_t border = 0;
    for (uint32_t attempt = 0;; ++attempt) {
        const float z0 = bin < kBins ? least_of_bin(bins, bin) : INFINITY;
        const float z1 = bin == kBins ? bins.floor : bin ? least_of_bin(bins, bin - 1) : INFINITY;
        const double above = row.min_p > 0 ? sum_runs<F32, true>(p, at, q, top, row, z0, z1, s)
                                           : sum_runs<F32, false>(p, at, q, top, row, z0, z1, s);
        s.bin_mass[threadIdx.x] = 0;  // of the bin's kept tokens, by runs
        if (bin == kBins) break;
        const uint32_t n = s.pick_count;
        if (n > kMaxCandidates) return false;
        sort_tokens(n, s);
        double e[kOwn], part = 0, whole, before;
#pragma unroll
        for (uint32_t c = 0; c < kOwn; ++c) {
            const uint32_t i = threadIdx.x * kOwn + c;
            e[c] = i < n ? weight_near(unordered((uint32_t)(s.sorted[i] >> 32)), top, row.scale) : 0.0;
            part += e[c];
        }
        block_scan(above, s.mass, before);
        double run = block_scan(part, s.mass, whole) + before;
        uint32_t kept = 0, keep;
#pragma unroll
        for (uint32_t c = 0; c < kOwn; ++c) {
            const uint32_t i = threadIdx.x * kOwn + c;
            if (i < n && run < reach) {
                ++kept;
                const uint32_t token = kNone - (uint32_t)s.sorted[i];
                uint32_t j = token / W;
                if (!q.all) {  // the last read that begins at or before it
                    uint32_t lo = 0, hi = q.count;
                    while (hi - lo > 1) {
                        const uint32_t mid = (lo + hi) / 2;
                        if (s.reads[mid] <= token) lo = mid;
                        else hi = mid;
                    }
                    j = lo;
                }
                if (e[c] >= row.min_p)
                    atomicAdd((unsigned long long *)&s.bin_mass[j / kCell], (unsigned long long)(e[c] * unit + 0.5));
            }
            run += e[c];
        }
        block_scan(kept, s.count, keep);
        if (keep && !(keep == n && before + whole < reach)) {
            border = s.sorted[keep - 1];
            break;
        }
        const bool up = keep == 0;
        if (attempt == 2 || (up && bin == 0) || (!up && bin >= end)) return false;
        bin += up ? ~0u : 1u;
        __syncthreads();
    }
    if (threadIdx.x == 0) s.pick = kNone;
    __syncthreads();
    const double mine[1] = {threadIdx.x < runs ? s.cell[threadIdx.x] + (double)s.bin_mass[threadIdx.x] / unit : 0.0};
    double whole;
    double run = block_scan(mine[0], s.mass, whole);
    const double want = uniform_of(p, r) * whole;
    const uint32_t cell = first_over(mine, run, want, s);
    if (threadIdx.x == cell) s.total = run;
    // the run again, a read a lane
    const uint32_t j = cell * kCell + threadIdx.x, i = threadIdx.x < kCell && j < q.count ? read_at<F32>(s, q, j) : p.vocab;
    float v[W];
    double e[W], sum = 0;
    read_values<F32>(p, at, i, v);
#pragma unroll
    for (uint32_t c = 0; c < W; ++c) {
        const bool in = v[c] >= bins.floor && ((uint64_t)ordered(v[c]) << 32 | (kNone - (i + c))) >= border;
        const double x = in ? weight_near(v[c], top, row.scale) : 0.0;
        e[c] = x >= row.min_p ? x : 0.0;
        sum += e[c];
    }
    __syncthreads();
    if (threadIdx.x == 0) s.pick = kNone;
    run = block_scan(sum, s.mass, whole) + s.total;
    const uint32_t place = first_over(e, run, want, s);
#pragma unroll
    for (uint32_t c = 0; c < W; ++c)
        if (threadIdx.x * W + c == place) finish(p, r, i + c, v[c], top, row.heat, all);
    return true;
}

// A workgroup a row, after the survey.  Latency, in steps of 0.5 to 2 us: one
// row with top-k 12 us, 64 without filters 7; a row with top-p that has to be
// read whole 70 us, bound by its operations; 139 where it ends among tokens too
// faint for the histogram in fp32 (one logit 22 above the others, top_p 0.99999).
template <bool F32>
__global__ __launch_bounds__(kThreads) void k_draw(SampleParams p) {
    __shared__ Shared s;
    const uint32_t r = blockIdx.x;
    const uint64_t at = (uint64_t)r * p.stride;
    const Row row = row_of(p, r);
    const Segment *segs = p.segment + (uint64_t)r * p.segments;
    // thread i has segments PER i .. , so that sums over the threads before it are those of the tokens before
    constexpr uint32_t PER = kMaxVocab / kSegment / kThreads;
    uint32_t best = 0, nan = 0, lowest = 0;
    Segment mine[PER];
#pragma unroll
    for (uint32_t c = 0; c < PER; ++c) {
        const uint32_t i = threadIdx.x * PER + c;
        mine[c] = i < p.segments ? segs[i] : Segment{0.0, -INFINITY, INFINITY};
        best = max(best, ordered(mine[c].top));
        lowest = max(lowest, ~ordered(mine[c].low));
        nan |= mine[c].sum != mine[c].sum;
    }
    Groups g;
    load_groups(g, p.groups + (uint64_t)r * p.segments * 128, p.segments * 2, 0);
    best = wave_max(best);
    lowest = wave_max(lowest);
    nan = __any(nan);
    if ((threadIdx.x & 63) == 0) s.count[threadIdx.x >> 6] = nan ? kNone : best, s.other[threadIdx.x >> 6] = lowest;
    __syncthreads();
    best = lane_of(row_scan<Max>(s.count[threadIdx.x & (kWaves - 1)]), kWaves - 1);
    lowest = ~lane_of(row_scan<Max>(s.other[threadIdx.x & (kWaves - 1)]), kWaves - 1);
    if (best == kNone || best <= kKeyMinusInf || row.bad) {
        if (threadIdx.x == 0) {
            p.token[r] = -1;
            if (p.logprob) p.logprob[r] = __builtin_nanf("");
        }
        return;
    }
    const float top = unordered(best);
    double share[PER], part = 0, all;
#pragma unroll
    for (uint32_t c = 0; c < PER; ++c) {
        share[c] = mine[c].sum * weight(mine[c].top, top, row.scale);
        part += share[c];
    }
    double run = block_scan(part, s.mass, all);
    if (top < INFINITY && row.k == 1) {
        // the first of the largest
        uint32_t first = 0;
#pragma unroll
        for (uint32_t c = PER; c-- > 0;)
            if (mine[c].top == top) first = kNone - (threadIdx.x * PER + c);
        const uint32_t seg = kNone - block_max(first, s.count);
        first = 0;
#pragma unroll
        for (uint32_t c = 0; c < kSegment / kThreads; ++c) {
            const uint32_t i = seg * kSegment + c * kThreads + threadIdx.x;
            if (i < p.vocab && value(p.logits, at + i, F32) == top) first = max(first, kNone - i);
        }
        first = block_max(first, s.other);
        if (threadIdx.x == 0) finish(p, r, kNone - first, top, top, row.heat, all);
        return;
    }
    if (top < INFINITY && !row.k && row.top_p >= 1 && row.min_p <= 0) {
        // the segment, then the token, at which the running sum exceeds the draw
        const double want = uniform_of(p, r) * all;
        if (threadIdx.x == 0) s.pick = kNone;
        __syncthreads();
        const uint32_t seg = first_over(share, run, want, s);
#pragma unroll
        for (uint32_t c = 0; c < PER; ++c) {
            if (threadIdx.x * PER + c == seg) s.total = run;
            run += share[c];
        }
        constexpr uint32_t OWN = kSegment / kThreads;
        const uint32_t i0 = seg * kSegment + threadIdx.x * OWN;
        float z[OWN];
        double e[OWN], sum = 0, whole;
#pragma unroll
        for (uint32_t c = 0; c < OWN; ++c) {
            z[c] = i0 + c < p.vocab ? value(p.logits, at + i0 + c, F32) : -INFINITY;
            e[c] = weight(z[c], top, row.scale);
            sum += e[c];
        }
        __syncthreads();
        if (threadIdx.x == 0) s.pick = kNone;
        run = block_scan(sum, s.mass, whole) + s.total;
        const uint32_t place = first_over(e, run, want, s);
#pragma unroll
        for (uint32_t c = 0; c < OWN; ++c)
            if (threadIdx.x * OWN + c == place) finish(p, r, i0 + c, z[c], top, row.heat, all);
        return;
    }
    if (top < INFINITY) {
        // Tokens that weigh less than 2^-80 of the largest change no sum in 64 bits and are left out, as -inf is.
        Bins bins;
        bins.top = top;
        bins.floor = fmaxf(fmaxf(unordered(lowest), (float)((double)top - 80.0 / row.scale)), -FLT_MAX);
        const float range = top - bins.floor;
        bins.inv = range > 0 ? (kBins - 0.01f) / range : 0.0f;  // (0 where the range overflows: all in the first bin, NaN converts to 0)
        // the last coarse bin with tokens that min_p keeps (top-p of the first k needs the sum of the others too)
        uint32_t least = kCoarse - 1;
        if (row.min_p > 0 && !(row.k && row.top_p < 1)) {
            const double z = (double)top + log(row.min_p) * row.heat * 1.000001 - fabs((double)top) * 1e-6;
            least = min(bin_of(bins, (float)z) / 4 + 1, kCoarse - 1);
        }
        if (row.k ? by_sorting<F32>(p, r, row, bins, all, least, g, s) : by_sums<F32>(p, r, row, bins, all, least, g, s)) return;
        __syncthreads();
    } else {  // the infinite ones share alike
        double n = 0;
        for (uint32_t i = threadIdx.x; i < p.vocab; i += kThreads) n += value(p.logits, at + i, F32) == INFINITY;
        block_scan(n, s.mass, all);
        __syncthreads();
    }
    by_histograms(p, r, row, top, all, s);
}

}  // namespace

hipError_t launch_sample(const SampleParams &p, hipStream_t s) {
    const uint32_t wgs = (uint32_t)(((uint64_t)p.rows * p.segments + 3) / 4);
    if (p.f32) {
        k_survey<true><<<wgs, 256, 0, s>>>(p);
        k_draw<true><<<p.rows, kThreads, 0, s>>>(p);
    } else {
        k_survey<false><<<wgs, 256, 0, s>>>(p);
        k_draw<false><<<p.rows, kThreads, 0, s>>>(p);
    }
    return hipGetLastError();
}

}  // namespace uzip
