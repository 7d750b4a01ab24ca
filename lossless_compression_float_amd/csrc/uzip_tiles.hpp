// uzip_tiles.hpp -- device code that the products with packed weights share:
// packed tiles in registers, activations, the forward epilogue and buffer
// reads (internal).
//
// Matrix instructions: v_mfma_f32_16x16x32_bf16.  Lane l = 16 q + c of a wave
// gives eight consecutive contraction values of row (first operand) or column
// (second operand) c, and holds rows 4 q .. 4 q + 3 of column c of the fp32
// result.  Which contraction index a (q, j) slot stands for is free as long as
// both operands agree; here, in half h of a block of 64, it is 32 h + 8 q + j,
// the order of a packed tile.
#pragma once

#include <stdint.h>

#include <type_traits>

#include <hip/hip_runtime.h>

#include "uzip_linear.hpp"

namespace uzip {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// Vectors at any value's address: the hardware takes them, so that rows of any
// stride move 16 bytes a lane (a lane a value, 239 x 116 outputs with their
// residual took 22 us instead of 14).
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

__device__ inline uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ inline uint32_t pack_bf16(float a, float b) {
    const bf16x2 v = __builtin_convertvector(f32x2{a, b}, bf16x2);
    return __builtin_bit_cast(uint32_t, v);
}
__device__ inline uint16_t to_bf16(float a) { return __builtin_bit_cast(uint16_t, (__bf16)a); }
__device__ inline float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ inline float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
__device__ inline float from_bf16(uint16_t u) { return __uint_as_float((uint32_t)u << 16); }

// ---- packed tiles -----------------------------------------------------------

// A tile's header: base exponent, count << 8 and flags; offset of its list or
// exponent bytes; the first kInline entries of the list.
struct Tile {
    uint4 sm;    // sign+mantissa bytes of this lane's 16 values
    uint2 code;  // their 4-bit codes
    uint4 h;     // header, uniform
};

// A list that would reach behind the extra region is dropped, so that damaged
// weights cannot make a kernel read out of range.
__device__ inline uint4 head_checked(const WeightView &w, uint4 h) {
    const uint32_t cnt = (h.x >> 8) & 0xFF;
    const uint32_t units = cnt == kTileRaw ? 64 : cnt <= kInline ? 0 : (cnt + 3) / 4;
    if (units > w.extra_units || (units && h.y > w.extra_units - units)) h.x &= ~0xFF00u;
    return h;
}
__device__ inline uint4 tile_head(const WeightView &w, uint64_t tile) { return head_checked(w, w.head[tile]); }

__device__ inline void tile_load(Tile &t, const WeightView &w, uint64_t tile, uint4 head, uint32_t lane) {
    const uint8_t *p = w.tiles + tile * kTileBytes;
    t.sm = *reinterpret_cast<const uint4 *>(p + lane * 16);
    t.code = *reinterpret_cast<const uint2 *>(p + kTileSm + lane * 8);
    t.h = make_uint4(uniform(head.x), uniform(head.y), uniform(head.z), uniform(head.w));
}

// Eight pairs of bf16 values from a lane's tile registers, no branches, 4 1/4
// operations a pair: the byte of sign and mantissa is spread over a half word;
// the code is masked out where it is and one packed multiplication brings it to
// the exponent's place, negative, and adds the base (two of four codes need a
// shift by 8 first, one for both); a bit select joins the two.  (Shifted to
// their place, masked, subtracted and joined: six.)
__device__ inline uint32_t tile_signs(const Tile &t, int p) {  // with the mantissa's top bits where the exponent goes
    const uint32_t sm[4] = {t.sm.x, t.sm.y, t.sm.z, t.sm.w};
    return __builtin_amdgcn_perm(0, sm[p >> 1], p & 1 ? 0x03030202u : 0x01010000u);
}
constexpr uint32_t kNotExponent = 0x807F807Fu;
__device__ inline uint32_t tile_join(uint32_t signs, uint32_t exponents) {
    return (signs & kNotExponent) | (exponents & ~kNotExponent);
}
__device__ inline uint32_t tile_pair(const Tile &t, int p, uint32_t base) {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    uint32_t by = p & 1 ? 0xFFF8FFF8u : 0xFF80FF80u;  // -8, -128
    asm("" : "+s"(by));                                // (a constant would become a shift and a subtraction)
    const uint32_t c = (p < 4 ? t.code.x : t.code.y) >> (p & 2 ? 8 : 0) & (p & 1 ? 0x00F000F0u : 0x000F000Fu);
    const u16x2 e = __builtin_bit_cast(u16x2, c) * __builtin_bit_cast(u16x2, by) + __builtin_bit_cast(u16x2, base);
    return tile_join(tile_signs(t, p), __builtin_bit_cast(uint32_t, e));
}
__device__ inline void tile_decode_plain(const Tile &t, uint32_t v[8]) {
    const uint32_t base = (t.h.x & 0xFF) * 0x00800080u;
#pragma unroll
    for (int p = 0; p < 8; ++p) v[p] = tile_pair(t, p, base);
}

// The two kinds of tile for which that is not enough: exponent bytes, and
// code 15 for exponent 0.
__device__ inline bool tile_special(uint32_t h) { return (h & kTileZero) || (h >> 8 & 0xFF) == kTileRaw; }
__device__ inline bool tile_raw(uint32_t h) { return (h >> 8 & 0xFF) == kTileRaw; }
__device__ inline void tile_decode_raw(const Tile &t, const WeightView &w, uint32_t lane, uint32_t v[8]) {
    const uint4 ex = *reinterpret_cast<const uint4 *>(w.extra + (uint64_t)t.h.y * 16 + lane * 16);
    const uint32_t e[4] = {ex.x, ex.y, ex.z, ex.w};
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const uint32_t x = e[p >> 1] >> (p & 1 ? 16 : 0);
        v[p] = tile_join(tile_signs(t, p), ((x & 0xFF) << 7) | ((x & 0xFF00) << 15));
    }
}
__device__ inline void tile_decode_zero(const Tile &t, uint32_t v[8]) {
    const uint32_t base = (t.h.x & 0xFF) * 0x00800080u;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const uint32_t c = p < 4 ? t.code.x : t.code.y;
        const int k = p & 3;
        const uint32_t x = (k == 0 ? c << 7 : k == 1 ? c << 3 : k == 2 ? c >> 1 : c >> 5) & 0x07800780u;
        const uint32_t z = (x + 0x00800080u) & 0x08000800u;  // bit 11 of the halves whose code is 15
        const uint32_t m = (z << 4) - (z >> 4);              // 0x7F80 there
        v[p] = tile_join(tile_signs(t, p), (base - (x & ~m)) & ~m);
    }
}

__device__ inline uint32_t tile_listed(uint32_t h) {
    const uint32_t cnt = h >> 8 & 0xFF;
    return cnt == kTileRaw ? 0 : min(cnt, kMaxListed);
}
// This lane's entry of a tile's list (lanes below tile_listed).
__device__ inline uint32_t tile_entry(const WeightView &w, uint4 h, uint32_t lane) {
    const uint32_t n = tile_listed(h.x);
    if (n <= kInline) return lane ? h.w : h.z;
    return reinterpret_cast<const uint32_t *>(w.extra + (uint64_t)h.y * 16)[min(lane, n - 1)];
}

// Puts one entry (uniform) into its place in registers.
__device__ inline void tile_patch(uint32_t e, uint32_t lane, uint32_t v[8]) {
    const uint32_t at = lane == (e >> 4 & 63) ? e >> 1 & 7 : 8;
    const uint32_t keep = e & 1 ? 0x0000FFFFu : 0xFFFF0000u, put = e >> 16 << (e & 1 ? 16 : 0);
#pragma unroll
    for (int p = 0; p < 8; ++p) v[p] = at == (uint32_t)p ? (v[p] & keep) | put : v[p];
}

// All of it, in registers.
__device__ inline void tile_decode(const Tile &t, const WeightView &w, uint32_t lane, uint32_t v[8]) {
    tile_decode_plain(t, v);
    if (!(t.h.x & (0xFF00u | kTileZero))) return;
    if (tile_raw(t.h.x)) tile_decode_raw(t, w, lane, v);
    else if (t.h.x & kTileZero) tile_decode_zero(t, v);
    const uint32_t n = tile_listed(t.h.x);
    if (n == 0) return;
    const uint32_t ent = tile_entry(w, t.h, lane);
    for (uint32_t i = 0; i < n; ++i) tile_patch(__builtin_amdgcn_readlane(ent, i), lane, v);
}

// ---- activations ----------------------------------------------------------------

__device__ inline float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)

// gelu(z) = z Phi(z).  In the lower tail 1 + erf(z / sqrt 2) is 0 or a few units of
// 2^-24, all of the result for z under -5; here Phi keeps its bits: with x = |z| /
// sqrt 2, erfc(x) exp(x^2) is smooth in t = 1 / (1 + 0.48 x), t times a polynomial of
// degree 8 (least squares over Chebyshev nodes of x up to 9.6, weighted until the
// largest relative error stops falling: 3e-8, and 3e-7 in fp32).  One branch-free
// path; the library's erfc took 2.1 us more for 777 x 4099 outputs.  Likewise the
// tanh form, (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)).
__device__ inline float normal_cdf(float z) {
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.33941125497f * fabsf(z));
    float p = -0.05212825909256935f;
    p = p * t + 0.27955687046051025f;
    p = p * t - 0.5505302548408508f;
    p = p * t + 0.41219520568847656f;
    p = p * t - 0.09404245018959045f;
    p = p * t + 0.2327471524477005f;
    p = p * t + 0.22962015867233276f;
    p = p * t + 0.27181339263916016f;
    p = p * t + 0.2707681953907013f;
    const float tail = 0.5f * (p * t) * expf(-0.5f * z * z);
    return z < 0 ? tail : 1.0f - tail;
}
__device__ inline float gelu_tanh_2u(float z) { return 2.0f * kGeluC * (z + 0.044715f * z * z * z); }

__device__ inline float activate(float z, uint32_t act) {
    switch (act) {
    case kActRelu: return z < 0 ? 0.0f : z;  // NaN stays
    case kActGelu: return z * normal_cdf(z);
    case kActGeluTanh: return z * sigmoid(gelu_tanh_2u(z));
    case kActSilu: return z * sigmoid(z);
    default: return z;
    }
}

__device__ inline float activate_grad(float z, uint32_t act) {
    switch (act) {
    case kActRelu: return z > 0 ? 1.0f : 0.0f;
    case kActGelu: return normal_cdf(z) + z * 0.3989422804014327f * expf(-0.5f * z * z);
    case kActGeluTanh: {
        const float u2 = gelu_tanh_2u(z), s = sigmoid(u2), r = sigmoid(-u2);  // r = 1 - s
        // (s r is 0 from |z| = 12 on: there z^2 must only not be infinite)
        return s + z * (s * r) * (2.0f * kGeluC * (1.0f + 0.134145f * fminf(z * z, 1e6f)));
    }
    case kActSilu: {
        const float s = sigmoid(z);
        return s * (1.0f + z * (1.0f - s));
    }
    default: return 1.0f;
    }
}

// ---- forward epilogue -----------------------------------------------------------

// W (4 or 8) consecutive values at `at`, of which the first `count` exist;
// those from `count` on are read as zeros.
template <int W>
__device__ inline void load(const void *p, uint64_t at, bool f32, uint32_t count, float v[W]) {
    if (f32) {
        const float *s = static_cast<const float *>(p) + at;
        if (count == W) {
#pragma unroll
            for (int k = 0; k < W; k += 4) {
                const f32x4 x = *reinterpret_cast<const f32x4_any *>(s + k);
                for (int i = 0; i < 4; ++i) v[k + i] = x[i];
            }
        } else {
#pragma unroll
            for (uint32_t i = 0; i < W; ++i) v[i] = i < count ? s[i] : 0.0f;
        }
    } else {
        const uint16_t *s = static_cast<const uint16_t *>(p) + at;
        if (count == W) {
            std::conditional_t<W == 8, u32x4, u32x2> x;
            if constexpr (W == 8)
                x = *reinterpret_cast<const u32x4_any *>(s);
            else
                x = *reinterpret_cast<const u32x2_any *>(s);
#pragma unroll
            for (int i = 0; i < W; ++i) v[i] = i & 1 ? bf16_hi(x[i / 2]) : bf16_lo(x[i / 2]);
        } else {
#pragma unroll
            for (uint32_t i = 0; i < W; ++i) v[i] = i < count ? from_bf16(s[i]) : 0.0f;
        }
    }
}

template <int W>
__device__ inline void store(void *p, uint64_t at, bool f32, uint32_t count, const float v[W]) {
    if (f32) {
        float *d = static_cast<float *>(p) + at;
        if (count == W) {
#pragma unroll
            for (int k = 0; k < W; k += 4) *reinterpret_cast<f32x4_any *>(d + k) = f32x4{v[k], v[k + 1], v[k + 2], v[k + 3]};
        } else {
#pragma unroll
            for (uint32_t i = 0; i < W; ++i)
                if (i < count) d[i] = v[i];
        }
    } else {
        uint16_t *d = static_cast<uint16_t *>(p) + at;
        if (count == W) {
            if constexpr (W == 8)
                *reinterpret_cast<u32x4_any *>(d) = u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                          pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
            else
                *reinterpret_cast<u32x2_any *>(d) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        } else {
#pragma unroll
            for (uint32_t i = 0; i < W; ++i)
                if (i < count) d[i] = to_bf16(v[i]);
        }
    }
}

// W consecutive outputs n .. n + W - 1 of row m.  z[0]: the product's values
// (of the gate's rows when gated), z[1]: of the up rows.  All sums are in fp32;
// y and the kept pre-activation are each rounded once, from the unrounded
// values.
template <bool GATED, int W>
__device__ inline void linear_out(const LinearEpi &e, uint64_t bias_at, uint32_t part_rows, uint64_t m, uint32_t n,
                                  float z[GATED ? 2 : 1][W]) {
    if (n >= part_rows) return;
    const uint32_t count = part_rows - n < W ? part_rows - n : W;
#pragma unroll
    for (int h = 0; h < (GATED ? 2 : 1); ++h) {
        if (e.bias) {
            float b[W];
            load<W>(e.bias, bias_at + h * part_rows + n, e.bias_f32, count, b);
            for (int i = 0; i < W; ++i) z[h][i] += b[i];
        }
        if (e.preact) store<W>(e.preact, m * e.preact_stride + h * part_rows + n, e.preact_f32, count, z[h]);
    }
    float y[W];
    if (GATED) {
        for (int i = 0; i < W; ++i) y[i] = z[0][i] * sigmoid(z[0][i]) * z[GATED ? 1 : 0][i];
    } else if (e.act == kActNone) {
        for (int i = 0; i < W; ++i) y[i] = z[0][i];
    } else {
        for (int i = 0; i < W; ++i) y[i] = activate(z[0][i], e.act);
    }
    if (e.residual) {
        float r[W];
        load<W>(e.residual, m * e.residual_stride + n, e.y_f32, count, r);
        for (int i = 0; i < W; ++i) y[i] += r[i];
    }
    store<W>(e.y, m * e.y_stride + n, e.y_f32, count, y);
}

// Rows [begin, end) of group g: offsets are clamped to the rows that exist, so
// that wrong ones cannot lead out of range.
__device__ inline void group_rows(const int32_t *offsets, uint32_t g, uint32_t tokens, uint32_t &begin, uint32_t &end) {
    if (!offsets) {
        begin = 0;
        end = tokens;
        return;
    }
    const int32_t a = offsets[g], b = offsets[g + 1];
    begin = a < 0 ? 0u : min((uint32_t)a, tokens);
    end = b < 0 ? 0u : min((uint32_t)b, tokens);
    if (end < begin) end = begin;
}

// A run of memory of which `bytes` may be read; reads behind them give zeros.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
constexpr uint32_t kRsrcWord3 = 0x00020000u;  // raw 32-bit buffer access on the gfx9 family
__device__ inline rsrc_t buffer(const uint8_t *p, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const uint64_t u = (uint64_t)uniform((uint32_t)(a >> 32)) << 32 | uniform((uint32_t)a);
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(u), (short)0, (int)uniform(bytes), (int)kRsrcWord3);
}
__device__ inline uint4 read16(rsrc_t r, uint32_t off) {
    const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
    return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ inline uint2 read8(rsrc_t r, uint32_t off) {
    const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, 0);
    return make_uint2(v[0], v[1]);
}
constexpr uint32_t kNowhere = 0xFFFFFF00u;  // an offset that is behind every buffer

}  // namespace
}  // namespace uzip
