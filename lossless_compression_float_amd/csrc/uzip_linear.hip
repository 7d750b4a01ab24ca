// uzip_linear.hip -- gfx950 kernels of the products that read losslessly
// packed bf16 weights: packing, the skinny product for few rows, the tiled
// product with its epilogues (bias, activation, gate, residual; the softmax
// loss), the two products of the backward pass, and the small kernels around
// them.
//
// Matrix instructions: v_mfma_f32_16x16x32_bf16.  Lane l = 16 q + c of a wave
// gives eight consecutive contraction values of row (first operand) or column
// (second operand) c, and holds rows 4 q .. 4 q + 3 of column c of the fp32
// result.  Which contraction index a (q, j) slot stands for is free as long as
// both operands agree; here, in half h of a block of 64, it is 16 q + 8 h + j,
// the order of a packed tile.
#include <stdint.h>

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

__device__ inline uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ inline uint32_t pack_bf16(float a, float b) {
    const bf16x2 v = __builtin_convertvector(f32x2{a, b}, bf16x2);
    return __builtin_bit_cast(uint32_t, v);
}
__device__ inline uint16_t to_bf16(float a) { return __builtin_bit_cast(uint16_t, (__bf16)a); }
__device__ inline float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ inline float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
__device__ inline float from_bf16(uint16_t u) { return __uint_as_float((uint32_t)u << 16); }

// Waits for this wave's LDS operations and for the workgroup's other waves.
// Loads from memory that are still on their way into registers stay so.
__device__ inline void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// ---- packed tiles -----------------------------------------------------------

struct Tile {
    uint4 sm;      // sign+mantissa bytes of this lane's 16 values
    uint2 code;    // their 4-bit codes
    uint32_t ent;  // this lane's list entry
    uint32_t h;    // header word 0, uniform
    uint32_t off;  // header word 1, uniform
};

// A tile's header.  A list that would reach behind the extra region is
// dropped, so that damaged weights cannot make a kernel read out of range.
__device__ inline uint2 tile_head(const WeightView &w, uint64_t tile) {
    uint2 h = w.head[tile];
    const uint32_t cnt = (h.x >> 8) & 0xFF;
    const uint32_t units = cnt == kTileRaw ? 64 : (cnt + 3) / 4;
    if (units > w.extra_units || h.y > w.extra_units - units) h.x &= ~0xFF00u;
    return h;
}

__device__ inline void tile_load(Tile &t, const WeightView &w, uint64_t tile, uint2 head, uint32_t lane) {
    const uint8_t *p = w.tiles + tile * kTileBytes;
    t.sm = *reinterpret_cast<const uint4 *>(p + lane * 16);
    t.code = *reinterpret_cast<const uint2 *>(p + kTileSm + lane * 8);
    t.h = uniform(head.x);
    t.off = uniform(head.y);
    t.ent = 0;
    const uint32_t cnt = (t.h >> 8) & 0xFF;
    if (cnt != 0 && cnt != kTileRaw) {
        const uint32_t *list = reinterpret_cast<const uint32_t *>(w.extra + (uint64_t)t.off * 16);
        if (lane < cnt) t.ent = list[lane];
    }
}

// Eight pairs of bf16 values from a lane's tile registers: five operations a
// pair.  The byte of sign and mantissa is spread over a half word and masked,
// the code shifted to the exponent's place and taken from the base.
__device__ inline void tile_decode(const Tile &t, const WeightView &w, uint32_t lane, uint32_t v[8]) {
    const uint32_t sm[4] = {t.sm.x, t.sm.y, t.sm.z, t.sm.w};
    const uint32_t cnt = (t.h >> 8) & 0xFF;
    if (cnt == kTileRaw) {
        const uint4 ex = *reinterpret_cast<const uint4 *>(w.extra + (uint64_t)t.off * 16 + lane * 16);
        const uint32_t e[4] = {ex.x, ex.y, ex.z, ex.w};
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const uint32_t s = __builtin_amdgcn_perm(0, sm[p >> 1], p & 1 ? 0x03030202u : 0x01010000u) & 0x807F807Fu;
            const uint32_t x = e[p >> 1] >> (p & 1 ? 16 : 0);
            v[p] = s | ((x & 0xFF) << 7) | ((x & 0xFF00) << 15);
        }
        return;
    }
    const uint32_t base = (t.h & 0xFF) * 0x00800080u;
    const bool zero = (t.h & kTileZero) != 0;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const uint32_t c = p < 4 ? t.code.x : t.code.y;
        const int k = p & 3;
        uint32_t x = (k == 0 ? c << 7 : k == 1 ? c << 3 : k == 2 ? c >> 1 : c >> 5) & 0x07800780u;
        const uint32_t s = __builtin_amdgcn_perm(0, sm[p >> 1], p & 1 ? 0x03030202u : 0x01010000u);
        if (zero) {
            const uint32_t z = (x + 0x00800080u) & 0x08000800u;  // bit 11 of the halves whose code is 15
            const uint32_t m = (z << 4) - (z >> 4);              // 0x7F80 there
            x = (base - (x & ~m)) & ~m;
        } else {
            x = base - x;
        }
        v[p] = (s & 0x807F807Fu) | x;
    }
    if (cnt != 0) {
        const uint32_t n = cnt < kMaxListed ? cnt : kMaxListed;
        for (uint32_t i = 0; i < n; ++i) {
            const uint32_t e = __builtin_amdgcn_readlane(t.ent, i);
            const uint32_t at = (e >> 4) & 63, idx = e & 15;
            const bool mine = lane == at;
            const uint32_t val = e >> 16;
#pragma unroll
            for (int p = 0; p < 8; ++p)
                if ((idx >> 1) == (uint32_t)p)
                    v[p] = !mine ? v[p] : idx & 1 ? (v[p] & 0xFFFFu) | (val << 16) : (v[p] & 0xFFFF0000u) | val;
        }
    }
}

// ---- packing ------------------------------------------------------------------

// This lane's 16 values of a tile, zero outside the matrix.
__device__ inline void tile_gather(const PackParams &p, uint64_t tile, uint32_t lane, uint16_t v[16]) {
    const uint32_t q = lane >> 4, r = lane & 15;
    const uint64_t kb = tile % p.l.col_blocks, t = tile / p.l.col_blocks;
    const uint64_t rb = t % p.l.row_blocks, e = t / p.l.row_blocks;
    const uint64_t part = rb / p.l.part_blocks, row = (rb % p.l.part_blocks) * kTileRows + r;
    const uint64_t c0 = kb * kTileCols + q * 16;
    const uint16_t *src = p.in + e * p.matrix_stride + (part * p.l.part_rows + row) * p.row_stride + c0;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = row < p.l.part_rows && c0 + i < p.cols ? src[i] : (uint16_t)0;
}

// A wave packs a tile: the histogram of its exponents picks the window that
// holds most of them.  Bound by the reads and writes of memory.
__global__ __launch_bounds__(256) void k_pack(PackParams p) {
    __shared__ uint32_t hist[4][256 + 16];
    const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const uint64_t tile = (uint64_t)blockIdx.x * 4 + wave;
    uint32_t *h = hist[wave];
    for (uint32_t i = lane; i < 272; i += 64) h[i] = 0;
    __syncthreads();
    if (tile >= p.l.tiles) return;
    uint16_t v[16];
    tile_gather(p, tile, lane, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) atomicAdd(&h[16 + ((v[i] >> 7) & 0xFF)], 1u);  // h[16 + e]: exponent e
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_wave_barrier();
    // windows [b - 15, b], and [b - 14, b] with exponent 0; of equals the highest base, then the plain kind
    const uint32_t zeros = h[16];
    uint32_t best = 0;
    for (uint32_t j = 0; j < 4; ++j) {
        const uint32_t b = j * 64 + lane;
        uint32_t s = 0;
        for (uint32_t i = 0; i < 15; ++i) s += h[16 + b - i];
        const uint32_t plain = s + h[16 + b - 15];
        const uint32_t with0 = b >= 15 ? s + zeros : 0;
        best = max(best, plain << 10 | b << 1 | 1u);
        best = max(best, with0 << 10 | b << 1);
    }
    for (int d = 32; d; d >>= 1) best = max(best, (uint32_t)__shfl_xor((int)best, d));
    const uint32_t base = (best >> 1) & 0xFF, zero = !(best & 1);
    const uint32_t outside = 1024 - (best >> 10);
    uint32_t sm[4] = {0, 0, 0, 0}, cd[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t e = (v[i] >> 7) & 0xFF;
        sm[i >> 2] |= (((v[i] >> 8) & 0x80u) | (v[i] & 0x7Fu)) << (8 * (i & 3));
        uint32_t c = base - e;
        if (zero && e == 0) c = 15;
        else if (e > base || c > (zero ? 14u : 15u)) c = 0;  // listed
        cd[i >> 3] |= c << (4 * ((i >> 1) & 3) + 16 * (i & 1));
    }
    uint8_t *out = p.out + p.l.tile_off + tile * kTileBytes;
    *reinterpret_cast<uint4 *>(out + lane * 16) = make_uint4(sm[0], sm[1], sm[2], sm[3]);
    *reinterpret_cast<uint2 *>(out + kTileSm + lane * 8) = make_uint2(cd[0], cd[1]);
    if (lane == 0) {
        const uint32_t cnt = outside > kMaxListed ? kTileRaw : outside;
        reinterpret_cast<uint2 *>(p.out + p.l.head_off)[tile] =
            make_uint2(base | cnt << 8 | (zero ? kTileZero : 0u), cnt == kTileRaw ? 64 : (cnt + 3) / 4);
    }
}

// Sums over a block of 256 threads; every thread gets the exclusive prefix.
__device__ inline uint64_t block_scan(uint64_t v, uint64_t *lds, uint64_t &total) {
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint64_t x = v;
    for (int d = 1; d < 64; d <<= 1) {
        const uint64_t y = __shfl_up((unsigned long long)x, d);
        if (lane >= (uint32_t)d) x += y;
    }
    if (lane == 63) lds[wave] = x;
    __syncthreads();
    uint64_t before = 0;
    total = 0;
    for (uint32_t i = 0; i < 4; ++i) {
        if (i < wave) before += lds[i];
        total += lds[i];
    }
    __syncthreads();
    return before + x - v;
}

// Extra units of each block of kScanTiles tiles.
__global__ __launch_bounds__(256) void k_pack_sums(PackParams p) {
    __shared__ uint64_t lds[4];
    const uint2 *head = reinterpret_cast<const uint2 *>(p.out + p.l.head_off);
    uint64_t s = 0, total;
    for (uint32_t i = threadIdx.x; i < kScanTiles; i += 256) {
        const uint64_t t = (uint64_t)blockIdx.x * kScanTiles + i;
        if (t < p.l.tiles) s += head[t].y;
    }
    block_scan(s, lds, total);
    if (threadIdx.x == 0) p.sums[blockIdx.x] = total;
}

// Exclusive scan of those sums, the header and the size.
__global__ __launch_bounds__(256) void k_pack_scan(PackParams p) {
    __shared__ uint64_t lds[4];
    const uint64_t blocks = (p.l.tiles + kScanTiles - 1) / kScanTiles;
    uint64_t carry = 0;
    for (uint64_t b = 0; b < blocks; b += 256) {
        const uint64_t i = b + threadIdx.x;
        uint64_t total;
        const uint64_t v = i < blocks ? p.sums[i] : 0;
        const uint64_t x = block_scan(v, lds, total);
        if (i < blocks) p.sums[i] = carry + x;
        carry += total;
    }
    if (threadIdx.x < kWeightHeader / 8) {
        const uint64_t total = p.l.extra_off + carry * 16;
        const uint64_t f[8] = {kWeightMagic | 1ull << 32, p.matrices, p.rows, p.cols, p.gated, p.l.tile_off, p.l.extra_off, total};
        uint64_t x = 0;
        for (uint32_t i = 0; i < 8; ++i)
            if (threadIdx.x == i) x = f[i];
        reinterpret_cast<uint64_t *>(p.out)[threadIdx.x] = x;
        if (threadIdx.x == 0) *p.out_size = total;
    }
    // between the tile headers and the tiles
    const uint64_t gap = p.l.head_off + 8 * p.l.tiles + 8 * threadIdx.x;
    if (gap < p.l.tile_off) *reinterpret_cast<uint64_t *>(p.out + gap) = 0;
}

// The tiles' offsets.
__global__ __launch_bounds__(256) void k_pack_place(PackParams p) {
    __shared__ uint64_t lds[4];
    uint2 *head = reinterpret_cast<uint2 *>(p.out + p.l.head_off);
    uint64_t at = p.sums[blockIdx.x];
    for (uint32_t i = 0; i < kScanTiles; i += 256) {
        const uint64_t t = (uint64_t)blockIdx.x * kScanTiles + i + threadIdx.x;
        uint64_t total;
        const uint32_t v = t < p.l.tiles ? head[t].y : 0;
        const uint64_t x = block_scan(v, lds, total);
        if (t < p.l.tiles) head[t].y = (uint32_t)(at + x);
        at += total;
    }
}

// The lists, in position order, and the exponent bytes of the other tiles.
__global__ __launch_bounds__(256) void k_pack_extra(PackParams p) {
    const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const uint64_t tile = (uint64_t)blockIdx.x * 4 + wave;
    if (tile >= p.l.tiles) return;
    const uint2 head = reinterpret_cast<const uint2 *>(p.out + p.l.head_off)[tile];
    const uint32_t cnt = (head.x >> 8) & 0xFF;
    if (cnt == 0) return;
    uint16_t v[16];
    tile_gather(p, tile, lane, v);
    uint8_t *out = p.out + p.l.extra_off + (uint64_t)head.y * 16;
    if (cnt == kTileRaw) {
        uint32_t e[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 16; ++i) e[i >> 2] |= ((v[i] >> 7) & 0xFFu) << (8 * (i & 3));
        *reinterpret_cast<uint4 *>(out + lane * 16) = make_uint4(e[0], e[1], e[2], e[3]);
        return;
    }
    const uint32_t base = head.x & 0xFF, span = head.x & kTileZero ? 14 : 15;
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t e = (v[i] >> 7) & 0xFF;
        const bool coded = (e <= base && base - e <= span) || (e == 0 && (head.x & kTileZero));
        mine |= coded ? 0u : 1u << i;
    }
    uint32_t n = __popc(mine), before = n;
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t y = __shfl_up(before, d);
        if (lane >= (uint32_t)d) before += y;
    }
    uint32_t slot = before - n;
    uint32_t *list = reinterpret_cast<uint32_t *>(out);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (mine >> i & 1) list[slot++] = lane << 4 | i | (uint32_t)v[i] << 16;
    // the last unit's unused entries
    const uint32_t pad = (cnt + 3) / 4 * 4;
    if (lane >= cnt && lane < pad) list[lane] = 0;
}

__global__ __launch_bounds__(256) void k_unpack(UnpackParams p) {
    const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const uint64_t tile = (uint64_t)blockIdx.x * 4 + wave;
    if (tile >= p.tiles) return;
    Tile t;
    uint32_t v[8];
    tile_load(t, p.w, tile, tile_head(p.w, tile), lane);
    tile_decode(t, p.w, lane, v);
    const uint32_t q = lane >> 4, r = lane & 15;
    const uint64_t kb = tile % p.w.col_blocks, u = tile / p.w.col_blocks;
    const uint64_t rb = u % p.w.row_blocks, e = u / p.w.row_blocks;
    const uint64_t part = rb / p.w.part_blocks, row = (rb % p.w.part_blocks) * kTileRows + r;
    if (row >= p.w.part_rows) return;
    const uint64_t c0 = kb * kTileCols + q * 16;
    uint16_t *dst = p.out + e * p.matrix_stride + (part * p.w.part_rows + row) * p.row_stride + c0;
    if (c0 + 16 <= p.cols && (reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (c0 + i < p.cols) dst[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
}

// Rows copied to a stride of whole 16-byte units, zeros behind the last column.
__global__ __launch_bounds__(256) void k_stage(const uint16_t *in, uint64_t in_stride, uint16_t *out, uint64_t out_stride,
                                               uint64_t rows, uint64_t cols) {
    const uint64_t units = out_stride / 8, n = rows * units;
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (uint64_t)gridDim.x * 256) {
        const uint64_t row = i / units, c = i % units * 8;
        uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < cols) v[j >> 1] |= (uint32_t)in[row * in_stride + c + j] << (16 * (j & 1));
        *reinterpret_cast<uint4 *>(out + row * out_stride + c) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

// ---- activations ----------------------------------------------------------------

__device__ inline float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)

__device__ inline float activate(float z, uint32_t act) {
    switch (act) {
    case kActRelu: return z < 0 ? 0.0f : z;  // NaN stays
    case kActGelu: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    case kActGeluTanh: return 0.5f * z * (1.0f + tanhf(kGeluC * (z + 0.044715f * z * z * z)));
    case kActSilu: return z * sigmoid(z);
    default: return z;
    }
}

__device__ inline float activate_grad(float z, uint32_t act) {
    switch (act) {
    case kActRelu: return z > 0 ? 1.0f : 0.0f;
    case kActGelu:
        return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) + z * 0.3989422804014327f * expf(-0.5f * z * z);
    case kActGeluTanh: {
        const float t = tanhf(kGeluC * (z + 0.044715f * z * z * z));
        return 0.5f * (1.0f + t) + 0.5f * z * (1.0f - t * t) * kGeluC * (1.0f + 0.134145f * z * z);
    }
    case kActSilu: {
        const float s = sigmoid(z);
        return s * (1.0f + z * (1.0f - s));
    }
    default: return 1.0f;
    }
}

// ---- forward epilogue -----------------------------------------------------------

// Four consecutive outputs n .. n + 3 of one row, of which the first `count`
// exist.  All sums are in fp32; y and the kept pre-activation are each rounded
// once, from the unrounded values.
__device__ inline void load4(const void *p, uint64_t at, bool f32, bool vec, uint32_t count, float v[4]) {
    if (f32) {
        const float *s = static_cast<const float *>(p) + at;
        if (vec) {
            const f32x4 x = *reinterpret_cast<const f32x4 *>(s);
            for (int i = 0; i < 4; ++i) v[i] = x[i];
        } else {
            for (uint32_t i = 0; i < 4; ++i) v[i] = i < count ? s[i] : 0.0f;
        }
    } else {
        const uint16_t *s = static_cast<const uint16_t *>(p) + at;
        if (vec) {
            const uint2 x = *reinterpret_cast<const uint2 *>(s);
            v[0] = bf16_lo(x.x), v[1] = bf16_hi(x.x), v[2] = bf16_lo(x.y), v[3] = bf16_hi(x.y);
        } else {
            for (uint32_t i = 0; i < 4; ++i) v[i] = i < count ? from_bf16(s[i]) : 0.0f;
        }
    }
}

__device__ inline void store4(void *p, uint64_t at, bool f32, bool vec, uint32_t count, const float v[4]) {
    if (f32) {
        float *d = static_cast<float *>(p) + at;
        if (vec) {
            *reinterpret_cast<f32x4 *>(d) = f32x4{v[0], v[1], v[2], v[3]};
        } else {
            for (uint32_t i = 0; i < 4; ++i)
                if (i < count) d[i] = v[i];
        }
    } else {
        uint16_t *d = static_cast<uint16_t *>(p) + at;
        if (vec) {
            *reinterpret_cast<uint2 *>(d) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        } else {
            for (uint32_t i = 0; i < 4; ++i)
                if (i < count) d[i] = to_bf16(v[i]);
        }
    }
}

// z[0]: the product's values (gate rows when gated), z[1]: the up rows.
template <bool GATED>
__device__ inline void linear_out(const LinearEpi &e, uint64_t bias_at, uint32_t part_rows, uint64_t m, uint32_t n,
                                  float z[GATED ? 2 : 1][4]) {
    if (n >= part_rows) return;
    const uint32_t count = part_rows - n < 4 ? part_rows - n : 4;
    const bool vec = e.vec && count == 4;
#pragma unroll
    for (int h = 0; h < (GATED ? 2 : 1); ++h) {
        if (e.bias) {
            float b[4];
            load4(e.bias, bias_at + h * part_rows + n, e.bias_f32, vec, count, b);
            for (int i = 0; i < 4; ++i) z[h][i] += b[i];
        }
        if (e.preact) store4(e.preact, m * e.preact_stride + h * part_rows + n, e.preact_f32, vec, count, z[h]);
    }
    float y[4];
    if (GATED) {
        for (int i = 0; i < 4; ++i) y[i] = z[0][i] * sigmoid(z[0][i]) * z[GATED ? 1 : 0][i];
    } else {
        for (int i = 0; i < 4; ++i) y[i] = activate(z[0][i], e.act);
    }
    if (e.residual) {
        float r[4];
        load4(e.residual, m * e.residual_stride + n, e.y_f32, vec, count, r);
        for (int i = 0; i < 4; ++i) y[i] += r[i];
    }
    store4(e.y, m * e.y_stride + n, e.y_f32, vec, count, y);
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

// ---- few rows ---------------------------------------------------------------------

// y = W x for up to 16 MT rows of x at a time.  A workgroup owns RB row blocks
// of W; its waves split K and add their parts in LDS in a fixed order.  The
// weights go from memory to the matrix instructions without touching LDS.
template <int MT, int RB, bool GATED, int NW>
__global__ __launch_bounds__(NW * 64) void k_skinny(SkinnyParams p) {
    __shared__ f32x4 part[NW][RB * MT * 64];
    const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const uint32_t q = lane >> 4, r = lane & 15;
    uint32_t begin, end;
    group_rows(p.offsets, blockIdx.y, p.tokens, begin, end);
    const uint32_t KB = p.w.col_blocks;
    uint64_t tile0[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        uint32_t b = GATED ? blockIdx.x * (RB / 2) + i / 2 : blockIdx.x * RB + i;
        if (b >= p.w.part_blocks) b = p.w.part_blocks - 1;  // computed and dropped
        if (GATED && (i & 1)) b += p.w.part_blocks;
        tile0[i] = ((uint64_t)blockIdx.y * p.w.row_blocks + b) * KB;
    }
    for (uint32_t m0 = begin; m0 < end; m0 += 16 * MT) {
        f32x4 acc[RB][MT];
#pragma unroll
        for (int i = 0; i < RB; ++i)
            for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
        const uint16_t *xr[MT];
        bool xv[MT];
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const uint32_t m = m0 + j * 16 + r;
            xv[j] = m < end;
            xr[j] = static_cast<const uint16_t *>(p.x.p) + (uint64_t)(xv[j] ? m : begin) * p.x.stride;
        }
        Tile t[RB];
        uint2 hd[RB];
        uint4 x[MT][2];
        auto load_x = [&](uint32_t kb) {
            const uint32_t k = kb * kTileCols + q * 16;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    x[j][h] = make_uint4(0, 0, 0, 0);
                    const uint32_t kk = k + h * 8;
                    if (p.x_vec) {
                        if (xv[j] && kk < p.cols) x[j][h] = *reinterpret_cast<const uint4 *>(xr[j] + kk);
                    } else if (xv[j]) {
                        uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (kk + i < p.cols) u[i >> 1] |= (uint32_t)xr[j][kk + i] << (16 * (i & 1));
                        x[j][h] = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                }
            }
        };
        if (wave < KB) {
#pragma unroll
            for (int i = 0; i < RB; ++i) tile_load(t[i], p.w, tile0[i] + wave, tile_head(p.w, tile0[i] + wave), lane);
            load_x(wave);
            if (wave + NW < KB)
#pragma unroll
                for (int i = 0; i < RB; ++i) hd[i] = tile_head(p.w, tile0[i] + wave + NW);
        }
        for (uint32_t kb = wave; kb < KB; kb += NW) {
            Tile c[RB];
            uint4 xc[MT][2];
#pragma unroll
            for (int i = 0; i < RB; ++i) c[i] = t[i];
#pragma unroll
            for (int j = 0; j < MT; ++j) xc[j][0] = x[j][0], xc[j][1] = x[j][1];
            if (kb + NW < KB) {
#pragma unroll
                for (int i = 0; i < RB; ++i) tile_load(t[i], p.w, tile0[i] + kb + NW, hd[i], lane);
                load_x(kb + NW);
                if (kb + 2 * NW < KB)
#pragma unroll
                    for (int i = 0; i < RB; ++i) hd[i] = tile_head(p.w, tile0[i] + kb + 2 * NW);
            }
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                uint32_t v[8];
                tile_decode(c[i], p.w, lane, v);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bf16x8 a = __builtin_bit_cast(bf16x8, u32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]});
#pragma unroll
                    for (int j = 0; j < MT; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, xc[j][h]),
                                                                            acc[i][j], 0, 0, 0);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < RB; ++i)
            for (int j = 0; j < MT; ++j) part[wave][(i * MT + j) * 64 + lane] = acc[i][j];
        __syncthreads();
        // a thread finishes four outputs of one row (and their up rows): element u of the result list
        constexpr int STEP = GATED ? 2 : 1;
        for (uint32_t u = threadIdx.x; u < RB / STEP * MT * 64; u += NW * 64) {
            const uint32_t l = u & 63, j = (u >> 6) % MT, i = (u >> 6) / MT * STEP;
            float z[STEP][4];
#pragma unroll
            for (int h = 0; h < STEP; ++h) {
                f32x4 s = part[0][((i + h) * MT + j) * 64 + l];
                for (int g = 1; g < NW; ++g) s += part[g][((i + h) * MT + j) * 64 + l];
                for (int d = 0; d < 4; ++d) z[h][d] = s[d];
            }
            const uint32_t b = GATED ? blockIdx.x * (RB / 2) + i / 2 : blockIdx.x * RB + i;
            const uint32_t m = m0 + j * 16 + (l & 15);
            if (m < end && b < p.w.part_blocks)
                linear_out<GATED>(p.lin, (uint64_t)blockIdx.y * p.rows, p.w.part_rows, m, b * 16 + (l >> 4) * 4, z);
        }
        __syncthreads();
    }
}

// ---- tiled products -----------------------------------------------------------------
//
// C[r][c] = sum over a of R[r][a] S[c][a], the result stored with r contiguous.
// forward, loss: r = weight row, c = token,      a = column of x
// dx:            r = column of x, c = token,     a = weight row
// dw:            r = column of x, c = weight row, a = token
//
// The operands of each block of 64 contraction values are staged in LDS, two
// blocks deep: while one is multiplied, the next is decoded or copied from
// registers, and the one after it is on its way from memory.

enum Operand { kPacked, kPackedT, kRows, kCols };

// Place of 16-byte unit `unit` of row `row` in a [TC][64] operand (128-byte
// rows): the xor spreads the 16 rows that a read touches over the banks.
__device__ inline uint32_t rows_at(uint32_t row, uint32_t unit) { return row * 128 + ((unit ^ (row & 7)) * 16); }

// Place of the 32-byte granule `g` of contraction row `a` in a [64][T]
// operand that is read transposed.  A transposing read takes four consecutive
// rows a of two quads 16 rows apart: these eight get eight different granules
// of the 256 bytes that the banks span.
template <int T>
__device__ inline uint32_t cols_at(uint32_t a, uint32_t g) {
    const uint32_t s = (a & 3) | ((a >> 2 ^ a >> 4) & 1) << 2;
    return a * (T * 2) + ((g ^ s) * 32);
}

// Eight contraction values of column c0 + (lane & 15): a = 16 q + 8 h + j.
template <int T>
__device__ inline bf16x8 cols_frag(const uint8_t *lds, uint32_t c0, uint32_t h, uint32_t lane) {
    const uint32_t q = lane >> 4, l = lane & 15;
    s16x4 v[2];
#pragma unroll
    for (uint32_t t = 0; t < 2; ++t) {
        const uint32_t a = q * 16 + h * 8 + t * 4 + (l >> 2);
        const uint8_t *p = lds + cols_at<T>(a, c0 >> 4) + (l & 3) * 8;
        v[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)p);
    }
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    const s16x8 x = __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, x);
}

// Expert and first row of token tile `ct`, or false behind the last one.
// Uniform over the wave; every wave of a workgroup finds the same.
__device__ inline bool find_group(const GemmParams &p, uint32_t ct, uint32_t edge, uint32_t lane, uint32_t &g,
                                  uint32_t &row, uint32_t &end) {
    if (!p.offsets) {
        g = 0;
        row = ct * edge;
        end = p.tokens;
        return row < end;
    }
    uint32_t before = 0;
    for (uint32_t g0 = 0; g0 < p.groups; g0 += 64) {
        uint32_t b = 0, e = 0;
        if (g0 + lane < p.groups) group_rows(p.offsets, g0 + lane, p.tokens, b, e);
        const uint32_t n = (e - b + edge - 1) / edge;
        uint32_t x = n;
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t y = __shfl_up(x, d);
            if (lane >= (uint32_t)d) x += y;
        }
        const uint64_t hit = __ballot(n != 0 && ct < before + x);
        if (hit) {
            const uint32_t l = __builtin_ctzll(hit);
            g = g0 + l;
            const uint32_t first = before + __builtin_amdgcn_readlane(x, l) - __builtin_amdgcn_readlane(n, l);
            row = __builtin_amdgcn_readlane(b, l) + (ct - first) * edge;
            end = __builtin_amdgcn_readlane(e, l);
            return true;
        }
        before += __builtin_amdgcn_readlane(x, 63);
    }
    return false;
}

template <Operand RK, int TR, int WAVES>
struct RSide {  // the operand whose index is contiguous in the output
    static constexpr int TILES = TR * 64 / 1024 / WAVES;  // packed tiles a wave decodes
    static constexpr int UNITS = TR * 64 / 8 / (WAVES * 64);
    Tile t[RK == kCols ? 1 : TILES];
    uint2 hd[RK == kCols ? 1 : TILES];
    bool live[RK == kCols ? 1 : TILES];
    uint4 u[RK == kCols ? UNITS : 1];
};

template <Operand RK, Operand CK, GemmKind KIND, bool GATED, int TR, int TC, int WR, int WC>
__global__ __launch_bounds__(WR *WC * 64) void k_gemm(GemmParams p) {
    constexpr int WAVES = WR * WC, THREADS = WAVES * 64;
    constexpr int FR = TR / WR / 16, FC = TC / WC / 16;
    constexpr int RBYTES = TR * 128, CBYTES = TC * 128;
    constexpr int CUNITS = TC * 8 / THREADS;
    __shared__ __align__(16) uint8_t lds[2 * (RBYTES + CBYTES)];
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const uint32_t q = lane >> 4, l15 = lane & 15;
    const uint32_t wr = wave % WR, wc = wave / WR;

    // Workgroups go to the 8 XCDs in turn: give each XCD a run of neighbouring
    // tiles, four column tiles wide, so that its L2 holds what they share.
    const uint32_t total = p.r_tiles * p.c_tiles;
    uint32_t id = blockIdx.x;
    {
        const uint32_t x = id & 7, i = id >> 3, full = total >> 3, rest = total & 7;
        id = x * full + min(x, rest) + i;
    }
    uint32_t rt, ct;
    {
        const uint32_t band = 4 * p.r_tiles, b = id / band, first = b * 4;
        const uint32_t wide = min(4u, p.c_tiles - first), j = id - b * band;
        ct = first + j % wide;
        rt = j / wide;
    }

    uint32_t g = 0, c0, c_end, a0 = 0, a_end = 0;
    if (KIND == kGemmDw) {
        g = blockIdx.y;
        group_rows(p.offsets, g, p.tokens, a0, a_end);
        c0 = ct * TC;
        c_end = p.c_limit;
    } else {
        if (!find_group(p, ct, TC, lane, g, c0, c_end)) return;
        g = uniform(g);
        c0 = uniform(c0);
        c_end = uniform(c_end);
    }
    const uint32_t steps = KIND == kGemmDw ? (a_end - a0 + 63) / 64 : p.steps;

    RSide<RK, TR, WAVES> R;
    uint4 cu[CUNITS];
    const uint32_t KB = p.w.col_blocks;

    // place of the wave's i-th packed tile: forward: 16-row block of the tile; dx: (row block, column block)
    auto tile_index = [&](int i, uint32_t s, bool &live) -> uint64_t {
        const uint32_t j = wave * R.TILES + i;
        uint32_t rb, kb;
        if (RK == kPacked) {
            if (GATED) {
                rb = rt * (TR / 32) + (j >> 1);
                live = rb < p.w.part_blocks;
                rb = live ? rb + (j & 1 ? p.w.part_blocks : 0) : 0;
            } else {
                rb = rt * (TR / 16) + j;
                live = rb < p.row_blocks;
                rb = live ? rb + p.row_block0 : 0;
            }
            kb = s;
        } else {
            rb = s * 4 + (j & 3);
            kb = rt * (TR / 64) + (j >> 2);
            live = rb < p.row_blocks && kb < KB;
            rb = live ? rb + p.row_block0 : 0;
            kb = live ? kb : 0;
        }
        return ((uint64_t)g * p.w.row_blocks + rb) * KB + kb;
    };
    auto load_heads = [&](uint32_t s) {
        if constexpr (RK != kCols) {
#pragma unroll
            for (int i = 0; i < R.TILES; ++i) {
                bool live;
                R.hd[i] = tile_head(p.w, tile_index(i, s, live));
            }
        }
    };
    auto load_cols = [&](const Mat &m, uint32_t s, uint32_t x0, uint32_t limit, uint4 *u, int units, int width) {
        // [64 rows][width columns] of a matrix whose rows are the contraction
        for (int i = 0; i < units; ++i) {
            const uint32_t j = i * THREADS + tid, row = j / (width / 8), c = x0 + j % (width / 8) * 8;
            const uint32_t a = a0 + s * 64 + row;
            u[i] = make_uint4(0, 0, 0, 0);
            if (a < a_end && c < limit)
                u[i] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(m.p) + (uint64_t)a * m.stride + c);
        }
    };
    auto load = [&](uint32_t s) {
        if constexpr (RK == kCols) {
            load_cols(p.rmat, s, rt * TR, p.r_limit, R.u, R.UNITS, TR);
        } else {
#pragma unroll
            for (int i = 0; i < R.TILES; ++i) {
                bool live;
                const uint64_t t = tile_index(i, s, live);
                tile_load(R.t[i], p.w, t, R.hd[i], lane);
                R.live[i] = live;
            }
        }
        if constexpr (CK == kCols) {
            load_cols(p.cmat, s, c0, p.c_limit, cu, CUNITS, TC);
        } else {
#pragma unroll
            for (int i = 0; i < CUNITS; ++i) {
                const uint32_t j = i * THREADS + tid, row = c0 + (j >> 3), a = s * 64 + (j & 7) * 8;
                cu[i] = make_uint4(0, 0, 0, 0);
                if (row < c_end && a < p.c_limit)
                    cu[i] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.cmat.p) +
                                                             (uint64_t)row * p.cmat.stride + a);
            }
        }
    };
    auto stage = [&](uint8_t *rl, uint8_t *cl) {
        if constexpr (RK == kCols) {
#pragma unroll
            for (int i = 0; i < R.UNITS; ++i) {
                const uint32_t j = i * THREADS + tid, row = j / (TR / 8), c = j % (TR / 8);
                *reinterpret_cast<uint4 *>(rl + cols_at<TR>(row, c >> 1) + (c & 1) * 16) = R.u[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < R.TILES; ++i) {
                const uint32_t j = wave * R.TILES + i;
                uint32_t v[8];
                tile_decode(R.t[i], p.w, lane, v);
                if (!R.live[i])
                    for (int d = 0; d < 8; ++d) v[d] = 0;
                const uint4 a = make_uint4(v[0], v[1], v[2], v[3]), b = make_uint4(v[4], v[5], v[6], v[7]);
                if constexpr (RK == kPacked) {
                    *reinterpret_cast<uint4 *>(rl + j * 2048 + lane * 16) = a;
                    *reinterpret_cast<uint4 *>(rl + j * 2048 + 1024 + lane * 16) = b;
                } else {
                    const uint32_t row = (j & 3) * 16 + l15, flip = (lane >> 3 & 1) * 16;
                    uint8_t *d = rl + cols_at<TR>(row, (j >> 2) * 4 + q);
                    *reinterpret_cast<uint4 *>(d + flip) = flip ? b : a;
                    *reinterpret_cast<uint4 *>(d + (16 - flip)) = flip ? a : b;
                }
            }
        }
        if constexpr (CK == kCols) {
#pragma unroll
            for (int i = 0; i < CUNITS; ++i) {
                const uint32_t j = i * THREADS + tid, row = j / (TC / 8), c = j % (TC / 8);
                *reinterpret_cast<uint4 *>(cl + cols_at<TC>(row, c >> 1) + (c & 1) * 16) = cu[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < CUNITS; ++i) {
                const uint32_t j = i * THREADS + tid;
                *reinterpret_cast<uint4 *>(cl + rows_at(j >> 3, j & 7)) = cu[i];
            }
        }
    };

    f32x4 acc[FR][FC];
#pragma unroll
    for (int i = 0; i < FR; ++i)
        for (int j = 0; j < FC; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    auto multiply = [&](const uint8_t *rl, const uint8_t *cl) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            bf16x8 cf[FC];
#pragma unroll
            for (int j = 0; j < FC; ++j) {
                const uint32_t col = (wc * FC + j) * 16;
                if constexpr (CK == kCols)
                    cf[j] = cols_frag<TC>(cl, col, h, lane);
                else
                    cf[j] = *reinterpret_cast<const bf16x8 *>(cl + rows_at(col + l15, q * 2 + h));
            }
#pragma unroll
            for (int i = 0; i < FR; ++i) {
                bf16x8 rf;
                if constexpr (RK == kPacked)
                    rf = *reinterpret_cast<const bf16x8 *>(rl + (wr * FR + i) * 2048 + h * 1024 + lane * 16);
                else
                    rf = cols_frag<TR>(rl, (wr * FR + i) * 16, h, lane);
#pragma unroll
                for (int j = 0; j < FC; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(rf, cf[j], acc[i][j], 0, 0, 0);
            }
        }
    };

    if (steps > 0) {
        load_heads(0);
        load(0);
        if (steps > 1) load_heads(1);
        stage(lds, lds + 2 * RBYTES);
        if (steps > 1) load(1);
        if (steps > 2) load_heads(2);
        lds_barrier();
        for (uint32_t s = 0; s < steps; ++s) {
            const uint32_t b = s & 1;
            if (s + 1 < steps) stage(lds + (b ^ 1) * RBYTES, lds + 2 * RBYTES + (b ^ 1) * CBYTES);
            if (s + 2 < steps) load(s + 2);
            if (s + 3 < steps) load_heads(s + 3);
            multiply(lds + b * RBYTES, lds + 2 * RBYTES + b * CBYTES);
            lds_barrier();
        }
    }

    // ---- epilogues: acc[i][j][d] is row r0 + 16 i + 4 q + d, column cc0 + 16 j + l15 ----
    const uint32_t cc0 = c0 + wc * FC * 16 + l15;
    if constexpr (KIND == kGemmForward) {
#pragma unroll
        for (int j = 0; j < FC; ++j) {
            const uint32_t m = cc0 + j * 16;
            if (m >= c_end) continue;
            const uint64_t bias_at = (uint64_t)g * p.rows;
            if constexpr (GATED) {
#pragma unroll
                for (int i = 0; i < FR; i += 2) {
                    const uint32_t n = (rt * (TR / 32) + (wr * FR + i) / 2) * 16 + q * 4;
                    float z[2][4];
                    for (int d = 0; d < 4; ++d) z[0][d] = acc[i][j][d], z[1][d] = acc[i + 1][j][d];
                    linear_out<true>(p.lin, bias_at, p.w.part_rows, m, n, z);
                }
            } else {
#pragma unroll
                for (int i = 0; i < FR; ++i) {
                    const uint32_t n = (rt * (TR / 16) + wr * FR + i) * 16 + q * 4;
                    float z[1][4];
                    for (int d = 0; d < 4; ++d) z[0][d] = acc[i][j][d];
                    linear_out<false>(p.lin, bias_at, p.w.part_rows, m, n, z);
                }
            }
        }
    } else if constexpr (KIND == kGemmLossStat) {
        // every token's largest logit in this tile, and the sum of exp(logit - that)
        f32x2 *red = reinterpret_cast<f32x2 *>(lds);  // [WR][TC]
#pragma unroll
        for (int j = 0; j < FC; ++j) {
            const uint32_t m = cc0 + j * 16;
            const bool live = m < c_end;
            const int64_t want = live ? p.loss.target[m] : -1;
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < FR; ++i)
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const uint32_t n = rt * TR + (wr * FR + i) * 16 + q * 4 + d;
                    if (n >= p.rows) acc[i][j][d] = -INFINITY;
                    if (live && (int64_t)n == want && n < p.rows) p.loss.picked[m] = acc[i][j][d];
                    top = fmaxf(top, acc[i][j][d]);
                }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            // a finite reference, whatever the logits: exp of -inf, +inf and NaN then say what they should
            const float ref = fminf(fmaxf(top, -3.0e38f), 3.0e38f);
            float sum = 0;
#pragma unroll
            for (int i = 0; i < FR; ++i)
#pragma unroll
                for (int d = 0; d < 4; ++d) sum += __expf(acc[i][j][d] - ref);
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (q == 0) red[wr * TC + (wc * FC + j) * 16 + l15] = f32x2{ref, sum};
        }
        __syncthreads();
        for (uint32_t c = tid; c < TC; c += THREADS) {
            if (c0 + c >= c_end) continue;
            float ref = red[c][0];
            for (int w = 1; w < WR; ++w) ref = fmaxf(ref, red[w * TC + c][0]);
            float sum = 0;
            for (int w = 0; w < WR; ++w) sum += red[w * TC + c][1] * __expf(red[w * TC + c][0] - ref);
            p.loss.part[(uint64_t)rt * p.tokens + c0 + c] = make_float2(ref, sum);
        }
    } else if constexpr (KIND == kGemmLossDz) {
        // g (softmax - one at the target), rounded to bf16 for the two products that follow; zero behind the last row
#pragma unroll
        for (int j = 0; j < FC; ++j) {
            const uint32_t m = cc0 + j * 16;
            if (m >= c_end) continue;
            const int64_t want = p.loss.target[m];
            const bool counts = want != p.loss.ignore && want >= 0 && want < (int64_t)p.rows;
            const float gr = counts ? p.loss.dloss[m] : 0.0f, lse = p.loss.lse[m];
#pragma unroll
            for (int i = 0; i < FR; ++i) {
                const uint32_t at = rt * TR + (wr * FR + i) * 16 + q * 4;
                float z[4];
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const uint32_t n = p.row_block0 * 16 + at + d;
                    float v = __expf(acc[i][j][d] - lse);
                    if ((int64_t)n == want) v -= 1.0f;
                    z[d] = n < p.rows && counts ? gr * v : 0.0f;
                }
                store4(p.loss.dz, (uint64_t)m * p.loss.dz_stride + at, false, true, 4, z);
            }
        }
    } else {
        const StoreEpi &e = p.store;
        const uint32_t r_end = p.cols;
#pragma unroll
        for (int j = 0; j < FC; ++j) {
            const uint32_t c = cc0 + j * 16;
            uint64_t row = c;
            if constexpr (KIND == kGemmDw) {
                // padded row of the stack's part -> row of the matrix; pieces start at row_block0
                const uint32_t n = c + p.row_block0 * 16, pad = p.w.part_blocks * 16, part = n / pad, in = n - part * pad;
                if (in >= p.w.part_rows || part >= p.w.parts || c >= p.row_blocks * 16) continue;
                row = (uint64_t)g * p.rows + (uint64_t)part * p.w.part_rows + in;
            } else {
                if (c >= c_end) continue;
            }
#pragma unroll
            for (int i = 0; i < FR; ++i) {
                const uint32_t r = rt * TR + (wr * FR + i) * 16 + q * 4;
                if (r >= r_end) continue;
                const uint32_t count = r_end - r < 4 ? r_end - r : 4;
                float v[4];
                for (int d = 0; d < 4; ++d) v[d] = acc[i][j][d];
                if (e.sum) {
                    const bool sv = count == 4;  // the sums' stride is a multiple of four
                    if (e.add) {
                        float o[4];
                        load4(e.sum, row * e.sum_stride + r, true, sv, count, o);
                        for (int d = 0; d < 4; ++d) v[d] += o[d];
                    }
                    if (!e.out) store4(e.sum, row * e.sum_stride + r, true, sv, count, v);
                }
                if (e.out) store4(e.out, row * e.stride + r, false, e.vec && count == 4, count, v);
            }
        }
    }
}

// ---- the loss's join -------------------------------------------------------------

// A wave per token: reference and sum over the row tiles, in a fixed order.
__global__ __launch_bounds__(256) void k_loss_join(LossEpi e, float *loss, float *lse, uint32_t tokens, uint32_t parts,
                                                   uint64_t vocab) {
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t m = blockIdx.x * 4 + uniform(threadIdx.x >> 6);
    if (m >= tokens) return;
    float ref = -3.0e38f, sum = 0;
    for (uint32_t i = lane; i < parts; i += 64) {
        const float2 v = e.part[(uint64_t)i * tokens + m];
        const float top = fmaxf(ref, v.x);
        sum = sum * expf(ref - top) + v.y * expf(v.x - top);
        ref = top;
    }
    for (int d = 1; d < 64; d <<= 1) {
        const float r2 = __shfl_xor(ref, d), s2 = __shfl_xor(sum, d), top = fmaxf(ref, r2);
        // the same order of the two on both lanes
        const float a = (lane & d) ? s2 * expf(r2 - top) : sum * expf(ref - top);
        const float b = (lane & d) ? sum * expf(ref - top) : s2 * expf(r2 - top);
        sum = a + b;
        ref = top;
    }
    if (lane == 0) {
        const float z = sum == 0.0f ? -INFINITY : ref + logf(sum);
        const int64_t t = e.target[m];
        lse[m] = z;
        loss[m] = t == e.ignore ? 0.0f : t >= 0 && t < (int64_t)vocab ? z - e.picked[m] : NAN;
    }
}

// ---- the pre-activation's gradient --------------------------------------------------

__device__ inline float read1(const void *p, uint64_t at, bool f32) {
    return f32 ? static_cast<const float *>(p)[at] : from_bf16(static_cast<const uint16_t *>(p)[at]);
}

// dz = dy act'(z) in the padded column order of the packed rows, and the sums
// of its columns over a run of the group's rows, from the unrounded values.
// A thread takes eight columns (of both halves when gated).
template <bool GATED>
__global__ __launch_bounds__(256) void k_dz(DzParams p) {
    constexpr int H = GATED ? 2 : 1;
    __shared__ float red[3][H][64][9];
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t c = (blockIdx.x * 64 + lane) * 8;
    uint32_t begin, end;
    group_rows(p.offsets, blockIdx.z, p.tokens, begin, end);
    const uint32_t each = (end - begin + p.chunks - 1) / p.chunks;
    const uint32_t m0 = begin + min(blockIdx.y * each, end - begin), m1 = min(m0 + each, end);
    // columns behind the last part only hold zeros
    const bool tail = GATED && c >= p.part_pad;
    const uint32_t at = tail ? c + p.part_pad : c;
    float sum[H][8];
#pragma unroll
    for (int h = 0; h < H; ++h)
        for (int i = 0; i < 8; ++i) sum[h][i] = 0;
    if (at < p.width) {
        for (uint32_t m = m0 + wave; m < m1; m += 4) {
            float v[H][8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool live = !tail && c + i < p.part_rows;
                const float dy = live ? read1(p.dy, m * p.dy_stride + c + i, p.dy_f32) : 0.0f;
                const uint64_t z = m * p.z_stride + c + i;
                if (GATED) {
                    const float a = live ? read1(p.z, z, p.z_f32) : 0.0f;
                    const float b = live ? read1(p.z, z + p.part_rows, p.z_f32) : 0.0f;
                    const float s = sigmoid(a);
                    v[0][i] = live ? dy * b * s * (1.0f + a * (1.0f - s)) : 0.0f;
                    v[H - 1][i] = live ? dy * a * s : 0.0f;
                } else {
                    v[0][i] = dy;
                    if (p.act != kActNone && live)
                        v[0][i] = dy * activate_grad(read1(p.z, z, p.z_f32), p.act);
                }
            }
#pragma unroll
            for (int h = 0; h < H; ++h) {
                for (int i = 0; i < 8; ++i) sum[h][i] += v[h][i];
                if (p.dz && (h == 0 || !tail))
                    *reinterpret_cast<uint4 *>(p.dz + (uint64_t)m * p.dz_stride + at + h * p.part_pad) =
                        make_uint4(pack_bf16(v[h][0], v[h][1]), pack_bf16(v[h][2], v[h][3]), pack_bf16(v[h][4], v[h][5]),
                                   pack_bf16(v[h][6], v[h][7]));
            }
        }
    }
    if (!p.colsum) return;
    if (wave)
        for (int h = 0; h < H; ++h)
            for (int i = 0; i < 8; ++i) red[wave - 1][h][lane][i] = sum[h][i];
    __syncthreads();
    if (wave || tail || at >= p.width) return;
    float *out = p.colsum + ((uint64_t)blockIdx.z * p.chunks + blockIdx.y) * p.width;
    for (int h = 0; h < H; ++h)
        for (int i = 0; i < 8; ++i)
            out[at + h * p.part_pad + i] = ((sum[h][i] + red[0][h][lane][i]) + red[1][h][lane][i]) + red[2][h][lane][i];
}

__global__ __launch_bounds__(256) void k_dbias(DzParams p) {
    const uint32_t n = blockIdx.x * 256 + threadIdx.x, g = blockIdx.y;
    if (n >= p.part_rows * p.parts) return;
    const uint32_t part = n / p.part_rows, at = part * p.part_pad + n - part * p.part_rows;
    float s = 0;
    for (uint32_t i = 0; i < p.chunks; ++i) s += p.colsum[((uint64_t)g * p.chunks + i) * p.width + at];
    const uint64_t o = (uint64_t)g * p.part_rows * p.parts + n;
    if (p.dbias_f32)
        static_cast<float *>(p.dbias)[o] = s;
    else
        static_cast<uint16_t *>(p.dbias)[o] = to_bf16(s);
}

template <int MT, int RB, bool GATED, int NW>
hipError_t skinny(const SkinnyParams &p, hipStream_t s) {
    const uint32_t per = GATED ? RB / 2 : RB;
    const dim3 grid((p.w.part_blocks + per - 1) / per, p.groups);
    k_skinny<MT, RB, GATED, NW><<<grid, NW * 64, 0, s>>>(p);
    return hipGetLastError();
}

template <Operand RK, Operand CK, GemmKind KIND, bool GATED>
hipError_t gemm(uint32_t edge, const GemmParams &p, hipStream_t s) {
    const dim3 grid(p.r_tiles * p.c_tiles, KIND == kGemmDw ? p.groups : 1);
    if (edge == 256)
        k_gemm<RK, CK, KIND, GATED, 256, 256, 2, 4><<<grid, 512, 0, s>>>(p);
    else
        k_gemm<RK, CK, KIND, GATED, 128, 128, 2, 2><<<grid, 256, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_pack(const PackParams &p, hipStream_t s) {
    const uint32_t wgs = (uint32_t)((p.l.tiles + 3) / 4), blocks = (uint32_t)((p.l.tiles + kScanTiles - 1) / kScanTiles);
    k_pack<<<wgs, 256, 0, s>>>(p);
    k_pack_sums<<<blocks, 256, 0, s>>>(p);
    k_pack_scan<<<1, 256, 0, s>>>(p);
    k_pack_place<<<blocks, 256, 0, s>>>(p);
    k_pack_extra<<<wgs, 256, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_unpack(const UnpackParams &p, hipStream_t s) {
    k_unpack<<<(uint32_t)((p.tiles + 3) / 4), 256, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_stage(const uint16_t *in, uint64_t in_stride, uint16_t *out, uint64_t out_stride, uint64_t rows,
                        uint64_t cols, hipStream_t s) {
    const uint64_t units = rows * (out_stride / 8), wgs = (units + 255) / 256;
    if (wgs == 0) return hipSuccess;
    k_stage<<<(uint32_t)(wgs < 8192 ? wgs : 8192), 256, 0, s>>>(in, in_stride, out, out_stride, rows, cols);
    return hipGetLastError();
}

bool skinny_fits(uint64_t tokens, uint64_t groups) { return groups == 1 ? tokens <= 64 : tokens <= 16 * groups; }

hipError_t launch_skinny(const SkinnyParams &p, hipStream_t s) {
    const bool one = p.groups > 1 || p.tokens <= 16;
    if (p.lin.act == kActSwiglu) {
        if (one) return skinny<1, 2, true, 8>(p, s);
        return p.tokens <= 32 ? skinny<2, 2, true, 8>(p, s) : skinny<4, 2, true, 8>(p, s);
    }
    if (one) return skinny<1, 1, false, 16>(p, s);
    return p.tokens <= 32 ? skinny<2, 1, false, 16>(p, s) : skinny<4, 2, false, 8>(p, s);
}

uint32_t gemm_edge(uint64_t r, uint64_t c, uint64_t groups) {
    return ((r + 255) / 256) * ((c + 255) / 256) * groups >= 256 ? 256 : 128;
}

hipError_t launch_gemm(GemmKind kind, uint32_t edge, const GemmParams &p, hipStream_t s) {
    if (p.r_tiles == 0 || p.c_tiles == 0) return hipSuccess;
    switch (kind) {
    case kGemmForward:
        return p.lin.act == kActSwiglu ? gemm<kPacked, kRows, kGemmForward, true>(edge, p, s)
                                       : gemm<kPacked, kRows, kGemmForward, false>(edge, p, s);
    case kGemmLossStat: return gemm<kPacked, kRows, kGemmLossStat, false>(edge, p, s);
    case kGemmLossDz: return gemm<kPacked, kRows, kGemmLossDz, false>(edge, p, s);
    case kGemmDx: return gemm<kPackedT, kRows, kGemmDx, false>(edge, p, s);
    case kGemmDw: return gemm<kCols, kCols, kGemmDw, false>(edge, p, s);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_loss_join(const LossEpi &e, float *loss, float *lse, uint32_t tokens, uint32_t parts, uint64_t vocab,
                            hipStream_t s) {
    k_loss_join<<<(tokens + 3) / 4, 256, 0, s>>>(e, loss, lse, tokens, parts, vocab);
    return hipGetLastError();
}

hipError_t launch_dz(const DzParams &p, hipStream_t s) {
    const uint32_t cols = p.parts == 2 ? p.part_pad + (p.width - 2 * p.part_pad) : p.width;
    const dim3 grid((cols / 8 + 63) / 64, p.chunks, p.groups);
    if (p.parts == 2)
        k_dz<true><<<grid, 256, 0, s>>>(p);
    else
        k_dz<false><<<grid, 256, 0, s>>>(p);
    if (p.dbias) k_dbias<<<dim3((p.part_rows * p.parts + 255) / 256, p.groups), 256, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace uzip
