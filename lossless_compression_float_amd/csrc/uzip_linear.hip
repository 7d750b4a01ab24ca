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
// both operands agree; here, in half h of a block of 64, it is 32 h + 8 q + j,
// the order of a packed tile.
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

// ---- packing ------------------------------------------------------------------

// This lane's 16 values of a tile, zero outside the matrix.
__device__ inline void tile_gather(const PackParams &p, uint64_t tile, uint32_t lane, uint16_t v[16]) {
    const uint32_t q = lane >> 4, r = lane & 15;
    const uint64_t kb = tile % p.l.col_blocks, t = tile / p.l.col_blocks;
    const uint64_t rb = t % p.l.row_blocks, e = t / p.l.row_blocks;
    const uint64_t part = rb / p.l.part_blocks, row = (rb % p.l.part_blocks) * kTileRows + r;
    const uint64_t c0 = kb * kTileCols + q * 8;
    const uint16_t *src = p.in + e * p.matrix_stride + (part * p.l.part_rows + row) * p.row_stride + c0;
    if (row < p.l.part_rows && c0 + 40 <= p.cols) {
        const u32x4 a[2] = {*reinterpret_cast<const u32x4_any *>(src), *reinterpret_cast<const u32x4_any *>(src + 32)};
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = (uint16_t)(a[i >> 3][i >> 1 & 3] >> (16 * (i & 1)));
        return;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t c = (i >> 3) * 32 + (i & 7);
        v[i] = row < p.l.part_rows && c0 + c < p.cols ? src[c] : (uint16_t)0;
    }
}

// A wave packs a tile.  Its window is the one that holds most of its exponents
// and, of those, has the highest base: where all lie within 16 and none is 0
// (19 of 20 tiles of normal weights), the lowest says it; else their histogram,
// whose LDS atomics meet at a few addresses (taken for every tile, 28672 x 4096
// took 224 us instead of 87, 4.7 TB/s).
__global__ __launch_bounds__(256) void k_pack(PackParams p) {
    __shared__ uint32_t hist[4][256 + 16];
    const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const uint64_t tile = (uint64_t)blockIdx.x * 4 + wave;
    if (tile >= p.l.tiles) return;
    uint16_t v[16];
    tile_gather(p, tile, lane, v);
    uint32_t low = 255, high = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t e = (v[i] >> 7) & 0xFF;
        low = min(low, e);
        high = max(high, e);
    }
    for (int d = 32; d; d >>= 1) {
        low = min(low, (uint32_t)__shfl_xor((int)low, d));
        high = max(high, (uint32_t)__shfl_xor((int)high, d));
    }
    low = uniform(low);
    high = uniform(high);
    uint32_t base = min(low + 15, 255u), zero = 0, outside = 0;
    if (low == 0 || high - low > 15) {
        uint32_t *h = hist[wave];
        for (uint32_t i = lane; i < 272; i += 64) h[i] = 0;
        __builtin_amdgcn_s_waitcnt(0);
        __builtin_amdgcn_wave_barrier();
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
        base = (best >> 1) & 0xFF;
        zero = !(best & 1);
        outside = 1024 - (best >> 10);
    }
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
        reinterpret_cast<uint4 *>(p.out + p.l.head_off)[tile] =
            make_uint4(base | cnt << 8 | (zero ? kTileZero : 0u), cnt == kTileRaw ? 64 : cnt <= kInline ? 0 : (cnt + 3) / 4, 0, 0);
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
    const uint4 *head = reinterpret_cast<const uint4 *>(p.out + p.l.head_off);
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
    const uint64_t gap = p.l.head_off + 16 * p.l.tiles + 8 * threadIdx.x;
    if (gap < p.l.tile_off) *reinterpret_cast<uint64_t *>(p.out + gap) = 0;
}

// The tiles' offsets.
__global__ __launch_bounds__(256) void k_pack_place(PackParams p) {
    __shared__ uint64_t lds[4];
    uint4 *head = reinterpret_cast<uint4 *>(p.out + p.l.head_off);
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
    uint4 &head = reinterpret_cast<uint4 *>(p.out + p.l.head_off)[tile];
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
        if (mine >> i & 1) {
            const uint32_t e = lane << 4 | i | (uint32_t)v[i] << 16;
            if (slot == 0) head.z = e;
            if (slot == 1) head.w = e;
            if (cnt > kInline) list[slot] = e;
            ++slot;
        }
    // the last unit's unused entries
    const uint32_t pad = cnt > kInline ? (cnt + 3) / 4 * 4 : 0;
    if (lane >= cnt && lane < pad) list[lane] = 0;
}

// A wave decodes a tile and writes its rows.  Bound by memory: 28672 x 4096 in
// 67 us, 411 MB read and written (part of it from the last-level cache).
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
    const uint64_t c0 = kb * kTileCols + q * 8;
    uint16_t *dst = p.out + e * p.matrix_stride + (part * p.w.part_rows + row) * p.row_stride + c0;
    if (c0 + 40 <= p.cols) {
        *reinterpret_cast<u32x4_any *>(dst) = u32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<u32x4_any *>(dst + 32) = u32x4{v[4], v[5], v[6], v[7]};
        return;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t c = (i >> 3) * 32 + (i & 7);
        if (c0 + c < p.cols) dst[c] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
    }
}

// Columns c .. c + 7 of a row, zeros behind the last column.
__device__ inline u32x4 stage_unit(const uint16_t *row, uint64_t c, uint64_t cols) {
    u32x4 v = {0, 0, 0, 0};
    if (c + 8 <= cols) {
        v = *reinterpret_cast<const u32x4_any *>(row + c);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < cols) v[j >> 1] |= (uint32_t)row[c + j] << (16 * (j & 1));
    }
    return v;
}

// Rows copied to a stride of whole 16-byte units, zeros behind the last column:
// the tiled products read x 16 bytes at a time, and what lies behind a row must
// not meet the zeros of a packed weight as a NaN.  1999 x 2050 in 6.5 us, 2.5
// TB/s: latency and the launch.
__global__ __launch_bounds__(256) void k_stage(const uint16_t *in, uint64_t in_stride, uint16_t *out, uint64_t out_stride,
                                               uint64_t rows, uint64_t cols) {
    const uint64_t units = out_stride / 8, n = rows * units;
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (uint64_t)gridDim.x * 256) {
        const uint64_t row = i / units, c = i % units * 8;
        *reinterpret_cast<u32x4 *>(out + row * out_stride + c) = stage_unit(in + row * in_stride, c, cols);
    }
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

// Zeros in columns [c0, c1) of the rows that no group holds (all of a
// workgroup's threads together).  Where the offsets ascend these are the rows
// before the first and behind the last.  A descending pair is an empty group, and the
// groups around it may lie anywhere: then a run of such rows begins at 0 or at a group's
// end and goes to the next group's begin.  Rows of a group are other workgroups'
// results and never touched here.
// A call, since inlined it takes registers from the products' main loops.  At
// most 1,024 bytes a row, a lane for each 16.
__device__ __noinline__ void clear_rest(const int32_t *offsets, uint32_t groups, uint32_t tokens, void *out,
                                        uint64_t stride, uint32_t elem, uint32_t c0, uint32_t c1, uint32_t threads) {
    const uint32_t lane = threadIdx.x & 63, wide = c1 - c0, each = 16 / elem, units = (wide + each - 1) / each;
    auto clear = [&](uint32_t row, uint32_t u) {  // 16 bytes, at any value's address
        uint8_t *const at = static_cast<uint8_t *>(out) + ((uint64_t)row * stride + c0 + u * each) * elem;
        if ((u + 1) * each <= wide) {
            *reinterpret_cast<u32x4_any *>(at) = u32x4{0, 0, 0, 0};
            return;
        }
        for (uint32_t b = 0; b < (wide - u * each) * elem; b += 2) *reinterpret_cast<uint16_t *>(at + b) = 0;
    };
    auto clamped = [&](uint32_t i) { return (uint32_t)min(max(offsets[i], 0), (int32_t)tokens); };
    const uint32_t first = clamped(0), last = clamped(groups);
    bool down = false;
#pragma unroll 1
    for (uint32_t g = lane; g < groups; g += 64) down |= clamped(g + 1) < clamped(g);
    uint32_t per = 1;  // lanes a row
    while (per < units) per *= 2;
    if (!__any(down)) {
        const uint32_t rest = first + (tokens - last), u = threadIdx.x & (per - 1);
        if (u < units)
            for (uint32_t i = threadIdx.x / per; i < rest; i += threads / per) clear(i < first ? i : last + (i - first), u);
        return;
    }
    for (uint32_t i = threadIdx.x >> 6; i <= groups; i += threads / 64) {  // a wave a group's end; row 0 behind the last
        uint32_t end = 0;
        if (i < groups) {
            end = clamped(i + 1);
            if (end <= clamped(i)) continue;
        }
        bool held = false;
        uint32_t next = tokens;  // where the next group begins
#pragma unroll 1
        for (uint32_t g = lane; g < groups; g += 64) {
            const uint32_t b = clamped(g), e = clamped(g + 1);
            held |= b <= end && end < e;
            if (b < e && b >= end) next = min(next, b);
        }
        if (__any(held)) continue;
        for (int d = 1; d < 64; d <<= 1) next = min(next, (uint32_t)__shfl_xor((int)next, d));
        if (const uint32_t u = lane & (per - 1); u < units)
            for (uint32_t row = end + lane / per; row < next; row += 64 / per) clear(row, u);
    }
}

// The same for columns [c0, c1) of a part in y and in the pre-activation.
template <class P>
__device__ inline void clear_rest_linear(const P &p, uint32_t c0, uint32_t c1, uint32_t threads) {
    const LinearEpi &e = p.lin;
    clear_rest(p.offsets, p.groups, p.tokens, e.y, e.y_stride, e.y_f32 ? 4 : 2, c0, c1, threads);
    if (!e.preact) return;
    for (uint32_t n = 0; n < p.w.parts * p.w.part_rows; n += p.w.part_rows)
        clear_rest(p.offsets, p.groups, p.tokens, e.preact, e.preact_stride, e.preact_f32 ? 4 : 2, n + c0, n + c1, threads);
}

// ---- few rows ---------------------------------------------------------------------

// y = W x for up to 16 MT rows of x at a time.  Bound by the reads of W: 28672
// x 4096 gated, 16 rows, 37 us from memory, 4.9 TB/s of packed bytes, about as fast as
// a large copy (29.5 us when half of them are in the last-level cache).  A workgroup owns RB row blocks of W; its NW waves split K and add their
// parts in LDS in a fixed order.  The weights go from memory to the matrix
// instructions without touching LDS; a wave has one column block on its way and
// the bytes in flight come from the number of waves (blocks loaded two or four
// ahead took more registers, so fewer waves, and were slower: one row of 4096 x
// 4096 in 1.1 and 1.5 times the time, which is 5.8 us now, 8.4 with weights from memory).  Headers: lane l of `heads` holds that of
// the wave's l-th block.  What lies behind the last block, row or column is read
// as zeros.
template <int MT, int RB, bool GATED, int NW>
__global__ __launch_bounds__(NW * 64) void k_skinny(SkinnyParams p) {
    __shared__ f32x4 part[NW][RB * MT * 64];
    const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const uint32_t q = lane >> 4, r = lane & 15;
    uint32_t begin, end;
    group_rows(p.offsets, blockIdx.y, p.tokens, begin, end);
    if (p.lin.clear && blockIdx.y == 0) {
        constexpr uint32_t WIDE = (GATED ? RB / 2 : RB) * 16;
        const uint32_t c = min(blockIdx.x * WIDE, p.w.part_rows);
        clear_rest_linear(p, c, min(c + WIDE, p.w.part_rows), NW * 64);
    }
    if (begin == end) return;
    const uint32_t KB = p.w.col_blocks, n = (KB + NW - 1 - wave) / NW;  // blocks of this wave
    uint64_t tile0[RB];
    rsrc_t rows[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        uint32_t b = GATED ? blockIdx.x * (RB / 2) + i / 2 : blockIdx.x * RB + i;
        if (b >= p.w.part_blocks) b = p.w.part_blocks - 1;  // computed and dropped
        if (GATED && (i & 1)) b += p.w.part_blocks;
        tile0[i] = ((uint64_t)blockIdx.y * p.w.row_blocks + b) * KB;
        rows[i] = buffer(p.w.tiles + tile0[i] * kTileBytes, KB * kTileBytes);
    }
    for (uint32_t m0 = begin; m0 < end; m0 += 16 * MT) {
        f32x4 acc[RB][MT];
#pragma unroll
        for (int i = 0; i < RB; ++i)
            for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
        const uint32_t here = min(end - m0, 16u * MT);
        const rsrc_t xb = buffer(static_cast<const uint8_t *>(p.x.p) + (uint64_t)m0 * p.x.stride * 2,
                                 ((here - 1) * (uint32_t)p.x.stride + p.cols) * 2);
        Tile t[RB];
        uint4 x[MT][2], heads[RB];
        auto load = [&](uint32_t k) __attribute__((always_inline)) {
            const uint32_t kb = wave + k * NW;
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                const uint32_t at = kb < KB ? kb * kTileBytes : KB * kTileBytes;
                t[i].sm = read16(rows[i], at + lane * 16);
                t[i].code = read8(rows[i], at + kTileSm + lane * 8);
            }
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t c = kb * kTileCols + h * 32 + q * 8, m = j * 16 + r;
                    x[j][h] = read16(xb, m < here && c < p.cols ? (m * (uint32_t)p.x.stride + c) * 2 : kNowhere);
                }
        };
        auto multiply = [&](uint32_t k) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                uint32_t v[8];
                t[i].h.x = __builtin_amdgcn_readlane(heads[i].x, k & 63);
                tile_decode_plain(t[i], v);
                if (t[i].h.x & (0xFF00u | kTileZero)) {
                    t[i].h.y = __builtin_amdgcn_readlane(heads[i].y, k & 63);
                    t[i].h.z = __builtin_amdgcn_readlane(heads[i].z, k & 63);
                    t[i].h.w = __builtin_amdgcn_readlane(heads[i].w, k & 63);
                    tile_decode(t[i], p.w, lane, v);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bf16x8 a = __builtin_bit_cast(bf16x8, u32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]});
#pragma unroll
                    for (int j = 0; j < MT; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, x[j][h]),
                                                                            acc[i][j], 0, 0, 0);
                }
            }
        };
        auto load_heads = [&](uint32_t k0) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < RB; ++i) heads[i] = p.w.head[tile0[i] + min(wave + (k0 + lane) * NW, KB - 1)];
        };
        load_heads(0);  // (first: loads come back in order)
        load(0);
        for (uint32_t k0 = 0; k0 < n; k0 += 64) {
            if (k0) load_heads(k0);
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                heads[i] = head_checked(p.w, heads[i]);
                if (wave + (k0 + lane) * NW >= KB) heads[i].x = 0;
            }
            for (uint32_t k = k0; k < min(n, k0 + 64); ++k) {
                multiply(k);
                load(k + 1);
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
                linear_out<GATED, 4>(p.lin, (uint64_t)blockIdx.y * p.rows, p.w.part_rows, m, b * 16 + (l >> 4) * 4, z);
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
// The contraction goes in stages of 32 through a ring of four LDS stages.  In
// step s a wave multiplies fragments of stage s and reads those of stage s + 1
// behind them, starts the copies of stage s + 3 from memory to LDS, and decodes
// its share of the weights of the stages after next; one barrier ends the step.
// Two waves a SIMD: a wave alone issues an instruction every four cycles, and a
// step has too many of them for the matrix instructions' time.  256 x 256: 8192
// x 4096 x 14336 in 880 to 970 us, 990 to 1090 TFLOP/s as the clock allows; dx 1000, dw
// (nothing to decode) 1270 to 1320, the loss's logits 1040, their gradient 1000; a large
// library product reaches 1310 here.  Forward and dx are bound by the instructions of the decoder, which
// share the SIMD with the matrix instructions' issue and its power.
//
// With 64 or 128 columns a tile (and packed rows) the traffic of LDS and a
// step's latencies weigh more than the matrix instructions: there a wave takes
// two row blocks and all columns, so that its weights go from memory through
// the decoder to the matrix instructions in registers, and only the tokens'
// values go through LDS.  128 x 128: two times four waves, each half of the
// contraction, added up at the end (1024 x 4096 x 4096 in 49 us; with one wave a
// SIMD 67 where this took 55, decoded tiles through the ring 70); 256 x 64: eight
// waves (128256 x 4096, 64 tokens: 151 us, 5.3 TB/s of packed bytes; through the
// ring 212).

enum Operand { kPacked, kPackedT, kRows, kCols };

// Place of 16-byte unit `unit` of row `row` in a stage of [T][32] values (64
// bytes a row): the xor makes 16 rows cover the 256 bytes of the banks, and
// also rows 0-3 and 12-15 of one unit with rows 4-11 of the next, the lanes
// that a read of 16 bytes takes together.
__device__ inline uint32_t rows_swizzle(uint32_t row) { return (0u - (row >> 2)) & 3; }
__device__ inline uint32_t rows_at(uint32_t row, uint32_t unit) { return row * 64 + ((unit ^ rows_swizzle(row)) * 16); }

// Granule (32 bytes, 16 columns) `g` of contraction row `a` in a stage of
// [32][T] values that is read transposed.  A transposing read takes four
// consecutive rows of two quads eight rows apart: these eight get eight
// different granules of the 256 bytes that the banks span.
__device__ inline uint32_t cols_swizzle(uint32_t a) { return (a & 3) | (a >> 3 & 1) << 2; }
template <int T>
__device__ inline uint32_t cols_at(uint32_t a, uint32_t g) {
    return a * (T * 2) + ((g ^ cols_swizzle(a)) * 32);
}

// Eight contraction values 8 q + j of column c0 + (lane & 15).
template <int T>
__device__ inline bf16x8 cols_frag(const uint8_t *lds, uint32_t c0, uint32_t lane) {
    const uint32_t q = lane >> 4, l = lane & 15;
    s16x4 v[2];
#pragma unroll
    for (uint32_t t = 0; t < 2; ++t) {
        const uint32_t a = q * 8 + t * 4 + (l >> 2);
        const uint8_t *p = lds + cols_at<T>(a, c0 >> 4) + (l & 3) * 8;
        v[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)p);
    }
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    const s16x8 x = __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, x);
}

// 16 bytes a lane from memory straight to LDS, at `dst` + 16 lane.  In asm, so
// that the compiler does not wait for it before the next read of LDS: the
// kernel's own waits and barriers say when the bytes are there.  It has no
// result registers, and the asm statements around it keep their order.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // (m0 is reserved; it is set here all the same)
__device__ inline uint32_t lds_address(const uint8_t *p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t *)p;
}
__device__ inline void copy_to_lds(rsrc_t r, uint32_t off, uint32_t dst) {
    const uint32_t at = uniform(dst);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at), "v"(off), "s"(r) : "m0");
}
#pragma clang diagnostic pop

template <int N>
__device__ inline void wait_copies() {  // all but the last N memory operations of this wave, and its LDS operations
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
__device__ inline void barrier() { asm volatile("s_barrier" ::: "memory"); }

// acc += a b, in place in accumulation registers.  In asm, because with half
// of the registers taken by them the compiler's own choice of registers moves accumulators
// to and fro in the loop (and then spills); the statements keep their order.
// Between them and other instructions on the same registers there have to be
// 18 cycles that the compiler does not know of: settle().
__device__ inline void mfma(f32x4 &acc, bf16x8 a, bf16x8 b) {
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
template <int FR, int FC>
__device__ inline void settle(f32x4 (&acc)[FR][FC]) {
#pragma unroll
    for (int i = 0; i < FR * FC; ++i) asm volatile("" : "+a"(acc[i / FC][i % FC]));
    asm volatile("s_nop 15\n\ts_nop 15");
#pragma unroll
    for (int i = 0; i < FR * FC; ++i) asm volatile("" : "+a"(acc[i / FC][i % FC]));
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

// W results of column c, rows r .. r + W - 1 (of the tile's kind of rows).
template <GemmKind KIND, bool GATED, int W>
__device__ inline void emit(const GemmParams &p, uint32_t g, uint32_t c, uint32_t c_end, uint32_t r,
                            float v[GATED ? 2 : 1][W]) {
    if constexpr (KIND == kGemmLossStat) {
        return;  // (has an epilogue of its own)
    } else if constexpr (KIND == kGemmForward) {
        if (c < c_end) linear_out<GATED, W>(p.lin, (uint64_t)g * p.rows, p.w.part_rows, c, r, v);
    } else if constexpr (KIND == kGemmLossDz) {
        // g (softmax - one at the target), rounded to bf16 for the two products that follow; zeros behind the last row.
        // In units of the largest g, which the products' results are multiplied with in fp32: with one g for all tokens,
        // as a mean has, g (p - 1) would be off by the same part of itself, up to 2^-8, at nearly every target, and the
        // gradients' errors would add up instead of averaging out.  p - 1 itself is near -1, which is exact.  (A g under
        // 2^-126 of the largest is lost.)
        if (c >= c_end) return;
        const int64_t want = p.loss.target[c];
        const bool counts = want != p.loss.ignore && want >= 0 && want < (int64_t)p.rows;
        const float gr = counts ? p.loss.dloss[c] / *p.loss.unit : 0.0f, lse = p.loss.lse[c];
        const uint32_t n = p.row_block0 * 16 + r, hit = counts ? (uint32_t)want - n : W;
#pragma unroll
        for (int d = 0; d < W; ++d) {
            float e = __expf(v[0][d] - lse);
            if ((uint32_t)d == hit) e -= 1.0f;
            v[0][d] = n + d < p.rows && counts ? gr * e : 0.0f;
        }
        store<W>(p.loss.dz, (uint64_t)c * p.loss.dz_stride + r, false, W, v[0]);
    } else {
        const StoreEpi &e = p.store;
        uint64_t row = c;
        if constexpr (KIND == kGemmDw) {
            // padded row of the stack's part -> row of the matrix; pieces start at row_block0
            const uint32_t n = c + p.row_block0 * 16, pad = p.w.part_blocks * 16, part = n >= pad ? 1 : 0, in = n - part * pad;
            if (in >= p.w.part_rows || part >= p.w.parts || c >= p.row_blocks * 16) return;
            row = (uint64_t)g * p.rows + (uint64_t)part * p.w.part_rows + in;
        } else {
            if (c >= c_end) return;
        }
        if (r >= p.cols) return;
        const uint32_t count = p.cols - r < W ? p.cols - r : W;
        if (e.sum) {
            if (e.add) {
                float o[W];
                load<W>(e.sum, row * e.sum_stride + r, true, count, o);
                for (int d = 0; d < W; ++d) v[0][d] += o[d];
            }
            if (!e.out) store<W>(e.sum, row * e.sum_stride + r, true, count, v[0]);
        }
        if (e.out && e.unit) {
            const float unit = *e.unit;
            for (int d = 0; d < W; ++d) v[0][d] *= unit;
        }
        if (e.out) store<W>(e.out, row * e.stride + r, false, count, v[0]);
    }
}

// WR by WC waves share a tile's outputs; WK 2: twice, each half of the contraction.
template <Operand RK, Operand CK, GemmKind KIND, bool GATED, int TR, int TC, int WR, int WC, int WK = 1>
__global__ __launch_bounds__(WR *WC *WK * 64, 2) void k_gemm(GemmParams p) {
    constexpr int WAVES = WR * WC, ALL = WAVES * WK;
    constexpr bool DIRECT = RK == kPacked && WC == 1;      // every wave decodes its own rows, in registers
    static_assert(ALL == 8 && (DIRECT || WK == 1), "eight waves");
    constexpr int FR = TR / WR / 16, FC = TC / WC / 16;    // fragments of a wave
    constexpr int RSTAGE = DIRECT ? 0 : TR * 64, CSTAGE = TC * 64;  // bytes of an operand's stage
    constexpr int STAGES = DIRECT ? 8 : 4;
    constexpr int C_ALL = CSTAGE / 1024, R_ALL = TR / 16;      // copies that fill one
    constexpr int C_COPIES = C_ALL > WAVES ? C_ALL / WAVES : 1;      // a wave's (with fewer than waves, some twice)
    constexpr int R_COPIES = R_ALL > WAVES ? R_ALL / WAVES : 1;
    constexpr bool PACKED = RK == kPacked || RK == kPackedT;
    constexpr int TILES = DIRECT ? 1 : TR / 16 / WAVES;  // packed tiles a wave decodes in two steps: 2 or 1
    constexpr int SLOT = 2048;              // a packed tile on its way to the decoder
    // the stages of R and of C, the packed tiles
    constexpr int RING = WK * STAGES * (RSTAGE + CSTAGE);
    __shared__ __align__(16) uint8_t lds[RING + (PACKED && !DIRECT ? TILES * WAVES * SLOT : 0)];
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave_all = uniform(tid >> 6);
    const uint32_t wave = wave_all % WAVES, wk = wave_all / WAVES;
    const uint32_t q = lane >> 4, l15 = lane & 15;
    const uint32_t wr = wave % WR, wc = wave / WR;

    // Workgroups go to the 8 XCDs in turn: give each XCD a run of neighbouring
    // tiles, four column tiles wide, so that its L2 holds what they share.
    const uint32_t total = p.r_tiles * p.c_tiles;
    if constexpr (KIND == kGemmForward || KIND == kGemmDx) {
        if (blockIdx.x >= total) {  // behind the tiles, one a strip of columns: the rows of no group
            if (blockIdx.y) return;
            constexpr bool F = KIND == kGemmForward;
            const uint32_t wide = GATED ? TR / 2 : TR, limit = F ? p.w.part_rows : p.cols;
            const uint32_t c = min((blockIdx.x - total) * wide, limit), end = min(c + wide, limit);
            if constexpr (F)
                clear_rest_linear(p, c, end, ALL * 64);
            else
                clear_rest(p.offsets, p.groups, p.tokens, p.store.out, p.store.stride, 2, c, end, ALL * 64);
            return;
        }
    }
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
    // stages of 32 contraction values
    const uint32_t S_ALL = KIND == kGemmDw ? (a_end - a0 + 31) / 32 : 2 * p.steps;
    uint32_t s0 = 0, S = S_ALL;
    if (KIND != kGemmDw && p.splits > 1) {  // a run of the contraction
        s0 = 2 * (uint32_t)((uint64_t)p.steps * blockIdx.y / p.splits);
        S = 2 * (uint32_t)((uint64_t)p.steps * (blockIdx.y + 1) / p.splits) - s0;
    }
    const uint32_t KB = p.w.col_blocks;

    // ---- copies from memory ----
    // Rows: a copy takes 16 rows.  Cols: 1 KiB of the stage's rows.  What lies behind the last row or column (of Rows:
    // of the contraction) is read as zeros.
    constexpr int PARTS = C_COPIES + (RK == kCols ? R_COPIES : 0);
    uint32_t c_off[C_COPIES], r_off[RK == kCols ? R_COPIES : 1];
    const uint32_t c_unit = ((lane & 3) ^ rows_swizzle(lane >> 2)) * 8;  // Rows: this lane's columns of a stage
    auto c_index = [&](int i) __attribute__((always_inline)) -> uint32_t { return (wave * C_COPIES + i) % C_ALL; };
    auto r_index = [&](int i) __attribute__((always_inline)) -> uint32_t { return (wave * R_COPIES + i) % R_ALL; };
    auto cols_off = [&](uint32_t index, uint32_t wide, uint32_t x0, uint32_t limit, uint64_t stride)
                        __attribute__((always_inline)) -> uint32_t {
        const uint32_t j = index * 64 + lane, a = j / (wide / 8), u = j % (wide / 8);
        const uint32_t c = x0 + (((u >> 1) ^ cols_swizzle(a)) * 2 + (u & 1)) * 8;
        return c < limit ? (a * (uint32_t)stride + c) * 2 : kNowhere;
    };
#pragma unroll
    for (int i = 0; i < C_COPIES; ++i) {
        if constexpr (CK == kRows) {
            c_off[i] = ((c_index(i) * 16 + (lane >> 2)) * (uint32_t)p.cmat.stride + c_unit) * 2;
        } else {
            c_off[i] = cols_off(c_index(i), TC, c0, p.c_limit, p.cmat.stride);
        }
    }
    if constexpr (RK == kCols)
#pragma unroll
        for (int i = 0; i < R_COPIES; ++i) r_off[i] = cols_off(r_index(i), TR, rt * TR, p.r_limit, p.rmat.stride);
    uint8_t *const r_lds = lds, *const c_lds = lds + STAGES * RSTAGE + (WK > 1 ? wk * (STAGES * CSTAGE) : 0);
    const uint32_t r_at = lds_address(lds), c_at = r_at + STAGES * RSTAGE;
    // The i-th of a wave's copies of stage s.  Stages behind the last are zeros.
    auto copy_part = [&](uint32_t s, int i) __attribute__((always_inline)) {
        const uint8_t *cp = static_cast<const uint8_t *>(p.cmat.p);
        if constexpr (CK == kRows) {
            const uint32_t rows = min((uint32_t)TC, c_end - c0), a = (s0 + s) * 32;
            const uint32_t left = s < S && a < p.c_limit ? p.c_limit - a : 0;  // columns from here on
            const rsrc_t c = buffer(cp + ((uint64_t)c0 * p.cmat.stride + a) * 2,
                                    left ? ((rows - 1) * (uint32_t)p.cmat.stride + left) * 2 : 0);
            copy_to_lds(c, c_unit < left ? c_off[i] : kNowhere, c_at + s % STAGES * CSTAGE + c_index(i) * 1024);
        } else {
            const uint32_t a = a0 + s * 32, rows = s < S ? min(32u, a_end - a) : 0;
            const bool r = i >= C_COPIES;
            const Mat &m = r ? p.rmat : p.cmat;
            const rsrc_t x = buffer(static_cast<const uint8_t *>(m.p) + (uint64_t)a * m.stride * 2, rows * (uint32_t)m.stride * 2);
            if (r)
                copy_to_lds(x, r_off[i - C_COPIES], r_at + (s & 3) * RSTAGE + r_index(i - C_COPIES) * 1024);
            else
                copy_to_lds(x, c_off[i], c_at + s % STAGES * CSTAGE + c_index(i) * 1024);
        }
    };

    // ---- packed weights ----
    // A block of 64 contraction values (two stages) is TR / 16 tiles; a wave decodes TILES of them.
    // TILES 2: one in each step.  Forward: decode step d fills half of stages d & ~1 and (d & ~1) + 1; in step s,
    // d = s + 3 (stage s + 2 is whole after step s, when s is odd with the one after it).  dx: d fills stage d, d = s + 2.
    // TILES 1 (dx): one in every other step, d = s / 2 + 1, half of the waves in even steps into stage 2 d, half in odd
    // ones into 2 d + 1.
    // A tile is copied to LDS two steps before.
    constexpr bool FWD = RK == kPacked;
    const uint32_t half = TILES == 2 ? 0 : wave / (WAVES / 2);
    const uint32_t decodes = TILES == 2 ? S : (S + 1) / 2;
    auto tile_index = [&](uint32_t d, bool &live) __attribute__((always_inline)) -> uint64_t {
        uint32_t rb, kb;
        d = min(d, decodes - 1);
        if (FWD) {
            const uint32_t j = wave * 2 + (d & 1);
            kb = (s0 >> 1) + (d >> 1);
            if (GATED) {
                rb = rt * (TR / 32) + (j >> 1);
                live = rb < p.w.part_blocks;
                rb = live ? rb + (j & 1 ? p.w.part_blocks : 0) : 0;
            } else {
                rb = rt * (TR / 16) + j;
                live = rb < p.row_blocks;
                rb = live ? rb + p.row_block0 : 0;
            }
        } else {
            const uint32_t j = TILES == 2 ? wave : wave % (WAVES / 2), stage = s0 + (TILES == 2 ? d : 2 * d + half);
            rb = stage * 2 + (j & 1);
            kb = rt * (TR / 64) + (j >> 1);
            live = rb < p.row_blocks && kb < KB;
            rb = live ? rb + p.row_block0 : 0;
            kb = live ? kb : 0;
        }
        return ((uint64_t)g * p.w.row_blocks + rb) * KB + kb;
    };
    // Headers: lane l holds that of decode step 64 i + l; the next 64 are loaded meanwhile.
    constexpr uint32_t kDead = 1u << 31;  // header flag here: the tile lies outside the weight
    uint4 heads = make_uint4(0, 0, 0, 0), heads_next = heads;
    auto load_heads = [&](uint32_t d0) __attribute__((always_inline)) -> uint4 {
        bool live;
        return p.w.head[tile_index(d0 + lane, live)];
    };
    auto use_heads = [&](uint32_t d0, uint4 h) __attribute__((always_inline)) {
        bool live;
        tile_index(d0 + lane, live);
        heads = head_checked(p.w, h);
        if (!FWD && !live) heads.x |= kDead;
    };
    constexpr int SLOTS = TILES;
    uint8_t *const slots = lds + RING + wave * SLOTS * SLOT;
    const uint32_t slots_at = r_at + RING + wave * SLOTS * SLOT;
    auto copy_tile = [&](uint32_t d) __attribute__((always_inline)) {
        bool live;
        const rsrc_t r = buffer(p.w.tiles + tile_index(d, live) * kTileBytes, kTileBytes);
        copy_to_lds(r, lane * 16, slots_at + d % SLOTS * SLOT);
        copy_to_lds(r, kTileSm + (lane & 31) * 16, slots_at + d % SLOTS * SLOT + kTileSm);  // (the codes twice)
    };
    auto read_tile = [&](uint32_t d, Tile &t) __attribute__((always_inline)) {
        const uint8_t *at = slots + d % SLOTS * SLOT;
        t.sm = *reinterpret_cast<const uint4 *>(at + lane * 16);
        t.code = *reinterpret_cast<const uint2 *>(at + kTileSm + lane * 8);
        t.h.x = __builtin_amdgcn_readlane(heads.x, d & 63);
    };
    // Places in LDS of the two halves of a lane's 16 values; dx: both in one stage.
    auto tile_place = [&](uint32_t d, uint32_t l, uint32_t &at0, uint32_t &at1) __attribute__((always_inline)) {
        if (FWD) {
            const uint32_t j = wave * 2 + (d & 1), at = j * 1024 + l * 16;
            at0 = (d & 2) * RSTAGE + at;
            at1 = at0 + RSTAGE;
        } else {
            const uint32_t j = TILES == 2 ? wave : wave % (WAVES / 2), row = (j & 1) * 16 + (l & 15), lq = l >> 4;
            const uint32_t stage = (TILES == 2 ? d : 2 * d + half) & 3;
            at0 = stage * RSTAGE + cols_at<TR>(row, (j >> 1) * 4 + (lq >> 1)) + (lq & 1) * 16;
            at1 = stage * RSTAGE + cols_at<TR>(row, (j >> 1) * 4 + 2 + (lq >> 1)) + (lq & 1) * 16;
        }
    };
    auto store_tile = [&](uint32_t d, const uint32_t v[8]) __attribute__((always_inline)) {
        uint32_t at0, at1;
        tile_place(d, lane, at0, at1);
        *reinterpret_cast<uint4 *>(r_lds + at0) = make_uint4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<uint4 *>(r_lds + at1) = make_uint4(v[4], v[5], v[6], v[7]);
    };
    // What the plain decode does not cover is put right behind it.
    auto mend = [&](uint32_t d, uint32_t h0) __attribute__((always_inline)) {
        if ((h0 & (0xFF00u | kTileZero | kDead)) == 0 || d >= decodes) return;
        uint32_t at0, at1;
        if (h0 & kDead) {
            const uint32_t v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            store_tile(d, v);
            return;
        }
        Tile t;
        t.h = make_uint4(h0, __builtin_amdgcn_readlane(heads.y, d & 63), __builtin_amdgcn_readlane(heads.z, d & 63),
                         __builtin_amdgcn_readlane(heads.w, d & 63));
        if (tile_special(h0)) {
            bool live;
            uint32_t v[8];
            // (each branch uses all that it loads: a load left unused would be waited for in the next step)
            const uint8_t *from = p.w.tiles + tile_index(d, live) * kTileBytes;
            t.sm = *reinterpret_cast<const uint4 *>(from + lane * 16);
            if (tile_raw(h0)) {
                tile_decode_raw(t, p.w, lane, v);
            } else {
                t.code = *reinterpret_cast<const uint2 *>(from + kTileSm + lane * 8);
                tile_decode_zero(t, v);
            }
            store_tile(d, v);
        }
        if (lane < tile_listed(h0)) {
            const uint32_t e = tile_entry(p.w, t.h, lane);
            tile_place(d, e >> 4 & 63, at0, at1);
            *reinterpret_cast<uint16_t *>(r_lds + (e & 8 ? at1 : at0) + (e & 7) * 2) = (uint16_t)(e >> 16);
        }
    };
    auto next_heads = [&](uint32_t d) __attribute__((always_inline)) {  // before decode step d
        if ((d & 63) == 0 && d) {
            use_heads(d, heads_next);
            heads_next = load_heads(d + 64);
        }
    };

    // ---- fragments and products ----
    // rf[i] is read again behind its products; the last one has two places, so that no read is left for a step's end
    bf16x8 rf[FR + 1], cf[2][FC];
    auto place = [](int i, int b) __attribute__((always_inline)) { return i == FR - 1 && b ? FR : i; };
    auto read_r = [&](uint32_t s, int i, int at) __attribute__((always_inline)) {
        const uint8_t *rl = r_lds + (s & 3) * RSTAGE;
        const uint32_t rr = (wr * FR + i) * 16;
        if constexpr (FWD)
            rf[at] = *reinterpret_cast<const bf16x8 *>(rl + rr * 64 + lane * 16);
        else
            rf[at] = cols_frag<TR>(rl, rr, lane);
    };
    auto read_c = [&](uint32_t s, int b, int i) __attribute__((always_inline)) {
        const uint8_t *cl = c_lds + s % STAGES * CSTAGE;
        const uint32_t cc = (wc * FC + i) * 16;
        if constexpr (CK == kCols)
            cf[b][i] = cols_frag<TC>(cl, cc, lane);
        else
            cf[b][i] = *reinterpret_cast<const bf16x8 *>(cl + rows_at(cc + l15, q));
    };
    f32x4 acc[FR][FC];
#pragma unroll
    for (int i = 0; i < FR; ++i)
        for (int j = 0; j < FC; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    if constexpr (DIRECT) {
        // Blocks of 64 contraction values, two stages each.  In block k a wave multiplies with its rows' tiles k, decodes
        // its tiles k + 1 between the products, stores its share of block k + 2 of C and loads its tiles k + 3.
        const uint32_t each = (S / 2 + WK - 1) / WK, kb0 = s0 / 2 + wk * each, n = wk ? S / 2 - each : each;
        uint64_t tile0[FR];
        rsrc_t rows[FR];
#pragma unroll
        for (int i = 0; i < FR; ++i) {
            uint32_t rb;
            if (GATED) {
                rb = rt * (TR / 32) + wave * (FR / 2) + i / 2;
                rb = rb < p.w.part_blocks ? rb + (i & 1 ? p.w.part_blocks : 0) : 0;
            } else {
                rb = rt * (TR / 16) + wave * FR + i;
                rb = rb < p.row_blocks ? rb + p.row_block0 : 0;
            }
            tile0[i] = ((uint64_t)g * p.w.row_blocks + rb) * KB;
            rows[i] = buffer(p.w.tiles + tile0[i] * kTileBytes, KB * kTileBytes);
        }
        uint4 hd[FR], hd_next[FR];  // lane l: the header of block 64 j + l
        auto first_heads = [&](uint32_t k) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < FR; ++i) hd_next[i] = p.w.head[tile0[i] + min(kb0 + k + lane, KB - 1)];
        };
        auto turn_heads = [&](uint32_t k) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < FR; ++i) {
                hd[i] = head_checked(p.w, hd_next[i]);
                if (k + lane >= n) hd[i].x = 0;
            }
            first_heads(k + 64);
        };
        Tile t[2][FR];
        uint32_t v[2][FR][8];
        auto load_tiles = [&](uint32_t k, Tile (&to)[FR]) __attribute__((always_inline)) {
            const uint32_t at = (k < n ? kb0 + k : KB) * kTileBytes;  // (behind the last block: zeros)
#pragma unroll
            for (int i = 0; i < FR; ++i) {
                to[i].sm = read16(rows[i], at + lane * 16);
                to[i].code = read8(rows[i], at + kTileSm + lane * 8);
            }
        };
        auto begin_tiles = [&](uint32_t k, Tile (&from)[FR]) __attribute__((always_inline)) {
            if ((k & 63) == 0 && k) turn_heads(k);
#pragma unroll
            for (int i = 0; i < FR; ++i) from[i].h.x = __builtin_amdgcn_readlane(hd[i].x, k & 63);
        };
        auto decode_pair = [&](const Tile (&from)[FR], uint32_t (&to)[FR][8], int u) __attribute__((always_inline)) {
            const int i = u / 8, k = u % 8;
            to[i][k] = tile_pair(from[i], k, (from[i].h.x & 0xFF) * 0x00800080u);
        };
        auto end_tiles = [&](uint32_t k, Tile (&from)[FR], uint32_t (&to)[FR][8]) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < FR; ++i)
                if (const uint32_t odd = from[i].h.x & (0xFF00u | kTileZero)) {
                    from[i].h.z = __builtin_amdgcn_readlane(hd[i].z, k & 63);
                    from[i].h.w = __builtin_amdgcn_readlane(hd[i].w, k & 63);
                    if (odd <= kInline << 8) {
                        tile_patch(from[i].h.z, lane, to[i]);
                        if (odd == kInline << 8) tile_patch(from[i].h.w, lane, to[i]);
                    } else {
                        from[i].h.y = __builtin_amdgcn_readlane(hd[i].y, k & 63);
                        tile_decode(from[i], p.w, lane, to[i]);
                        __builtin_amdgcn_s_waitcnt(0x0F70);  // (so that no wait for what was loaded here stays in the loop)
                    }
                }
        };
        // A block's values of C: the i-th KiB of this wave.
        constexpr int BC = 2 * C_ALL / WAVES;
        static_assert(2 * C_ALL % WAVES == 0 && BC >= 1, "whole copies");
        // Blocks of C on their way in registers: two where that is a KiB each (64 rows by 32768 x 4096 41.6 us, with one
        // 43); with 128 columns one, since two spill unless they are stored and loaded at a block's start, in front of its
        // products (777 x 4096 x 1024 18.6 us instead of 17.5).
        constexpr int AHEAD = TC == 64 ? 2 : 1;
        uint4 cs[2][BC];
        uint32_t cs_off[BC], cs_col[BC];
#pragma unroll
        for (int i = 0; i < BC; ++i) {
            const uint32_t index = wave * BC + i;
            cs_col[i] = index / C_ALL * 32 + c_unit;
            cs_off[i] = ((index % C_ALL * 16 + (lane >> 2)) * (uint32_t)p.cmat.stride + cs_col[i]) * 2;
        }
        auto load_c = [&](uint32_t k, uint4 (&to)[BC], int i0, int i1) __attribute__((always_inline)) {
            const uint32_t wide = min((uint32_t)TC, c_end - c0), a = (kb0 + k) * 64;
            const uint32_t left = k < n && a < p.c_limit ? p.c_limit - a : 0;
            const rsrc_t c = buffer(static_cast<const uint8_t *>(p.cmat.p) + ((uint64_t)c0 * p.cmat.stride + a) * 2,
                                    left ? ((wide - 1) * (uint32_t)p.cmat.stride + left) * 2 : 0);
#pragma unroll
            for (int i = i0; i < i1; ++i) to[i] = read16(c, cs_col[i] < left ? cs_off[i] : kNowhere);
        };
        auto store_c = [&](uint32_t k, const uint4 (&from)[BC], int i0, int i1) __attribute__((always_inline)) {
#pragma unroll
            for (int i = i0; i < i1; ++i)
                *reinterpret_cast<uint4 *>(c_lds + k % 4 * (2 * CSTAGE) + (wave * BC + i) * 1024 + lane * 16) = from[i];
        };
        first_heads(0);
        load_tiles(0, t[0]);
        load_c(0, cs[0], 0, BC);
        load_c(1, cs[1], 0, BC);
        load_tiles(1, t[1]);
        turn_heads(0);
        begin_tiles(0, t[0]);
#pragma unroll
        for (int u = 0; u < FR * 8; ++u) decode_pair(t[0], v[0], u);
        end_tiles(0, t[0], v[0]);
        store_c(0, cs[0], 0, BC);
        load_c(2, cs[0], 0, BC);
        store_c(1, cs[1], 0, BC);
        if (AHEAD == 2) load_c(3, cs[1], 0, BC);
        load_tiles(2, t[0]);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        barrier();
#pragma unroll
        for (int j = 0; j < FC; ++j) read_c(0, 0, j);
        auto block = [&](uint32_t k, auto parity) __attribute__((always_inline)) {
            constexpr int b = decltype(parity)::value;
            begin_tiles(k + 1, t[b ^ 1]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int j = 0; j < FC; ++j) {
                    read_c(2 * k + h + 1, h ^ 1, j);
                    // block k + 2 over block k - 2, which no wave reads any more; all before this block's last FC reads
                    constexpr int EACH = (BC + FC - 1) / FC;
                    if (h == 0 && j * EACH < BC) store_c(k + 2, cs[AHEAD == 2 ? b : 0], j * EACH, (j + 1) * EACH);
                    if (h == 1 && j * EACH < BC) load_c(k + 2 + AHEAD, cs[AHEAD == 2 ? b : 0], j * EACH, (j + 1) * EACH);
#pragma unroll
                    for (int i = 0; i < FR; ++i) {
                        const bf16x8 a = __builtin_bit_cast(
                            bf16x8, u32x4{v[b][i][4 * h], v[b][i][4 * h + 1], v[b][i][4 * h + 2], v[b][i][4 * h + 3]});
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, cf[h][j], acc[i][j], 0, 0, 0);
                    }
                    if (h == 0)
#pragma unroll
                        for (int u = j * FR * 8 / FC; u < (j + 1) * FR * 8 / FC; ++u) decode_pair(t[b ^ 1], v[b ^ 1], u);
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (h == 0) {
                    end_tiles(k + 1, t[b ^ 1], v[b ^ 1]);
                    load_tiles(k + 3, t[b ^ 1]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            // block k + 2's values of C are in LDS; only the last reads may be on their way
            asm volatile("s_waitcnt lgkmcnt(%0)" ::"n"(FC) : "memory");
            barrier();
        };
        for (uint32_t k = 0; k < each; k += 2) {  // (blocks behind the last add zeros)
            block(k, std::integral_constant<int, 0>{});
            block(k + 1, std::integral_constant<int, 1>{});
        }
        __syncthreads();
        if constexpr (WK > 1) {  // the halves' sums
            f32x4 *half = reinterpret_cast<f32x4 *>(lds) + wave * (FR * FC * 64) + lane;
            static_assert(WAVES * FR * FC * 1024 <= RING, "fits");
            if (wk)
#pragma unroll
                for (int i = 0; i < FR * FC; ++i) half[i * 64] = acc[i / FC][i % FC];
            __syncthreads();
            if (!wk)
#pragma unroll
                for (int i = 0; i < FR * FC; ++i) acc[i / FC][i % FC] += half[i * 64];
            __syncthreads();
        }
    } else if (S > 0) {
        uint4 heads_first;
        if constexpr (PACKED) {
            heads_first = load_heads(0);
            heads_next = load_heads(64);
        }
        // the decode steps before those of step 0 take their tiles through registers, all at once
        constexpr uint32_t BEFORE = !PACKED ? 0 : TILES == 1 ? 1 : FWD ? 3 : 2;
        Tile first[BEFORE ? BEFORE : 1];
#pragma unroll
        for (uint32_t d = 0; d < BEFORE; ++d) {
            bool live;
            const uint8_t *from = p.w.tiles + tile_index(d, live) * kTileBytes;
            first[d].sm = *reinterpret_cast<const uint4 *>(from + lane * 16);
            first[d].code = *reinterpret_cast<const uint2 *>(from + kTileSm + lane * 8);
        }
        if constexpr (PACKED)
            for (uint32_t d = 0; d < SLOTS; ++d) copy_tile(BEFORE + d);
        for (uint32_t s = 0; s < 3; ++s)
#pragma unroll
            for (int i = 0; i < PARTS; ++i) copy_part(s, i);
        if constexpr (PACKED) use_heads(0, heads_first);
#pragma unroll
        for (uint32_t d = 0; d < BEFORE; ++d) {
            uint32_t v[8];
            first[d].h.x = __builtin_amdgcn_readlane(heads.x, d);
            tile_decode_plain(first[d], v);
            store_tile(d, v);
            mend(d, first[d].h.x);
        }
        wait_copies<0>();
        barrier();
#pragma unroll
        for (int i = 0; i < FR; ++i) read_r(0, i, i);
#pragma unroll
        for (int i = 0; i < FC; ++i) read_c(0, 0, i);
        settle(acc);  // the zeros
        auto step = [&](uint32_t s, auto parity) __attribute__((always_inline)) {
            constexpr int b = decltype(parity)::value;
            const uint32_t d = TILES == 1 ? s / 2 + 1 : FWD ? s + 3 : s + 2;
            // whether this wave decodes in this step (TILES 1: a uniform branch, else known)
            const bool mine = PACKED && (TILES == 2 || half == b);
            Tile t;
            uint32_t v[8];
            if constexpr (PACKED) {
                if (mine) {
                    next_heads(d);
                    read_tile(d, t);
                }
            }
            const uint32_t base = PACKED ? (t.h.x & 0xFF) * 0x00800080u : 0;
            // between the matrix instructions, whose shadow hides them: copies, reads and the decoder
#pragma unroll
            for (int i = 0; i < FR; ++i) {
                if (i < PARTS) copy_part(s + 3, i);
                if (i == FR - 1)
#pragma unroll
                    for (int k = FR; k < PARTS; ++k) copy_part(s + 3, k);
#pragma unroll
                for (int k = i * FC / FR; k < (i + 1) * FC / FR; ++k) read_c(s + 1, b ^ 1, k);
                if (i == FR - 1) {
                    read_r(s + 1, i, place(i, b ^ 1));
                    if constexpr (PACKED) {
                        if (mine) {
                            store_tile(d, v);  // behind the last stage: into stages that nothing reads any more
                            mend(d, t.h.x);
                            copy_tile(d + SLOTS);
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int j = 0; j < FC; ++j) mfma(acc[i][j], rf[place(i, b)], cf[b][j]);
                if (i < FR - 1) read_r(s + 1, i, i);
                if constexpr (PACKED) {
                    // eight pairs, between the first and the last group of products
                    constexpr int GROUPS = FR - 2;
                    if (i > 0 && i <= GROUPS)
#pragma unroll
                        for (int k = (i - 1) * 8 / GROUPS; k < i * 8 / GROUPS; ++k)
                            v[k] = tile_pair(t, k, base);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            // stage s + 2 and the tile of the step after next but one have arrived: only this step's copies may be on
            // their way
            if (mine)
                wait_copies<PARTS + 2>();
            else
                wait_copies<PARTS>();
            barrier();
        };
        for (uint32_t s = 0; s < S; s += 2) {  // (a step behind an odd number of stages adds zeros)
            step(s, std::integral_constant<int, 0>{});
            step(s + 1, std::integral_constant<int, 1>{});
        }
        wait_copies<0>();
        barrier();
        settle(acc);
    }

    // ---- epilogues: acc[i][j][d] is row 16 (wr FR + i) + 4 q + d of the tile, column 16 (wc FC + j) + l15 ----
    if (KIND == kGemmLossStat && p.splits == 1) {
        // every token's largest logit in this tile, and the sum of exp(logit - that)
        f32x2 *red = reinterpret_cast<f32x2 *>(lds);  // [WR][TC]
        const uint32_t n0 = rt * TR + wr * FR * 16 + q * 4;
        if (rt * TR + TR > p.rows) {  // rows behind the last
#pragma unroll
            for (int i = 0; i < FR; ++i)
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    if (n0 + i * 16 + d >= p.rows)
                        for (int j = 0; j < FC; ++j) acc[i][j][d] = -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < FC; ++j) {
            const uint32_t m = c0 + (wc * FC + j) * 16 + l15;
            // the target, where it is one of this lane's rows
            const int64_t want = m < c_end ? p.loss.target[m] : -1;
            const uint32_t hit = want >= 0 && want < (int64_t)p.rows ? (uint32_t)want - n0 : FR * 16;
            if (hit < FR * 16 && (hit & 15) < 4 && wk == 0) {
#pragma unroll
                for (int i = 0; i < FR; ++i)
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        if (hit == (uint32_t)(i * 16 + d)) p.loss.picked[m] = acc[i][j][d];
            }
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < FR; ++i)
#pragma unroll
                for (int d = 0; d < 4; ++d) top = fmaxf(top, acc[i][j][d]);
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
            if (q == 0 && wk == 0) red[wr * TC + (wc * FC + j) * 16 + l15] = f32x2{ref, sum};
        }
        __syncthreads();
        for (uint32_t c = tid; c < TC; c += ALL * 64) {
            if (c0 + c >= c_end) continue;
            float ref = red[c][0], sum = 0;
#pragma unroll
            for (int w = 1; w < WR; ++w) ref = fmaxf(ref, red[w * TC + c][0]);
#pragma unroll
            for (int w = 0; w < WR; ++w) sum += red[w * TC + c][1] * __expf(red[w * TC + c][0] - ref);
            p.loss.parts[(uint64_t)(c0 + c) * p.r_tiles + rt] = make_float2(ref, sum);
        }
        return;
    }

    // The others go through LDS, some fragments of columns at a time, so that a column's rows of the whole tile leave in
    // one run of 16 bytes a lane (256 bytes a wave and column, from registers in two halves, took 18 us a tile of 256 x
    // 256 instead of 7): [columns][TR] values for each wc, in units of four, the unit's place xored with the column
    // against bank conflicts.  The WR waves of a wc share its columns.
    constexpr int UNITS = TR / 4, FIT = RING / WC / (TR * 64);
    constexpr int JP = FIT >= FC ? FC : FIT >= 2 && FC % 2 == 0 ? 2 : 1;  // fragments at a time
    constexpr int SHARE = WR * WK, COLS = JP * 16 / SHARE;                // waves of a column, columns of a wave
    constexpr int ROWS = TR / (GATED ? 2 : 1), LANES = ROWS / 8;          // results of a column, lanes for them
    static_assert(FIT >= 1 && JP * 16 % SHARE == 0 && COLS * LANES % 64 == 0, "whole waves");
    f32x4 *out = reinterpret_cast<f32x4 *>(lds + wc * (JP * TR * 64));
    const uint32_t share = WK > 1 ? wave_all : wr;
#pragma unroll
    for (int ph = 0; ph < FC; ph += JP) {
        if (ph) __syncthreads();
        if (wk == 0)
#pragma unroll
            for (int j = 0; j < JP; ++j)
#pragma unroll
            for (int i = 0; i < FR; ++i)
                out[(j * 16 + l15) * UNITS + ((wr * FR * 4 + i * 4 + q) ^ l15)] = acc[i][ph + j];
        __syncthreads();
        const uint32_t cb = (wc * FC + ph) * 16;  // the first column
        if (KIND != kGemmDw && p.splits > 1) {
            // a run's part of the sums: [run][tile][column][row]
            float *to = p.part + ((uint64_t)blockIdx.y * total + ct * p.r_tiles + rt) * (TR * TC);
#pragma unroll 4
            for (uint32_t k = lane; k < COLS * UNITS; k += 64) {
                const uint32_t cl = share * COLS + k / UNITS, u = k % UNITS;
                *reinterpret_cast<f32x4 *>(to + (cb + cl) * TR + u * 4) = out[cl * UNITS + (u ^ (cl & 15))];
            }
            continue;
        }
#pragma unroll 2
        for (uint32_t k = lane; k < COLS * LANES; k += 64) {
            const uint32_t cl = share * COLS + k / LANES, l = k % LANES;
            float v[GATED ? 2 : 1][8];
#pragma unroll
            for (int h = 0; h < (GATED ? 2 : 1); ++h)
#pragma unroll
                for (int d = 0; d < 8; d += 4) {
                    // gated: eight results come from half a block of the gate and half of the block behind it
                    const uint32_t u = GATED ? (l >> 1) * 8 + h * 4 + (l & 1) * 2 + d / 4 : l * 2 + d / 4;
                    const f32x4 x = out[cl * UNITS + (u ^ (cl & 15))];
                    for (int e = 0; e < 4; ++e) v[h][d + e] = x[e];
                }
            emit<KIND, GATED, 8>(p, g, c0 + cb + cl, c_end, rt * ROWS + l * 8, v);
        }
    }
}

// The runs' parts added up in their order, a thread four rows of a column.
template <GemmKind KIND, bool GATED>
__global__ __launch_bounds__(256) void k_join(GemmParams p, uint32_t tr, uint32_t tc) {
    const uint32_t outs = tr / (GATED ? 8 : 4), k = blockIdx.y * 256 + threadIdx.x;
    const uint32_t cl = k / outs, u = k % outs, ct = blockIdx.x / p.r_tiles, rt = blockIdx.x % p.r_tiles;
    uint32_t g, c0, c_end;
    if (!find_group(p, ct, tc, threadIdx.x & 63, g, c0, c_end)) return;
    if (cl >= tc || c0 + cl >= c_end) return;
    float v[GATED ? 2 : 1][4];
#pragma unroll
    for (int h = 0; h < (GATED ? 2 : 1); ++h) {
        const uint32_t row = GATED ? (u >> 2) * 32 + h * 16 + (u & 3) * 4 : u * 4;
        const float *from = p.part + ((uint64_t)blockIdx.x * tc + cl) * tr + row;
        f32x4 x = *reinterpret_cast<const f32x4 *>(from);
#pragma unroll 8
        for (uint32_t i = 1; i < p.splits; ++i)  // (the loads of eight runs together)
            x += *reinterpret_cast<const f32x4 *>(from + (uint64_t)i * p.r_tiles * p.c_tiles * tr * tc);
        for (int d = 0; d < 4; ++d) v[h][d] = x[d];
    }
    emit<KIND, GATED, 4>(p, g, c0 + cl, c_end, rt * (tr / (GATED ? 2 : 1)) + u * 4, v);
}

// The same for the loss: a column's tr / 4 threads (32 or 64 lanes) find its reference and sum.
__global__ __launch_bounds__(256) void k_join_stat(GemmParams p, uint32_t tr, uint32_t tc) {
    const uint32_t outs = tr / 4, k = blockIdx.y * 256 + threadIdx.x;
    const uint32_t cl = k / outs, u = k % outs, ct = blockIdx.x / p.r_tiles, rt = blockIdx.x % p.r_tiles;
    const uint32_t m = ct * tc + cl;
    if (cl >= tc || m >= p.tokens) return;
    const float *from = p.part + ((uint64_t)blockIdx.x * tc + cl) * tr + u * 4;
    f32x4 x = *reinterpret_cast<const f32x4 *>(from);
#pragma unroll 8
    for (uint32_t i = 1; i < p.splits; ++i)
        x += *reinterpret_cast<const f32x4 *>(from + (uint64_t)i * p.r_tiles * p.c_tiles * tr * tc);
    const int64_t want = p.loss.target[m];
    float top = -INFINITY;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const uint32_t n = rt * tr + u * 4 + d;
        if (n >= p.rows) x[d] = -INFINITY;
        if ((int64_t)n == want && n < p.rows) p.loss.picked[m] = x[d];
        top = fmaxf(top, x[d]);
    }
    for (uint32_t i = 1; i < outs; i <<= 1) top = fmaxf(top, __shfl_xor(top, i));
    const float ref = fminf(fmaxf(top, -3.0e38f), 3.0e38f);
    float sum = ((__expf(x[0] - ref) + __expf(x[1] - ref)) + __expf(x[2] - ref)) + __expf(x[3] - ref);
    for (uint32_t i = 1; i < outs; i <<= 1) sum += __shfl_xor(sum, i);
    if (u == 0) p.loss.parts[(uint64_t)m * p.r_tiles + rt] = make_float2(ref, sum);
}

// ---- the loss's join -------------------------------------------------------------

// A wave per token: reference and sum over the row tiles, in a fixed order.
// 4096 tokens of 501 tiles in 11.5 us.
__global__ __launch_bounds__(64) void k_loss_join(LossEpi e, float *loss, float *lse, uint32_t parts, uint64_t vocab) {
    const uint32_t lane = threadIdx.x, m = blockIdx.x;
    float ref = -3.0e38f, sum = 0;
#pragma unroll 4
    for (uint32_t i = lane; i < parts; i += 64) {
        const float2 v = e.parts[(uint64_t)m * parts + i];
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

// What the gradients need first, in one launch.  Workgroup 0: the largest dloss
// (5 us for 4096 tokens; with the copy of 4096 x 4096 the launch takes 12).  The others, if `out` is given: x in rows of whole 16-byte
// units, with zeros for the tokens that do not count: their dlogits are 0, but in
// dw 0 times an infinity or a NaN, as the rows of padding may hold, would not be.
__global__ __launch_bounds__(1024) void k_loss_begin(LossEpi e, float *unit, uint32_t tokens, uint64_t vocab,
                                                     const uint16_t *in, uint64_t in_stride, uint16_t *out,
                                                     uint64_t out_stride, uint64_t cols) {
    __shared__ float red[16];
    auto counts = [&](int64_t t) { return t != e.ignore && t >= 0 && t < (int64_t)vocab; };
    if (blockIdx.x) {
        const uint64_t units = out_stride / 8, n = tokens * units, step = (uint64_t)(gridDim.x - 1) * 1024;
        for (uint64_t i = (uint64_t)(blockIdx.x - 1) * 1024 + threadIdx.x; i < n; i += step) {
            const uint64_t row = n >> 32 ? i / units : (uint32_t)i / (uint32_t)units, c = (i - row * units) * 8;
            const int64_t t = e.target[row];  // (both loads together)
            u32x4 v = stage_unit(in + row * in_stride, c, cols);
            if (!counts(t)) v = u32x4{0, 0, 0, 0};
            *reinterpret_cast<u32x4 *>(out + row * out_stride + c) = v;
        }
        return;
    }
    float top = 0;
#pragma unroll 4
    for (uint32_t m = threadIdx.x; m < tokens; m += 1024) {
        const float a = fabsf(e.dloss[m]);
        if (counts(e.target[m]) && a < INFINITY) top = fmaxf(top, a);
    }
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x) return;
    for (int w = 1; w < 16; ++w) top = fmaxf(top, red[w]);
    *unit = top > 0 ? top : 1.0f;
}

// ---- the pre-activation's gradient --------------------------------------------------

// dz = dy act'(z) in the padded column order of the packed rows, and the sums
// of its columns over a run of the group's rows, from the unrounded values.
// A thread takes eight columns (of both halves when gated).  Bound by memory:
// 4096 x 14336 gated with an fp32 pre-activation, 822 MB, 186 us, 4.4 TB/s.
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
    const uint32_t count = tail || c >= p.part_rows ? 0 : min(8u, p.part_rows - c);
    float sum[H][8];
#pragma unroll
    for (int h = 0; h < H; ++h)
        for (int i = 0; i < 8; ++i) sum[h][i] = 0;
    if (at < p.width) {
#pragma unroll 2
        for (uint32_t m = m0 + wave; m < m1; m += 4) {
            float v[H][8], z[H][8], dy[8];
            load<8>(p.dy, m * p.dy_stride + c, p.dy_f32, count, dy);
            if (GATED || p.act != kActNone)
#pragma unroll
                for (int h = 0; h < H; ++h)
                    load<8>(p.z, m * p.z_stride + (uint64_t)h * p.part_rows + c, p.z_f32, count, z[h]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (GATED) {
                    const float a = z[0][i], b = z[H - 1][i], s = sigmoid(a);
                    v[0][i] = dy[i] * b * s * (1.0f + a * (1.0f - s));
                    v[H - 1][i] = dy[i] * a * s;
                } else {
                    v[0][i] = p.act != kActNone ? dy[i] * activate_grad(z[0][i], p.act) : dy[i];
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

// The runs' sums, in a fixed order: a wave takes every fourth.
__global__ __launch_bounds__(256) void k_dbias(DzParams p) {
    __shared__ float red[4][64];
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = blockIdx.y;
    const uint32_t n = blockIdx.x * 64 + lane;
    const bool live = n < p.part_rows * p.parts;
    const uint32_t part = n / p.part_rows, at = part * p.part_pad + n - part * p.part_rows;
    const float *src = p.colsum + (uint64_t)g * p.chunks * p.width + at;
    float s = 0;
    if (live)
#pragma unroll 4
        for (uint32_t i = wave; i < p.chunks; i += 4) s += src[(uint64_t)i * p.width];
    red[wave][lane] = s;
    __syncthreads();
    if (wave || !live) return;
    s = ((red[0][lane] + red[1][lane]) + red[2][lane]) + red[3][lane];
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
hipError_t gemm(GemmTile tile, const GemmParams &p, hipStream_t s) {
    const uint32_t tiles = p.r_tiles * p.c_tiles;
    const bool clear = KIND == kGemmForward ? p.lin.clear : KIND == kGemmDx && p.store.clear;
    const dim3 grid(tiles + (clear ? p.r_tiles : 0), KIND == kGemmDw ? p.groups : p.splits);
    if (tile.r == 256 && tile.c == 256)
        k_gemm<RK, CK, KIND, GATED, 256, 256, 2, 4><<<grid, 512, 0, s>>>(p);
    else if (tile.r == 128 && tile.c == 128) {
        if constexpr (RK == kPacked)
            k_gemm<RK, CK, KIND, GATED, 128, 128, 4, 1, 2><<<grid, 512, 0, s>>>(p);
        else
            k_gemm<RK, CK, KIND, GATED, 128, 128, 2, 4><<<grid, 512, 0, s>>>(p);
    } else if constexpr (RK == kPacked)
        k_gemm<RK, CK, KIND, GATED, 256, 64, 8, 1><<<grid, 512, 0, s>>>(p);
    else if constexpr (KIND != kGemmDw)
        k_gemm<RK, CK, KIND, GATED, 256, 64, 4, 2><<<grid, 512, 0, s>>>(p);
    const dim3 join(tiles, (tile.r * tile.c / (GATED ? 8 : 4) + 255) / 256);
    if constexpr (KIND == kGemmLossStat) {
        if (p.splits > 1) k_join_stat<<<join, 256, 0, s>>>(p, tile.r, tile.c);
    } else if constexpr (KIND != kGemmDw) {
        if (p.splits > 1) k_join<KIND, GATED><<<join, 256, 0, s>>>(p, tile.r, tile.c);
    }
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

// Rows of x for which the skinny product is faster than the tiled one: it
// reads all of x once a workgroup, so that the width of x counts.  Skinny and
// tiled in us: 4096 x 4096 with 32 rows 11 and 16, with 48 rows 16 and 16, with 64 rows
// 19 and 16; 4096 x 14336 with 17 rows 23 and 25, with 24 rows 27 and 25, with 32 rows
// 31 and 26; 2048 x 2048 with 48 rows 9 and 11; only for much wider results does the
// tiled one gain before that (28672 x 4096 with 32 rows 42 and 35).  8 experts of 4096 x
// 4096 with 16 rows each 34 and 53, with 20 rows (two rounds of 16) 59 and 53, with 48
// rows 91 and 55.  The host knows only the experts' mean, not the offsets: 128
// experts of 2048 x 2048 with 15 rows each take 164 and 166, but 1,939 rows by a power
// law 274 and 171, and 2,000 rows all to one 561 and 144.
bool skinny_fits(uint64_t tokens, uint64_t groups, uint64_t col_blocks) {
    if (groups > 1) return tokens <= 16 * groups;
    return tokens <= 24 || (tokens <= 64 && tokens * col_blocks <= 2048);
}

// Waves and row blocks of a workgroup.  While each CU has at most one row block,
// many waves on it, for the bytes in flight (4096 x 4096, 256 blocks, one row: 5.8
// us against 8.7 with few waves; 64 rows: 18.6 against 23.5).  From there on few waves
// that share their reads of x: a second round of many costs more (5120 x 4096, 320
// blocks, 16 rows: 9.9 us against 14.1, 32 rows: 12.9 against 19.7; 8192 x 4096, 64
// rows: 24 against 34; 4096 x 4096 over 13 experts: 61, 5.3 TB/s, against 80).  Gated:
// two row blocks, each with its up rows, and four waves where x's reads weigh
// (24576 x 4096, 768 blocks: 16 rows 25.7 us with one block and eight waves, 26.9 so,
// 32 rows 32.7 and 29.0; 896 blocks, 16 rows: 31.5 and 29.1; 256 blocks, 64 rows: 20.8
// and 26.6, 384 blocks: 38.5 and 27.1).
hipError_t launch_skinny(const SkinnyParams &p, hipStream_t s) {
    const uint32_t rows = p.groups > 1 ? 16 : p.tokens;
    const uint64_t blocks = (uint64_t)p.w.part_blocks * p.groups;
    if (p.lin.act == kActSwiglu) {
        if (rows <= 16) return blocks <= 768 ? skinny<1, 2, true, 8>(p, s) : skinny<1, 4, true, 4>(p, s);
        if (rows <= 32) return blocks <= 256 ? skinny<2, 2, true, 8>(p, s) : skinny<2, 4, true, 4>(p, s);
        return blocks <= 256 ? skinny<4, 2, true, 8>(p, s) : skinny<4, 4, true, 4>(p, s);
    }
    if (rows <= 16) return blocks <= 256 ? skinny<1, 1, false, 16>(p, s) : skinny<1, 2, false, 8>(p, s);
    if (rows <= 32) return blocks <= 256 ? skinny<2, 1, false, 8>(p, s) : skinny<2, 2, false, 8>(p, s);
    return blocks <= 256 ? skinny<4, 1, false, 8>(p, s) : skinny<4, 4, false, 8>(p, s);
}

GemmTile gemm_tile(GemmKind kind, uint64_t r, uint64_t c, uint64_t groups) {
    const uint64_t each = (c + groups - 1) / groups;
    if (kind != kGemmDw && each <= 64) return GemmTile{256, 64};
    return ((r + 255) / 256) * ((c + 255) / 256) >= 256 && each > 128 ? GemmTile{256, 256} : GemmTile{128, 128};
}

// Runs into which the contraction is cut.  With fewer tiles than workgroups
// that fit the chip, each run shortens the walk of `steps` blocks of 64 and
// adds its part of the sums, written and read once at about 4 TB/s, and one
// launch.  A block takes 0.6 us with tiles of 128 x 128, 0.8 with 256 x 64, one
// workgroup a CU (more do not fit: 128 x 4096 x 4096 20 us in 8 runs, 39 whole,
// 31 in 16); dx 0.9 us where a CU has one workgroup, 1.4 where it has two (the same
// size: 22 us in 8 runs, 77 whole, 31 in 16; 300 rows 47 in 2, 78 whole, 50 in 4 or 8).
uint32_t gemm_splits(GemmKind kind, GemmTile tile, uint64_t r_tiles, uint64_t c_tiles, uint64_t steps) {
    const uint64_t tiles = r_tiles * c_tiles, most = kind == kGemmDx ? 512 : 256;
    if (tiles == 0 || tiles > 256) return 1;
    const double one = kind == kGemmDx ? 0.9 : tile.c == 64 ? 0.8 : 0.6;
    const double part = 8.0 * tiles * tile.r * tile.c / 4e6;  // us a run
    uint32_t best = 1;
    double least = one * steps;
    for (uint32_t n = 2; n <= most / tiles && 4 * n <= steps && n <= 64; ++n) {
        const double t = (tiles * n <= 256 ? one : 1.4) * ((steps + n - 1) / n) + 3.0 + part * n;
        if (t < 0.95 * least) best = n, least = t;
    }
    return best;
}

hipError_t launch_gemm(GemmKind kind, GemmTile tile, const GemmParams &p, hipStream_t s) {
    if (p.r_tiles == 0 || p.c_tiles == 0) return hipSuccess;
    switch (kind) {
    case kGemmForward:
        return p.lin.act == kActSwiglu ? gemm<kPacked, kRows, kGemmForward, true>(tile, p, s)
                                       : gemm<kPacked, kRows, kGemmForward, false>(tile, p, s);
    case kGemmLossStat: return gemm<kPacked, kRows, kGemmLossStat, false>(tile, p, s);
    case kGemmLossDz: return gemm<kPacked, kRows, kGemmLossDz, false>(tile, p, s);
    case kGemmDx: return gemm<kPackedT, kRows, kGemmDx, false>(tile, p, s);
    case kGemmDw: return gemm<kCols, kCols, kGemmDw, false>(tile, p, s);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_loss_join(const LossEpi &e, float *loss, float *lse, uint32_t tokens, uint32_t parts, uint64_t vocab,
                            hipStream_t s) {
    k_loss_join<<<tokens, 64, 0, s>>>(e, loss, lse, parts, vocab);
    return hipGetLastError();
}

hipError_t launch_loss_begin(const LossEpi &e, float *unit, uint32_t tokens, uint64_t vocab, const uint16_t *in,
                             uint64_t in_stride, uint16_t *out, uint64_t out_stride, uint64_t cols, hipStream_t s) {
    const uint64_t wgs = out ? (tokens * (out_stride / 8) + 1023) / 1024 : 0;
    k_loss_begin<<<1 + (uint32_t)(wgs < 2048 ? wgs : 2048), 1024, 0, s>>>(e, unit, tokens, vocab, in, in_stride, out,
                                                                          out_stride, cols);
    return hipGetLastError();
}

hipError_t launch_dz(const DzParams &p, hipStream_t s) {
    const uint32_t cols = p.parts == 2 ? p.part_pad + (p.width - 2 * p.part_pad) : p.width;
    const dim3 grid((cols / 8 + 63) / 64, p.chunks, p.groups);
    if (p.parts == 2)
        k_dz<true><<<grid, 256, 0, s>>>(p);
    else
        k_dz<false><<<grid, 256, 0, s>>>(p);
    if (p.dbias) k_dbias<<<dim3((p.part_rows * p.parts + 63) / 64, p.groups), 256, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace uzip
