// uzip_args.hpp -- host code that the C entry points of the operators on
// packed weights share: argument checks and workspace carving (internal).
#pragma once

#include <stdint.h>

#include <algorithm>

#include <hip/hip_runtime.h>

#include "uzip.h"
#include "uzip_linear.hpp"

namespace uzip {
namespace {

constexpr uint64_t kAlign = 256;
constexpr uint64_t kMaxDim = 0x7FFFFFFF;
constexpr uint64_t kMaxMatrices = 65535;
constexpr uint64_t kMaxTiles = 1ull << 25;
// Limits of a call: its launch grids stay within the 2^32 - 1 work-items of one
// grid dimension (512 threads a tile of at least 128 by 64 outputs).
constexpr uint64_t kMaxTokens = 1ull << 25;
constexpr uint64_t kMaxOutputTiles = 1ull << 22;
// and a tile's rows, up to 256 of these, are addressed with 32 bits.
constexpr uint64_t kMaxWide = (1ull << 22) - 512;

uint64_t up(uint64_t v, uint64_t a) { return (v + a - 1) / a * a; }
uint64_t blocks(uint64_t v, uint64_t a) { return (v + a - 1) / a; }
bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool dims_ok(uint64_t matrices, uint64_t rows, uint64_t cols, uint32_t gated) {
    if (matrices == 0 || rows == 0 || cols == 0 || gated > 1 || (gated && rows % 2)) return false;
    if (matrices > kMaxMatrices || rows > kMaxDim || cols > kMaxDim) return false;
    const uint64_t tiles = (gated + 1) * blocks(rows / (gated + 1), kTileRows) * blocks(cols, kTileCols);
    return tiles <= kMaxTiles / matrices;
}

bool weight_ok(const uzip_weight *w) {
    return w && w->reserved == 0 && dims_ok(w->matrices, w->rows, w->cols, w->gated) && w->data && aligned(w->data, 16) &&
           w->bytes >= weight_layout(w->matrices, w->rows, w->cols, w->gated).extra_off;
}

WeightView view(const uzip_weight *w) {
    const WeightLayout l = weight_layout(w->matrices, w->rows, w->cols, w->gated);
    const uint8_t *p = static_cast<const uint8_t *>(w->data);
    WeightView v{};
    v.head = reinterpret_cast<const uint4 *>(p + l.head_off);
    v.tiles = p + l.tile_off;
    v.extra = p + l.extra_off;
    v.extra_units = (uint32_t)std::min<uint64_t>((w->bytes - l.extra_off) / 16, 0xFFFFFFFFu);
    v.part_rows = (uint32_t)l.part_rows;
    v.part_blocks = (uint32_t)l.part_blocks;
    v.row_blocks = (uint32_t)l.row_blocks;
    v.col_blocks = (uint32_t)l.col_blocks;
    v.parts = (uint32_t)l.parts;
    return v;
}

// A matrix argument of `cols` values a row.
bool mat_ok(const void *p, uint64_t stride, uint64_t rows, uint64_t cols, uint32_t elem) {
    if (rows == 0) return true;
    return p && aligned(p, elem) && stride >= cols && stride < (1ull << 40);
}

// Whether products of `tokens` rows with this weight, and their gradients, fit the limits.
bool call_ok(const uzip_weight *w, uint64_t tokens) {
    const uint64_t wide = std::max(blocks(w->rows, 128) + 1, blocks(w->cols, 128));
    return w->rows <= kMaxWide && w->cols <= kMaxWide && tokens <= kMaxTokens && wide * (tokens / 64 + w->matrices + 1) <= kMaxOutputTiles;
}

bool type_ok(uint32_t t) { return t == UZIP_BF16 || t == UZIP_FP32; }
uint32_t type_size(uint32_t t) { return t == UZIP_FP32 ? 4 : 2; }

// Whether a bf16 matrix can be read 16 bytes at a time, and whether the tiled
// product can: a tile's rows are addressed with 32 bits.
bool by16(const void *p, uint64_t stride, uint64_t cols) { return aligned(p, 16) && stride % 8 == 0 && cols % 8 == 0; }
bool tiled(const void *p, uint64_t stride, uint64_t cols) { return by16(p, stride, cols) && stride < (1u << 22); }

// Carves a workspace; with a null base it only counts.
struct Carver {
    uint8_t *base;
    uint64_t used = 0;
    explicit Carver(void *ws) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(ws);
        base = ws ? reinterpret_cast<uint8_t *>((p + kAlign - 1) & ~(uintptr_t)(kAlign - 1)) : nullptr;
    }
    template <class T>
    T *take(uint64_t n) {
        uint8_t *p = base ? base + used : nullptr;
        used += up(n * sizeof(T), kAlign);
        return reinterpret_cast<T *>(p);
    }
    uint64_t bytes() const { return used ? used + kAlign : 0; }  // slack: the caller's pointer need only be 16-byte aligned
};

bool workspace_ok(void *ws, uint64_t have, uint64_t need) { return need == 0 || (ws && aligned(ws, 16) && have >= need); }

uzip_status done(hipError_t e) { return e == hipSuccess ? UZIP_OK : UZIP_ERR_DEVICE; }

}  // namespace
}  // namespace uzip
