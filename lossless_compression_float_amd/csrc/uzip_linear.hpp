// uzip_linear.hpp -- layout of packed weights, kernel parameter blocks and
// launchers of the products that read them (internal).
//
// A packed weight stack holds E matrices of N rows and K columns in bf16,
// without loss.  Its unit is a tile of 16 rows by 64 columns, in the order in
// which a wave's lanes feed the matrix instructions: lane l = 16 q + r holds
// of row r the columns 8 q + j and 32 + 8 q + j, j = 0 .. 7.  Every value keeps its sign and mantissa
// byte; its exponent e is a 4-bit code base - e within the tile's window of 16
// exponents (or of 15, code 15 then standing for exponent 0).  The few values
// outside the window are listed; a tile with more than kMaxListed of them
// keeps its exponents as bytes.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

#include "uzip.h"

namespace uzip {

constexpr uint32_t kTileRows = 16;
constexpr uint32_t kTileCols = 64;
constexpr uint32_t kTileBytes = 1536;  // 1024 sign+mantissa bytes, 512 bytes of codes
constexpr uint32_t kTileSm = 1024;
constexpr uint32_t kMaxListed = 64;    // one list entry a lane
constexpr uint32_t kInline = 2;
constexpr uint32_t kTileRaw = 255;     // count field of a tile that keeps exponent bytes
constexpr uint32_t kTileZero = 1u << 16;  // code 15 stands for exponent 0
constexpr uint32_t kWeightHeader = 256;
constexpr uint32_t kWeightMagic = 0x31575A55u;  // "UZW1"
constexpr uint32_t kScanTiles = 1024;  // tiles per block of the offset scan

// Tile header: word 0: base exponent, count << 8, flags; word 1: offset of the
// tile's list (u32 entries: position | bits << 16) or exponent bytes, in
// 16-byte units from the start of the extra region; words 2 and 3: the list's
// first entries.  A list of up to kInline entries is only there, so that a
// product hardly ever waits for one: of 1024 normal values 0.05 are listed on
// average.
struct WeightLayout {
    uint64_t parts;      // 2 when gated: gate rows, then up rows, each padded to whole tiles
    uint64_t part_rows;  // rows of one part
    uint64_t part_blocks;
    uint64_t row_blocks;  // of one matrix
    uint64_t col_blocks;
    uint64_t tiles;       // of the whole stack
    uint64_t head_off;    // 16 bytes a tile
    uint64_t tile_off;
    uint64_t extra_off;
    uint64_t max_bytes;
};

inline WeightLayout weight_layout(uint64_t matrices, uint64_t rows, uint64_t cols, bool gated) {
    WeightLayout l;
    l.parts = gated ? 2 : 1;
    l.part_rows = rows / l.parts;
    l.part_blocks = (l.part_rows + kTileRows - 1) / kTileRows;
    l.row_blocks = l.parts * l.part_blocks;
    l.col_blocks = (cols + kTileCols - 1) / kTileCols;
    l.tiles = matrices * l.row_blocks * l.col_blocks;
    l.head_off = kWeightHeader;
    l.tile_off = (l.head_off + 16 * l.tiles + 255) / 256 * 256;
    l.extra_off = l.tile_off + kTileBytes * l.tiles;
    l.max_bytes = l.extra_off + 1024 * l.tiles;
    return l;
}

// What kernels know of a packed stack.
struct WeightView {
    const uint4 *head;
    const uint8_t *tiles;
    const uint8_t *extra;
    uint32_t extra_units;  // 16-byte units readable at `extra`
    uint32_t part_rows, part_blocks, row_blocks, col_blocks;
    uint32_t parts;
};

struct PackParams {
    const uint16_t *in;
    uint64_t row_stride, matrix_stride;
    uint8_t *out;
    uint64_t *out_size;
    uint64_t *sums;  // workspace: extra units before each block of kScanTiles tiles
    WeightLayout l;
    uint64_t matrices, rows, cols;
    uint32_t gated;
};

struct UnpackParams {
    WeightView w;
    uint16_t *out;
    uint64_t row_stride, matrix_stride;
    uint64_t tiles;
    uint32_t cols;
};

// A matrix of bf16 (or, where said, fp32) values in memory.
struct Mat {
    const void *p;
    uint64_t stride;  // values between rows
};

enum ActKind { kActNone = 0, kActRelu, kActGelu, kActGeluTanh, kActSilu, kActSwiglu };

// The forward product's epilogue.
struct LinearEpi {
    const void *bias;       // matrices * rows values, or null
    const void *residual;   // y's type and shape, or null
    void *y;
    void *preact;           // or null
    uint64_t residual_stride, y_stride, preact_stride;
    uint32_t bias_f32, y_f32, preact_f32, act;
    uint32_t clear;         // zeros in y's and the pre-activation's rows of no group
};

// The loss's epilogues.
struct LossEpi {
    const int64_t *target;
    int64_t ignore;
    float2 *parts;       // (reference, sum) of every token and row tile
    float *picked;       // the target's logit
    const float *lse;    // backward
    const float *dloss;
    const float *unit;   // backward: the largest dloss, by which dz is divided
    uint16_t *dz;        // backward: one piece's gradient of the logits
    uint64_t dz_stride;
};

// The gradients' epilogue: bf16, optionally added up in fp32 over pieces.
struct StoreEpi {
    uint16_t *out;       // null while pieces remain
    float *sum;          // fp32 running sums, or null
    const float *unit;   // the results' factor, or null
    uint64_t stride, sum_stride;
    uint32_t add;        // read the running sums first
    uint32_t clear;      // zeros in the rows of no group
};

struct GemmParams {
    WeightView w;
    Mat rmat, cmat;         // operands in memory (those that are not weights)
    const int32_t *offsets; // grouped: matrices + 1 row offsets
    uint32_t groups;        // matrices (1 without offsets)
    uint32_t tokens;        // rows of x
    uint32_t r_tiles, c_tiles;
    uint32_t r_limit, c_limit;   // columns of rmat / cmat that can be read, multiples of 8; of a contraction, of 64
    uint32_t steps;         // contraction blocks of 64
    uint32_t splits;        // runs of them, each a workgroup's (1: none)
    float *part;            // their parts of the sums
    uint32_t row_block0;    // first row block of a piece of the weight
    uint32_t row_blocks;    // row blocks of the piece
    uint32_t rows, cols;    // N (all parts) and K of one matrix
    LinearEpi lin;
    LossEpi loss;
    StoreEpi store;
};

struct SkinnyParams {
    WeightView w;
    Mat x;
    const int32_t *offsets;
    uint32_t groups, tokens, rows, cols;
    LinearEpi lin;
};

struct DzParams {
    const void *dy;
    uint64_t dy_stride;
    const void *z;
    uint64_t z_stride;
    uint16_t *dz;        // null: only the bias gradient is wanted
    uint64_t dz_stride;
    float *colsum;       // [row chunks][groups? 1][width] partial sums, or null
    const int32_t *offsets;
    uint32_t groups, tokens;
    uint32_t part_rows, part_pad, parts, width;  // width: padded columns of dz
    uint32_t dy_f32, z_f32, act, chunks;
    void *dbias;
    uint32_t dbias_f32;
};

hipError_t launch_pack(const PackParams &p, hipStream_t s);
hipError_t launch_unpack(const UnpackParams &p, hipStream_t s);
hipError_t launch_stage(const uint16_t *in, uint64_t in_stride, uint16_t *out, uint64_t out_stride, uint64_t rows,
                        uint64_t cols, hipStream_t s);
hipError_t launch_skinny(const SkinnyParams &p, hipStream_t s);
bool skinny_fits(uint64_t tokens, uint64_t groups, uint64_t col_blocks);
enum GemmKind { kGemmForward, kGemmLossStat, kGemmLossDz, kGemmDx, kGemmDw };
// Outputs of a workgroup: r by c.
struct GemmTile {
    uint32_t r, c;
};
// The tile of a product with `r` by `c` outputs, c in all of `groups` groups.
GemmTile gemm_tile(GemmKind kind, uint64_t r, uint64_t c, uint64_t groups);
// Runs of the contraction (all but dw).
uint32_t gemm_splits(GemmKind kind, GemmTile tile, uint64_t r_tiles, uint64_t c_tiles, uint64_t steps);
hipError_t launch_gemm(GemmKind kind, GemmTile tile, const GemmParams &p, hipStream_t s);
hipError_t launch_loss_join(const LossEpi &e, float *loss, float *lse, uint32_t tokens, uint32_t parts, uint64_t vocab,
                            hipStream_t s);
// The largest finite |dloss| of the tokens that count (1 where all are 0); with `out`, x is staged there with zeros for
// those that do not.
hipError_t launch_loss_begin(const LossEpi &e, float *unit, uint32_t tokens, uint64_t vocab, const uint16_t *in,
                             uint64_t in_stride, uint16_t *out, uint64_t out_stride, uint64_t cols, hipStream_t s);
hipError_t launch_dz(const DzParams &p, hipStream_t s);

}  // namespace uzip
