// Launches of the 4-bit floating-point products and of the norms around a
// block: what the entry points in strata_moe.hip hand to k_mxfp.hip and
// k_norm.hip.
#pragma once

#include "internal.h"

namespace strata_moe {

constexpr int kF32 = 1, kF16 = 2, kBF16 = 3;  // STRATA_MOE_F32, _F16, _BF16
inline size_t dtype_bytes(int32_t t) { return t == kF32 ? 4 : 2; }

// ---- microscaled 4-bit floating point (k_mxfp.hip)
// A packed matrix: tiles of 16 rows, each its groups of 16 blocks of 32 reduction
// values; a group is the codes of its blocks, 256 bytes each, then its scales.
constexpr int kMxTileRows = 16;
constexpr int kMxBlockBytes = 256;  // codes of 16 rows x 32 values
constexpr int kMxScaleBytes = 256;  // scales of 16 rows x 512 values
constexpr int kMxGroupBytes = 16 * kMxBlockBytes + kMxScaleBytes;
constexpr int kMxMaxCols = 65536, kMxMaxRows = 65536;

inline int64_t mx_tile_bytes(int64_t cols) {
    const int64_t blocks = cols / 32;
    return blocks * kMxBlockBytes + (blocks + 15) / 16 * kMxScaleBytes;
}
// Where step s of a group of `have` blocks begins: step s holds blocks s, 4 + s,
// 8 + s and 12 + s, as far as they exist.
__host__ __device__ inline int mx_step_at(int have, int s) {
    return (s * (have / 4) + (s < have % 4 ? s : have % 4)) * kMxBlockBytes;
}
// Tiles of a matrix of `rows` rows; with paired set, the tiles of its first
// and second half alternate.
inline int64_t mx_tiles(int64_t rows, bool paired) {
    return paired ? 2 * ((rows / 2 + kMxTileRows - 1) / kMxTileRows) : (rows + kMxTileRows - 1) / kMxTileRows;
}

struct MxProduct {
    const uint8_t* codes;   // [x_rows][cols / 2]
    const uint8_t* scales;  // [x_rows][cols / 32]
    int64_t x_rows;
    const uint8_t* packed;
    int64_t stride;         // bytes between experts
    int32_t E, n, cols;     // n: rows of an expert's matrix
    int32_t paired;         // SwiGLU: n / 2 outputs
    const int32_t* offsets; // [E + 1] or null: E == 1, all rows
    const int32_t* src;     // [rows] or null
    int64_t rows;
    void* out;
    int32_t dtype;
    int64_t out_stride;
};
hipError_t launch_mx_quantize(const void* x, int32_t dtype, int64_t x_stride, int64_t rows, int32_t cols,
                              uint8_t* codes, uint8_t* scales, hipStream_t st);
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t cols, void* out,
                                int32_t dtype, int64_t out_stride, hipStream_t st);
hipError_t launch_mx_pack(const uint8_t* codes, const uint8_t* scales, int32_t ne, int32_t rows, int32_t cols,
                          bool paired, uint8_t* packed, int64_t stride, hipStream_t st);
hipError_t launch_mx_product(const MxProduct& p, hipStream_t st);

// ---- norms before and after a block (k_norm.hip)
constexpr int kNormMaxH = 16384;
struct NormScale {
    const float* weight;  // [H] or null: 1
    double offset, eps;
    int32_t on;           // 0: no norm
};
struct NormLaunch {
    int64_t T;
    int32_t H, dtype;     // of h and out
    const void* h;
    int64_t h_stride;
    // the block's output (null y: none, the stream stays h and out is not written)
    const void* y;
    int32_t y_dtype;
    int64_t y_stride, y_rows;
    const int32_t* slot;  // [T][K] or null
    const float* p;       // [T][K]
    int32_t K;
    NormScale after;
    const float* gate;    // or null
    int64_t gate_row_stride, gate_col_stride;
    double residual_scale, block_scale;
    void* out;
    int64_t out_stride;
    // the norm that the (next) block reads
    NormScale before;
    float* x;             // [T][H] or null
    uint8_t* codes;       // [T][H / 2] or null
    uint8_t* scales;      // [T][H / 32]
};
hipError_t launch_norm(const NormLaunch& l, hipStream_t st);

}  // namespace strata_moe
