// Host-side declarations shared by the W8A8 entry points (w8a8_api.cu) and kernels
// (gemm_w8a8.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/w4a8.h"
#include "w4a8_common.cuh"

namespace w4a8 {

// Packed W8A8 weights: a 256-byte header, the fp32 scales of every tile row
// [E][NT][128], then one block of 128 rows x 128 bytes per (matrix, 128-row tile, 128-wide
// K plane), each row's 16-byte chunk c at chunk position c ^ (row & 7) (act_tiled_offset).
constexpr int kW8BlockBytes = kTileRows * kGroup;
constexpr uint32_t kW8PackMagic = 0x38413857u;  // "W8A8"
constexpr int kW8StatusWords = 1024;
// INT32 holds the sum of kW8MaxK products: packed weights are within +-127, activation codes
// within -128 .. 127, so at most 127 * 128 * 2^17 = 2130706432 < 2^31
constexpr int kW8MaxK = 1 << 17;
inline size_t w8_blocks_offset(int E, int NT) { return (size_t)kHeaderBytes + (size_t)E * NT * kTileRows * 4; }
inline int w8_tiles(int N, int layout) {
    return layout == W4A8_LAYOUT_GATEUP ? ceil_div(N / 2, kTileRows / 2) : ceil_div(N, kTileRows);
}

enum { kW8Dense = 0, kW8Up = 1, kW8Down = 2 };

// Device arguments of one W8A8 GEMM launch (one projection of every expert, or a dense layer).
struct W8Args {
    int NT, G;                // 128-row tiles and 128-wide K planes per weight matrix
    const float* wscale;      // fp32 scale per tile row [E][NT][128]
    const float* act_scale;   // token scale per row
    const int4* mt_tab;       // grouped: per row tile (expert, first row, rows, 0); dense: null
    const int* n_mtiles;      // grouped: number of row tiles (device)
    int M;                    // dense: rows
    int BN;                   // tokens per row tile at most (the plan's)
    int mode;                 // kW8Dense / kW8Down: scaled output of out_type; kW8Up: SwiGLU -> bf16 h
    int out_type;             // W8A8_F32, ...
    void* out;
    int ldo;
    int nvalid;               // valid output columns (N, or F for kW8Up)
    const float* bias;        // optional, [nvalid]
    uint32_t* err;            // device error word (grouped), or null and
    uint32_t* status;         // kW8StatusWords words, one per CTA (dense), or null
    long long wait_limit;     // clock cycles a bounded wait may last
    uint32_t debug;           // test hook
    // set by the launcher
    int out_kind;             // the epilogue's variant
    int NP, nmt;              // weight tiles (of cg * 128 channels) per matrix; dense: row tiles
    int ns;                   // shared-memory stages
    uint32_t b_stage, recv;   // bytes of a stage's token block and of the K split's receive buffer
    int box_rows, small_rows; // token rows of the tile's tensor-map box and of the small one (0: none)
    // tensor-map coordinates of token row r in K plane g: (g * plane_x, r / row_unit + g * plane_y)
    int plane_x, plane_y, row_unit;
};

// What the tensor maps are built from.
struct W8Operands {
    const uint8_t* wblocks;   // packed weight blocks
    int matrices;             // number of weight matrices
    const int8_t* x;          // dense: rows of G * 128 bytes; grouped: tiled rows [G][x_rows][128]
    int x_rows;
};

// Tile shape: cg CTAs work on cg * 128 channels x up to bn tokens; split > 1 (cg = 1, dense):
// as many CTAs share a tile's K planes.
struct W8Plan {
    int cg, bn, split;
};

// the tile shape for both projections of nslots rows over E experts (weight tiles and K planes
// of each); the permutation's row-tile table must be built with bn
W8Plan w8_plan_grouped(int nslots, int E, int NT_up, int G_up, int NT_down, int G_down, int num_ctas);
// grouped: the plan of the row-tile table; dense (null): the launcher chooses
cudaError_t launch_gemm_w8a8(W8Args a, const W8Operands& op, const W8Plan* grouped, int num_ctas, cudaStream_t stream);
cudaError_t launch_pack_w8(const uint16_t* w, int E, int N, int K, int layout, uint8_t* packed, int8_t* codes, float* scale,
                           cudaStream_t stream);

}  // namespace w4a8
