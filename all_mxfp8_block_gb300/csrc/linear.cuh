// Interface between the linear layer's C ABI (operators_api.cu) and its GEMM
// kernel (linear.cu).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "kernels.cuh"

namespace mxa2a {

// One grouped block-scaled product
//   out[q][p] = epilogue( sum_c Q[q][c] P[p][c] )
// with P rows on the accumulator's lanes (128 to a tile) and Q rows on its
// columns (tile_q to a tile).  In the layer's forward product and in its input
// gradient P is the weights and Q the tokens; in its weight gradient P is the
// transposed input and Q the transposed output gradient.
struct LinParams {
    int groups;
    int by_contraction;        // 0: Q's rows are grouped, P has groups * p_rows rows;
                               // 1: the contraction is grouped (its range is the segment), out has groups * q_rows rows
    int p_rows, q_rows;        // rows of P per group; rows of Q
    int blocks;                // 32-blocks along the contraction
    int pt, qt;                // tiles of P per group; by_contraction: tiles of Q
    int p_row_tiles;           // 128-row tiles of one group's P scale array
    int q_row_tiles;           // 128-row tiles of Q's scale array
    int splits;                // CTAs of a cluster that share a tile's contraction (1, 2, 4, 8)
    int fmt_p, fmt_q;          // MMA element codes: 0 E4M3, 1 E5M2
    const int32_t *offsets, *counts;   // segments (null: one group of everything)
    const uint8_t *p_scale, *q_scale;
    size_t p_scale_group;      // bytes of one group's P scale tiles
    // epilogue
    const float* bias;         // [groups][p_rows] or null
    int act;
    const uint16_t* residual;  // bf16, laid out as out, or null
    uint16_t* preact;          // bf16, laid out as out, or null
    void* out;
    int out_type;              // kTypeBf16, kTypeF32, kTypeE4M3, kTypeE5M2
    uint8_t* out_scale;        // MX output: scale tiles
    // bounded waits
    DevStatus* status;
    unsigned long long launch_id;
    long long timeout_ns;
};

constexpr int kRoleScale = 7;

// A launch's products: one, or the two of a gradient (rows first, by contraction
// second), which then share the CTAs without a seam between them.  They agree in
// splits and segments.
struct LinMaps {
    CUtensorMap p, q, q32;   // P boxes of 128 rows; Q boxes of linear_q_box(tile_q) rows, of 32 rows (tile_q 256)
};
struct LinPack {
    LinMaps maps[2];
    LinParams p[2];
    int n;
};

// tile_q: 32, 64, 128, or 256 (the CTA-pair kernel: 256 P rows to a tile, ctas
// in pairs, no splits).  ctas: CTAs to launch, a multiple of splits (of 2 for pairs)
cudaError_t launch_linear(const LinPack& k, int tile_q, int ctas, cudaStream_t stream);
inline int linear_q_box(int tile_q) { return tile_q == 256 ? 128 : tile_q; }
inline int linear_p_tile(int tile_q) { return tile_q == 256 ? 256 : 128; }
// CTAs of the kernel that one SM holds at once
int linear_ctas_per_sm(int tile_q);

}  // namespace mxa2a
