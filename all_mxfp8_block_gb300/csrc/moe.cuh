// Launchers of the mixture-of-experts row kernels (moe.cu) and the MX
// quantiser (quantize.cu).  All return the cudaError_t of their launch.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace mxa2a {

struct MoeSort {
    long long assignments;   // tokens * topk
    long long rows;          // length of src
    int experts, align;
    const int32_t* expert;
    int32_t *offsets, *counts, *pos, *src;   // src may be null
};
cudaError_t launch_moe_sort(const MoeSort& a, cudaStream_t stream);

// expert segments in the sorted rows, as the sort wrote them
struct Segments {
    const int32_t *offsets, *counts;
    int experts;
    long long rows;          // rows that the row buffers hold: nothing past them is touched
};

struct MoeDispatch {
    long long tokens, hidden, ldx;
    int topk;
    const void* x;
    const int32_t* pos;
    Segments seg;
    void* out;
    uint8_t* out_scale;      // MX outputs: scale tiles
    int x_type, out_type;
};
cudaError_t launch_moe_dispatch(const MoeDispatch& a, cudaStream_t stream);

struct MoeCombine {
    long long tokens, hidden, rows;
    int topk;
    const void* y;
    const int32_t* pos;
    const float* weight;     // null: 1
    const void* residual;    // null: none
    void* out;
    int type;
    int sms;                 // SMs of the device
};
cudaError_t launch_moe_combine(const MoeCombine& a, cudaStream_t stream);

struct MoeCombineBackward {
    long long tokens, hidden;
    int topk;
    const void *dout, *y;
    const int32_t* pos;
    const float* weight;
    Segments seg;
    void* dy;
    float* dweight;
    int type;
};
cudaError_t launch_moe_combine_backward(const MoeCombineBackward& a, cudaStream_t stream);

struct Quantize {
    const void* x;           // [groups][rows][cols], row stride ldx
    int x_type;
    long long ldx;
    int groups;
    long long rows, cols;
    int e5m2;
    uint8_t *codes, *scale;      // along the columns (null: not wanted)
    uint8_t *codes_t, *scale_t;  // transposed, along the rows (null: not wanted)
    // the linear layer's gradient: x is dY, the quantised value dY * act'(preact)
    // inside the segments' tokens and 0 elsewhere, its column sums per 32 rows in colsum
    const void* preact;          // bf16 [rows][cols], null for no activation
    int act;
    Segments seg;                // offsets null: all rows
    float* colsum;               // [ceil(rows / 32)][cols], null: plain quantisation
};
cudaError_t launch_quantize(const Quantize& q, cudaStream_t stream);
// per-group sums of the colsum blocks: dbias[g][n] = sum over the group's 32-row blocks, in order
cudaError_t launch_bias_sums(const float* colsum, const Segments& seg, long long cols, float* dbias, cudaStream_t stream);
// E8M0 bytes [groups][rows][blocks] to scale tiles
cudaError_t launch_scale_tiles(const uint8_t* s, int groups, long long rows, long long blocks, uint8_t* tiles,
                               int sms, cudaStream_t stream);

}  // namespace mxa2a
