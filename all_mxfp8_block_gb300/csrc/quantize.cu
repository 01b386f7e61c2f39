// MX quantisation of rows and of columns (transposed), the linear layer's
// gradient through its activation with both quantisations and the bias sums
// in the same pass, and the reordering of plain scale rows into scale tiles.
#include <algorithm>

#include "moe.cuh"
#include "mxquant.cuh"

namespace mxa2a {

namespace {

// A CTA takes a tile of kTileRows x kTileCols elements, read once.  Thread
// (ty, tx) holds 8 consecutive columns of kPass rows: a row's 32-column block
// is 4 threads, its largest value two shuffles.  For the transposed
// quantisation the tile goes through shared memory (rows kTileCols + 1 words
// apart: no bank conflicts either way), and a thread takes one column's 32
// rows.  Bound by the bytes read and written; the tile's codes leave in
// 32-byte pieces (64-byte rows one way, 32 rows' bytes the other).
constexpr int kTileRows = 128, kTileCols = 64, kQThreads = 256;
constexpr int kPass = kTileRows * kTileCols / (kQThreads * 8);
constexpr int kLd = kTileCols + 1;

// segment of row r (offsets ascending), and whether r holds a token of it
__device__ __forceinline__ bool row_is_token(const Segments& s, long long r) {
    int lo = 0, hi = s.experts - 1;   // the last e with offsets[e] <= r
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(s.offsets + mid) <= r) lo = mid; else hi = mid - 1;
    }
    const long long o = __ldg(s.offsets + lo);
    return r >= o && r < o + __ldg(s.counts + lo);
}

template <typename T>
__global__ void __launch_bounds__(kQThreads) quantize_kernel(Quantize q, int row_tiles) {
    __shared__ float tile[kTileRows * kLd];
    __shared__ uint8_t token[kTileRows];
    const int g = (int)(blockIdx.x / row_tiles);
    const long long r0 = (long long)(blockIdx.x % row_tiles) * kTileRows;
    const int c0 = (int)blockIdx.y * kTileCols;
    const int tx = threadIdx.x % (kTileCols / 8), ty = threadIdx.x / (kTileCols / 8);
    const int emax = mx_emax(q.e5m2);
    const bool masked = q.seg.offsets != nullptr;
    if (masked) {
        if (r0 >= __ldg(q.seg.offsets + q.seg.experts)) return;   // past the last segment: nothing is read from there
        if (threadIdx.x < kTileRows)
            token[threadIdx.x] = r0 + threadIdx.x < q.rows && row_is_token(q.seg, r0 + threadIdx.x);
        __syncthreads();
    }
    const T* x = static_cast<const T*>(q.x) + (long long)g * q.rows * q.ldx;
    const int rt = (int)((q.rows + 127) / 128), kb = (c0 + tx * 8) >> 7;
    const int col = c0 + tx * 8;
    const bool in_cols = col < q.cols;   // (columns come in blocks of 32)
    float v[kPass][8];
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
        const long long r = r0 + ty + p * (kTileRows / kPass);
        const bool live = in_cols && r < q.rows && (!masked || token[r - r0]);
        if (live) {
            Vec<T, 8>::load(x + r * q.ldx + col, v[p]);
            if (q.preact) {
                float z[8];
                Vec<__nv_bfloat16, 8>::load(static_cast<const __nv_bfloat16*>(q.preact) + r * q.cols + col, z);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[p][i] *= act_slope(z[i], q.act);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[p][i] = 0.f;
        }
    }
    if (q.codes) {
        uint8_t* codes = q.codes + (long long)g * q.rows * q.cols;
        uint8_t* scale = q.scale + (size_t)g * ((q.cols + 127) / 128) * rt * 512;
#pragma unroll
        for (int p = 0; p < kPass; ++p) {
            const long long r = r0 + ty + p * (kTileRows / kPass);
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[p][i]) & 0x7fffffffu);
            m = max(m, __shfl_xor_sync(kLanes, m, 1));
            m = max(m, __shfl_xor_sync(kLanes, m, 2));
            const uint32_t byte = mx_scale_byte(m, emax);
            const float inv = mx_inv_scale(byte);
            const uint2 w = make_uint2(mx_codes4(v[p], inv, byte == 255, q.e5m2), mx_codes4(v[p] + 4, inv, byte == 255, q.e5m2));
            if (in_cols && r < q.rows) *reinterpret_cast<uint2*>(codes + r * q.cols + col) = w;
            // two blocks of the tile's row in one 16-bit store (a tile is half a scale word wide)
            const uint32_t other = __shfl_xor_sync(kLanes, byte, 4);
            if (tx == 0)   // (rows past the last get scale 0, so that every byte of a tile is written)
                *reinterpret_cast<uint16_t*>(scale + scale_word(kb, r, rt) + ((c0 >> 5) & 3)) =
                    (uint16_t)(byte | (c0 + 32 < q.cols ? other : 0u) << 8);
            // the last tile of columns also clears the word's bytes past the last column
            if (tx == 0 && c0 + kTileCols >= q.cols && (c0 & 64) == 0)
                *reinterpret_cast<uint16_t*>(scale + scale_word(kb, r, rt) + 2) = 0;
        }
    }
    if (!q.codes_t && !q.colsum) return;
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
        float* t = tile + (ty + p * (kTileRows / kPass)) * kLd + tx * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = v[p][i];
    }
    __syncthreads();
    // one column's 32 rows
    const int c = threadIdx.x % kTileCols, rb = threadIdx.x / kTileCols;
    const long long t0 = r0 + rb * 32;
    if (c0 + c >= q.cols) return;
    float u[32];
    uint32_t m = 0;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        u[i] = tile[(rb * 32 + i) * kLd + c];
        m = max(m, __float_as_uint(u[i]) & 0x7fffffffu);
        sum += u[i];
    }
    if (q.colsum && t0 < q.rows) q.colsum[(t0 >> 5) * q.cols + c0 + c] = sum;
    if (!q.codes_t) return;
    const long long ld_t = (q.rows + 31) / 32 * 32;
    const int ct = (int)((q.cols + 127) / 128);
    const uint32_t byte = mx_scale_byte(m, emax);
    const float inv = mx_inv_scale(byte);
    if (t0 < ld_t) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = mx_codes4(u + 4 * i, inv, byte == 255, q.e5m2);
        uint4* o = reinterpret_cast<uint4*>(q.codes_t + ((long long)g * q.cols + c0 + c) * ld_t + t0);
        o[0] = make_uint4(w[0], w[1], w[2], w[3]);
        o[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    uint8_t* scale_t = q.scale_t + (size_t)g * rt * ct * 512;
    scale_t[scale_word((int)(r0 >> 7), c0 + c, ct) + rb] = t0 < ld_t ? (uint8_t)byte : 0;
}

// Columns of the last scale tile past the last column (transposed output):
// their bytes are cleared so that a tile never holds stale bytes.
__global__ void clear_tail_kernel(uint8_t* scale_t, int groups, int rt, int ct, int cols) {
    const int tail = ct * 128 - cols;
    const long long n = (long long)groups * rt * tail;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
        const int c = cols + (int)(i % tail);
        const long long k = i / tail;   // group * rt + row tile
        *reinterpret_cast<uint32_t*>(scale_t + (size_t)(k / rt) * rt * ct * 512 + scale_word((int)(k % rt), c, ct)) = 0;
    }
}

__global__ void bias_sums_kernel(const float* colsum, Segments s, long long cols, float* dbias) {
    const long long c = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const int g = blockIdx.y;
    if (c >= cols) return;
    long long lo = 0, hi = (s.rows + 31) / 32;
    if (s.offsets) {
        lo = max(0, __ldg(s.offsets + g)) / 32;
        hi = min(hi, (long long)__ldg(s.offsets + g + 1) / 32);
    }
    float sum = 0.f;
    for (long long b = lo; b < hi; ++b) sum += __ldg(colsum + b * cols + c);
    dbias[(long long)g * cols + c] = sum;
}

__global__ void scale_tiles_kernel(const uint8_t* s, int groups, long long rows, long long blocks, uint32_t* tiles, int rt, int bt) {
    const long long per = (long long)bt * rt * 128, n = per * groups;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
        const long long g = i / per, j = i % per;
        const int w = (int)(j % 128), row_tile = (int)(j / 128 % rt), kb = (int)(j / 128 / rt);
        const long long r = (long long)row_tile * 128 + (w & 3) * 32 + (w >> 2);
        uint32_t v = 0;
        for (int b = 0; b < 4; ++b)
            if (r < rows && kb * 4 + b < blocks) v |= (uint32_t)s[(g * rows + r) * blocks + kb * 4 + b] << (8 * b);
        tiles[i] = v;
    }
}

}  // namespace

cudaError_t launch_quantize(const Quantize& q, cudaStream_t stream) {
    const int row_tiles = (int)((q.rows + kTileRows - 1) / kTileRows);
    const int ct = (int)((q.cols + 127) / 128);
    const dim3 grid((unsigned)((long long)row_tiles * q.groups), (unsigned)((q.cols + kTileCols - 1) / kTileCols));
    if (q.x_type == kTypeBf16)
        quantize_kernel<__nv_bfloat16><<<grid, kQThreads, 0, stream>>>(q, row_tiles);
    else if (q.x_type == kTypeF16)
        quantize_kernel<__half><<<grid, kQThreads, 0, stream>>>(q, row_tiles);
    else
        quantize_kernel<float><<<grid, kQThreads, 0, stream>>>(q, row_tiles);
    if (q.scale_t && q.cols % 128)
        clear_tail_kernel<<<std::min<long long>(1024, (long long)q.groups * row_tiles), 128, 0, stream>>>(
            q.scale_t, q.groups, row_tiles, ct, (int)q.cols);
    return cudaGetLastError();
}

cudaError_t launch_bias_sums(const float* colsum, const Segments& seg, long long cols, float* dbias, cudaStream_t stream) {
    const dim3 grid((unsigned)((cols + 127) / 128), (unsigned)seg.experts);
    bias_sums_kernel<<<grid, 128, 0, stream>>>(colsum, seg, cols, dbias);
    return cudaGetLastError();
}

cudaError_t launch_scale_tiles(const uint8_t* s, int groups, long long rows, long long blocks, uint8_t* tiles, cudaStream_t stream) {
    const int rt = (int)((rows + 127) / 128), bt = (int)((blocks + 3) / 4);
    const long long words = (long long)groups * rt * bt * 128;
    scale_tiles_kernel<<<(unsigned)std::min<long long>((words + 255) / 256, 152 * 16), 256, 0, stream>>>(
        s, groups, rows, blocks, reinterpret_cast<uint32_t*>(tiles), rt, bt);
    return cudaGetLastError();
}

}  // namespace mxa2a
