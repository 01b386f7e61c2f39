// MX quantisation of rows and of columns (transposed), the linear layer's
// gradient through its activation with both quantisations and the bias sums
// in the same pass, and the reordering of plain scale rows into scale tiles.
#include <algorithm>

#include "launch.cuh"
#include "moe.cuh"
#include "mxquant.cuh"

namespace mxa2a {

namespace {

// A CTA takes a tile of 128 rows x 64 columns, read once.  Thread (ty, tx) holds
// 8 consecutive columns of the rows ty, ty + 32, ...: a row's 32-column block is
// 4 threads, its largest value two shuffles.  For the transposed quantisation
// the tile goes through shared memory in 16-byte accesses; a thread then takes
// 8 rows of 4 columns, 4 threads (8 lanes apart) a column's 32 rows.  The bytes
// bound it on paper; measured, instructions do (each element is scaled,
// converted and compared twice, and the activation's slope costs a dozen), so
// the activation is a template argument and maxima are single instructions:
// 16384 x 4096 BF16 in both directions 66 us, 4.1 TB/s.
constexpr int kTileRows = 128, kTileCols = 64, kQThreads = 256;
constexpr int kPass = kTileRows * kTileCols / (kQThreads * 8);

// segment of row r (offsets ascending), and whether r holds a token of it
__device__ __forceinline__ bool row_is_token(const Segments& s, long long r) {
    int lo = 0, hi = s.experts - 1;   // the last e with offsets[e] <= r
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s.offsets[mid] <= r) lo = mid; else hi = mid - 1;
    }
    const long long o = s.offsets[lo];
    return r >= o && r < o + s.counts[lo];
}

template <typename T, int kAct, bool kE5m2>
__global__ void __launch_bounds__(kQThreads, 4) quantize_kernel(Quantize q, int row_tiles) {
    __shared__ float4 tile[kTileRows * (kTileCols / 4)];
    __shared__ uint8_t token[kTileRows];
    const int g = (int)(blockIdx.x / row_tiles), row_tile = (int)blockIdx.x - g * row_tiles;
    const long long r0 = (long long)row_tile * kTileRows;
    const int left = (int)min((long long)kTileRows, q.rows - r0);   // rows of the tile
    const int cols = (int)q.cols, c0 = (int)blockIdx.y * kTileCols, ct = (cols + 127) >> 7;
    const int tx = threadIdx.x % (kTileCols / 8), ty = threadIdx.x / (kTileCols / 8);
    constexpr int emax = mx_emax<kE5m2>();
    const bool masked = q.seg.offsets != nullptr;
    grid_wait();
    grid_launch_next();
    if (masked) {
        if (r0 >= q.seg.offsets[q.seg.experts]) return;   // past the last segment: nothing is read from there
        if (threadIdx.x < kTileRows) token[threadIdx.x] = (int)threadIdx.x < left && row_is_token(q.seg, r0 + threadIdx.x);
        __syncthreads();
    }
    // (addresses once per thread; a pass is 32 rows further)
    const int col = c0 + tx * 8;
    const bool in_cols = col < cols;   // (columns come in blocks of 32)
    const long long row = (long long)g * q.rows + r0 + ty;
    const T* x = static_cast<const T*>(q.x) + row * q.ldx + col;
    const __nv_bfloat16* pre = static_cast<const __nv_bfloat16*>(q.preact) + row * cols + col;
    const long long x_pass = 32 * q.ldx, c_pass = 32ll * cols;
    float2 v[kPass][4];
    typename Vec<T, 8>::Raw raw[kPass];
    uint4 zw[kPass];
    bool live[kPass];
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
        live[p] = in_cols && ty + p * 32 < left && (!masked || token[ty + p * 32]);
        if (live[p]) {
            raw[p] = Vec<T, 8>::raw(x + p * x_pass);
            if (kAct != kActNone) zw[p] = ptx::ld_nc_v4(pre + p * c_pass);
        }
    }
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
        float f[8];
        Vec<T, 8>::values(raw[p], f);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[p][j] = make_float2(f[2 * j], f[2 * j + 1]);
        if constexpr (kAct != kActNone) {
            float z[8];
            Vec<__nv_bfloat16, 8>::unpack(&zw[p], z);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[p][j] = act_back2<kAct>(v[p][j], make_float2(z[2 * j], z[2 * j + 1]));
        }
        // (the vote: no selects on whole tiles; the silu pass without codes 60.2 -> 56.5 us on 16384 x 4096)
        if (__any_sync(kLanes, !live[p]) && !live[p]) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[p][j] = make_float2(0.f, 0.f);
        }
    }
    if (q.codes) {
        uint8_t* codes = q.codes + row * cols + col;
        uint8_t* scale = q.scale + (((size_t)g * ct + (c0 >> 7)) * row_tiles + row_tile) * 512 + ty * 16 + ((c0 >> 5) & 3);
#pragma unroll
        for (int p = 0; p < kPass; ++p) {
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) m = abs_max(m, v[p][j].x, v[p][j].y);
            m = max_nan(m, __shfl_xor_sync(kLanes, m, 1));
            m = max_nan(m, __shfl_xor_sync(kLanes, m, 2));
            const uint32_t byte = mx_scale_byte(__float_as_uint(m), emax);
            const float inv = mx_inv_scale(byte);
            const uint2 w = make_uint2(mx_codes4<kE5m2>(v[p][0], v[p][1], inv), mx_codes4<kE5m2>(v[p][2], v[p][3], inv));
            if (in_cols && ty + p * 32 < left) *reinterpret_cast<uint2*>(codes + p * c_pass) = w;
            // two blocks of the tile's row in one 16-bit store (a tile is half a scale word wide)
            const uint32_t other = __shfl_xor_sync(kLanes, byte, 4);
            if (tx == 0) {   // (rows past the last and blocks past the last column get scale 0: every byte is written)
                uint16_t* s = reinterpret_cast<uint16_t*>(scale + p * 4);
                s[0] = (uint16_t)(byte | (c0 + 32 < cols ? other : 0u) << 8);
                if (c0 + kTileCols >= cols && (c0 & 64) == 0) s[1] = 0;
            }
        }
    }
    if (!q.codes_t && !q.colsum) return;
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
        // (the columns of the upper half of the tile lie in pairs of 4 swapped: no bank conflicts)
        float4* t = tile + (ty + p * 32) * (kTileCols / 4) + tx * 2;
        const int swap = tx >> 2;
        t[swap] = make_float4(v[p][0].x, v[p][0].y, v[p][1].x, v[p][1].y);
        t[swap ^ 1] = make_float4(v[p][2].x, v[p][2].y, v[p][3].x, v[p][3].y);
    }
    __syncthreads();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int c4 = (lane & 7) + 8 * (warp & 1), rg = lane >> 3, rb = warp >> 1;   // 4 columns; 8 of the 32 rows of block rb
    const int c = c0 + c4 * 4;
    const bool in_c = c < cols, in_t = in_c && rb * 32 < left;   // (rows past the last inside a block of 32 are zeros)
    float4 u[8];
    float2 s01 = make_float2(0.f, 0.f), s23 = s01;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        u[i] = tile[(rb * 32 + rg * 8 + i) * (kTileCols / 4) + (c4 ^ (c4 >> 3))];
        s01 = add2(s01, make_float2(u[i].x, u[i].y));
        s23 = add2(s23, make_float2(u[i].z, u[i].w));
    }
    float sum[4] = {s01.x, s01.y, s23.x, s23.y};
    if (q.colsum) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sum[j] += __shfl_xor_sync(kLanes, sum[j], 8);
            sum[j] += __shfl_xor_sync(kLanes, sum[j], 16);
        }
        if (rg == 0 && in_t)
            *reinterpret_cast<float4*>(q.colsum + (long long)(row_tile * 4 + rb) * cols + c) = make_float4(sum[0], sum[1], sum[2], sum[3]);
    }
    if (!q.codes_t) return;
    const long long ld_t = (q.rows + 31) / 32 * 32;
    uint8_t* codes_t = q.codes_t + ((long long)g * cols + c) * ld_t + r0 + rb * 32 + rg * 8;
    // (a thread's 4 columns are neighbours in one 32-row group of their scale tile)
    uint8_t* scale_t = q.scale_t + ((size_t)g * row_tiles + row_tile) * ct * 512;
    uint8_t* word = scale_t + (size_t)(c >> 7) * 512 + (c & 31) * 16 + ((c & 127) >> 5) * 4 + rb;
    float inv[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i += 2) m = abs_max(m, (&u[i].x)[j], (&u[i + 1].x)[j]);
        m = max_nan(m, __shfl_xor_sync(kLanes, m, 8));
        m = max_nan(m, __shfl_xor_sync(kLanes, m, 16));
        const uint32_t byte = mx_scale_byte(__float_as_uint(m), emax);
        inv[j] = mx_inv_scale(byte);
        if (in_c && rg == 0) word[j * 16] = in_t ? (uint8_t)byte : 0;
    }
    // (two columns a multiplication: they are neighbours in registers, the rows are not)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 lo = mul2(make_float2(u[i].x, u[i].y), make_float2(inv[0], inv[1]));
        const float2 hi = mul2(make_float2(u[i].z, u[i].w), make_float2(inv[2], inv[3]));
        u[i] = make_float4(lo.x, lo.y, hi.x, hi.y);
    }
    if (in_t) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = fp8x2<kE5m2>((&u[2 * i].x)[j], (&u[2 * i + 1].x)[j]);
            *reinterpret_cast<uint2*>(codes_t + j * ld_t) = make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
        }
    }
    // the words of the last scale tile past the last column
    if (c0 + kTileCols >= cols)
        for (int i = cols + threadIdx.x; i < ct * 128; i += kQThreads)
            *reinterpret_cast<uint32_t*>(scale_t + (size_t)(i >> 7) * 512 + (i & 31) * 16 + ((i & 127) >> 5) * 4) = 0;
}

// dbias: the 32-row blocks' column sums of a segment, added in order: a CTA
// takes 32 columns of a group, its 8 warps an eighth of the blocks each (bound
// by latency: 16384 x 4096 over 8 groups 7.6 us).
__global__ void __launch_bounds__(256) bias_sums_kernel(const float* colsum, Segments s, long long cols, float* dbias) {
    __shared__ float part[8][32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = blockIdx.y;
    const long long c = (long long)blockIdx.x * 32 + lane;   // (columns come in blocks of 32)
    long long lo = 0, hi = (s.rows + 31) / 32;
    grid_wait();
    grid_launch_next();
    if (s.offsets) {
        lo = max(0, s.offsets[g]) / 32;
        hi = min(hi, (long long)s.offsets[g + 1] / 32);
    }
    const long long per = (max(0ll, hi - lo) + 7) / 8, b1 = min(hi, lo + (warp + 1) * per);
    float sum = 0.f;
#pragma unroll 8
    for (long long b = lo + warp * per; b < b1; ++b) sum += colsum[b * cols + c];
    part[warp][lane] = sum;
    __syncthreads();
    if (warp == 0) {
        sum = 0.f;
        for (int w = 0; w < 8; ++w) sum += part[w][lane];
        dbias[(long long)g * cols + c] = sum;
    }
}

__global__ void scale_tiles_kernel(const uint8_t* s, int groups, long long rows, long long blocks, uint32_t* tiles, int rt, int bt) {
    const long long per = (long long)bt * rt * 128, n = per * groups;
    grid_wait();
    grid_launch_next();
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

template <typename T, int kAct, bool kE5m2>
cudaError_t launch_one(const Quantize& q, dim3 grid, int row_tiles, cudaStream_t stream) {
    return launch(quantize_kernel<T, kAct, kE5m2>, grid, kQThreads, 0, 1, stream, q, row_tiles);
}
template <bool kE5m2>
cudaError_t launch_format(const Quantize& q, dim3 grid, int row_tiles, cudaStream_t stream) {
    if (q.x_type == kTypeF16) return launch_one<__half, kActNone, kE5m2>(q, grid, row_tiles, stream);
    if (q.x_type == kTypeF32) return launch_one<float, kActNone, kE5m2>(q, grid, row_tiles, stream);
    if (!q.preact) return launch_one<__nv_bfloat16, kActNone, kE5m2>(q, grid, row_tiles, stream);
    if (q.act == kActRelu) return launch_one<__nv_bfloat16, kActRelu, kE5m2>(q, grid, row_tiles, stream);
    if (q.act == kActGelu) return launch_one<__nv_bfloat16, kActGelu, kE5m2>(q, grid, row_tiles, stream);
    return launch_one<__nv_bfloat16, kActSilu, kE5m2>(q, grid, row_tiles, stream);
}

}  // namespace

cudaError_t launch_quantize(const Quantize& q, cudaStream_t stream) {
    const int row_tiles = (int)((q.rows + kTileRows - 1) / kTileRows);
    const dim3 grid((unsigned)((long long)row_tiles * q.groups), (unsigned)((q.cols + kTileCols - 1) / kTileCols));
    return q.e5m2 ? launch_format<true>(q, grid, row_tiles, stream) : launch_format<false>(q, grid, row_tiles, stream);
}

cudaError_t launch_bias_sums(const float* colsum, const Segments& seg, long long cols, float* dbias, cudaStream_t stream) {
    const dim3 grid((unsigned)(cols / 32), (unsigned)seg.experts);
    return launch(bias_sums_kernel, grid, 256, 0, 1, stream, colsum, seg, cols, dbias);
}

cudaError_t launch_scale_tiles(const uint8_t* s, int groups, long long rows, long long blocks, uint8_t* tiles, int sms,
                               cudaStream_t stream) {
    const int rt = (int)((rows + 127) / 128), bt = (int)((blocks + 3) / 4);
    const long long words = (long long)groups * rt * bt * 128;
    return launch(scale_tiles_kernel, dim3((unsigned)std::min<long long>((words + 255) / 256, 16ll * sms)), 256, 0, 1, stream, s, groups,
                  rows, blocks, reinterpret_cast<uint32_t*>(tiles), rt, bt);
}

}  // namespace mxa2a
