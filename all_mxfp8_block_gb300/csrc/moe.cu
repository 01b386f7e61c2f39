// Mixture-of-experts row movement: the stable sort of token assignments by
// expert, the rows' copy into that order (as they are, or quantised to MXFP8
// on the way), the weighted way back, and its gradient.
#include <algorithm>

#include "launch.cuh"
#include "moe.cuh"
#include "mxquant.cuh"
#include "ptx.cuh"

namespace mxa2a {
using namespace ptx;

namespace {

// ------------------------------------------------------------------ sort
// A stable counting sort of the expert ids.  pos(i) = offsets[e] + #{j < i :
// expert(j) = e}.  One cluster of CTAs does it in one launch with no scratch
// memory: every warp owns a consecutive range of assignments and counts its
// experts in shared memory; prefix sums over warps (a lane per warp), then over
// the cluster's CTAs (each writes its counts to the others' shared memory), then over
// experts (rounded up to the alignment) give every warp its first place per
// expert; a second walk over the range hands out the places in order, 32
// assignments at a time, equal ids of a warp ranked by lane.  Bound by latency
// (the first ids of each lane stay in registers, the others are read twice):
// 16384 ids of 32 experts in 7 us.
__device__ __forceinline__ int load_expert(const MoeSort& a, long long i, long long end) {
    if (i >= end) return -1;
    const int e = a.expert[i];
    return (unsigned)e < (unsigned)a.experts ? e : -1;
}
__device__ __forceinline__ uint32_t scan_up(uint32_t v, int lane) {   // inclusive, over the warp
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t u = __shfl_up_sync(kLanes, v, d);
        if (lane >= d) v += u;
    }
    return v;
}

constexpr int kSortCtas = 8;
constexpr int kSortKeep = 4;   // ids of a lane that stay in registers between the two walks
__device__ __forceinline__ void st_shared_cluster_u32(uint32_t cluster_addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

__global__ void __launch_bounds__(1024, 1) moe_sort_kernel(MoeSort a, int ctas) {
    extern __shared__ uint32_t sort_smem[];
    const int nw = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int E = a.experts, ld = E | 1;     // (odd: a lane per warp reads without bank conflicts)
    uint32_t* hist = sort_smem;              // [nw][ld]: counts, then places before the warp's own
    uint32_t* peer = hist + nw * ld;         // [ctas][E]: the CTAs' counts, written by them
    uint32_t* base = peer + ctas * E;        // [E]: first place of this CTA
    uint32_t* scan = base + E;               // [32]
    const int cta = (int)blockIdx.x;
    if (ctas > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // (waited for before the first write to a peer)
    for (int i = threadIdx.x; i < nw * ld; i += blockDim.x) hist[i] = 0;
    const long long per = ((a.assignments + (long long)ctas * nw - 1) / ((long long)ctas * nw) + 31) / 32 * 32;
    const long long lo = min(a.assignments, ((long long)cta * nw + warp) * per);
    const long long hi = min(a.assignments, lo + per);
    uint32_t* mine = hist + warp * ld;
    grid_wait();
    grid_launch_next();
    int id[kSortKeep];
#pragma unroll
    for (int k = 0; k < kSortKeep; ++k) id[k] = load_expert(a, lo + 32 * k + lane, hi);
    __syncthreads();
    // (counts only: the order of the additions does not matter)
#pragma unroll
    for (int k = 0; k < kSortKeep; ++k)
        if (id[k] >= 0) atomicAdd(&mine[id[k]], 1u);
    for (long long i = lo + 32 * kSortKeep + lane; i < hi; i += 32) {
        const int e = load_expert(a, i, hi);
        if (e >= 0) atomicAdd(&mine[e], 1u);
    }
    __syncthreads();
    if (ctas > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (nw <= 4) {
        // few warps (a decode step): a thread per expert
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            uint32_t run = 0;
            for (int w = 0; w < nw; ++w) {
                const uint32_t n = hist[w * ld + e];
                hist[w * ld + e] = run;
                run += n;
            }
            if (ctas == 1) peer[e] = run;
            else
                for (int c = 0; c < ctas; ++c) st_shared_cluster_u32(mapa_shared(smem_u32(peer + cta * E + e), c), run);
        }
    } else {
        for (int e = warp; e < E; e += nw) {
            const uint32_t n = lane < nw ? hist[lane * ld + e] : 0u, inc = scan_up(n, lane);
            if (lane < nw) hist[lane * ld + e] = inc - n;
            const uint32_t sum = __shfl_sync(kLanes, inc, 31);
            if (lane < ctas) {
                if (ctas == 1) peer[e] = sum;
                else st_shared_cluster_u32(mapa_shared(smem_u32(peer + cta * E + e), lane), sum);
            }
        }
    }
    if (ctas > 1) cluster_sync(); else __syncthreads();
    // exclusive scan of the aligned totals over the experts, blockDim at a time
    uint32_t carry = 0;
    for (int e0 = 0; e0 < E; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x;
        uint32_t n = 0, before = 0;   // the expert's assignments, those of the CTAs before this one
        if (e < E)
            for (int c = 0; c < ctas; ++c) {
                const uint32_t v = peer[c * E + e];
                if (c < cta) before += v;
                n += v;
            }
        const uint32_t seg = (n + a.align - 1) / a.align * a.align;
        const uint32_t inc = scan_up(seg, lane);
        if (lane == 31) scan[warp] = inc;
        __syncthreads();
        const uint32_t w = scan_up(lane < nw ? scan[lane] : 0u, lane);   // (every warp scans the warps' sums)
        const uint32_t warps_before = __shfl_sync(kLanes, w, max(warp - 1, 0));
        const uint32_t first = carry + (warp ? warps_before : 0u) + inc - seg;   // offsets[e]
        if (e < E) {
            base[e] = first + before;
            if (cta == 0) {
                a.offsets[e] = (int32_t)first;
                a.counts[e] = (int32_t)n;
            }
            // padding of segment e, split over the cluster's CTAs
            if (a.src)
                for (uint32_t r = first + n + cta; r < first + seg; r += ctas)
                    if (r < a.rows) a.src[r] = -1;
        }
        carry += __shfl_sync(kLanes, w, 31);
        __syncthreads();
    }
    if (cta == 0 && threadIdx.x == 0) a.offsets[E] = (int32_t)carry;
    auto place = [&](long long i, int e) {   // the next place of each lane's expert, in lane order
        const uint32_t same = __match_any_sync(kLanes, e);
        const int rank = __popc(same & ((1u << lane) - 1));
        uint32_t at = 0;
        if (e >= 0) at = base[e] + mine[e] + rank;
        __syncwarp();
        if (e >= 0 && rank == 0) mine[e] += __popc(same);
        __syncwarp();
        if (i < hi) {
            a.pos[i] = e >= 0 ? (int32_t)at : -1;
            if (e >= 0 && a.src && at < a.rows) a.src[at] = (int32_t)i;
        }
    };
#pragma unroll
    for (int k = 0; k < kSortKeep; ++k)
        if (lo + 32 * k < hi) place(lo + 32 * k + lane, id[k]);
    if (lo + 32 * kSortKeep < hi) {
        int e = load_expert(a, lo + 32 * kSortKeep + lane, hi);
        for (long long i0 = lo + 32 * kSortKeep; i0 < hi; i0 += 32) {
            const int next = load_expert(a, i0 + 32 + lane, hi);
            place(i0 + lane, e);
            e = next;
        }
    }
    if (a.src)
        for (long long r = carry + (long long)cta * blockDim.x + threadIdx.x; r < a.rows; r += (long long)ctas * blockDim.x)
            a.src[r] = -1;
}

// ------------------------------------------------------------------ rows
// Zero the rows between a segment's last token and the next segment (share
// `part` of `parts` of expert e's), and, for MX rows, their scale words.
template <bool kMx>
__device__ void zero_padding(const Segments& s, int e, int part, int parts, void* rows_out, size_t row_bytes,
                             uint8_t* scale, int kbs, int rt) {
    const long long lo = (long long)s.offsets[e] + s.counts[e];
    const long long hi = min((long long)s.offsets[e + 1], s.rows);
    if (lo < 0 || lo >= hi) return;
    uint8_t* p = static_cast<uint8_t*>(rows_out) + (size_t)lo * row_bytes;
    const size_t bytes = (size_t)(hi - lo) * row_bytes;
    // the bulk in 16-byte stores from the first aligned address on
    const size_t head = min(bytes, (size_t)(-(intptr_t)p & 15)), n16 = (bytes - head) / 16;
    const size_t t0 = (size_t)part * blockDim.x + threadIdx.x, step = (size_t)parts * blockDim.x;
    for (size_t i = t0; i < n16; i += step) *reinterpret_cast<uint4*>(p + head + i * 16) = make_uint4(0, 0, 0, 0);
    for (size_t i = t0; i < head; i += step) p[i] = 0;
    for (size_t i = head + n16 * 16 + t0; i < bytes; i += step) p[i] = 0;
    if (kMx)
        for (size_t i = t0; i < (size_t)(hi - lo) * kbs; i += step)
            *reinterpret_cast<uint32_t*>(scale + scale_word((int)(i % kbs), lo + (long long)(i / kbs), rt)) = 0;
}
constexpr int kPadParts = 4;    // CTAs that share one expert's padding
constexpr int kRowThreads = 256;

// The row kernels' warps each take a piece of a token's row; a CTA's warps take
// neighbouring pieces.  Block b of the row part: token b / parts, piece
// (b % parts) * warps + warp.

// Dispatch: out[pos(t, j)] = x[t] for every expert j of token t.  A warp reads
// its piece once and writes it to all its places (quantised once).  Bound by
// the bytes written (topk per byte read): 16001 tokens x 2 x 4096 BF16 in 63 us
// with the sort before it, 6.3 TB/s.
constexpr int kDispatchUnroll = 4;   // vectors of a lane in flight

template <typename T>   // T: an unsigned word as wide as the rows' alignment allows
__global__ void __launch_bounds__(kRowThreads) moe_dispatch_copy_kernel(MoeDispatch a, unsigned row_ctas, int parts) {
    grid_wait();
    grid_launch_next();
    if (blockIdx.x >= row_ctas) {
        const int b = (int)(blockIdx.x - row_ctas);
        zero_padding<false>(a.seg, b / kPadParts, b % kPadParts, kPadParts, a.out, (size_t)a.hidden * sizeof(T), nullptr, 0, 0);
        return;
    }
    const unsigned t = blockIdx.x / parts;
    const int h0 = (int)((blockIdx.x - t * parts) * blockDim.x + threadIdx.x / 32 * 32) * kDispatchUnroll + (int)(threadIdx.x % 32);
    const T* x = static_cast<const T*>(a.x) + t * a.ldx;
    T v[kDispatchUnroll];
#pragma unroll
    for (int u = 0; u < kDispatchUnroll; ++u)
        if (h0 + 32 * u < a.hidden) v[u] = x[h0 + 32 * u];
    for (int j = 0; j < a.topk; ++j) {
        const long long r = a.pos[(long long)t * a.topk + j];
        if (r < 0 || r >= a.seg.rows) continue;
        T* o = static_cast<T*>(a.out) + r * a.hidden;
#pragma unroll
        for (int u = 0; u < kDispatchUnroll; ++u)
            if (h0 + 32 * u < a.hidden) o[h0 + 32 * u] = v[u];
    }
}

// MX: 8 elements a lane and vector, 4 lanes a scale block, 16 lanes a scale word.
template <typename T, bool kE5m2>
__global__ void __launch_bounds__(kRowThreads) moe_dispatch_mx_kernel(MoeDispatch a, unsigned row_ctas, int parts) {
    const int kbs = (int)((a.hidden + 127) / 128), rt = (int)((a.seg.rows + 127) / 128);
    grid_wait();
    grid_launch_next();
    if (blockIdx.x >= row_ctas) {
        const int b = (int)(blockIdx.x - row_ctas);
        zero_padding<true>(a.seg, b / kPadParts, b % kPadParts, kPadParts, a.out, (size_t)a.hidden, a.out_scale, kbs, rt);
        return;
    }
    const unsigned t = blockIdx.x / parts;
    const int lane = threadIdx.x % 32;
    const int h0 = (int)((blockIdx.x - t * parts) * blockDim.x + threadIdx.x / 32 * 32) * 8 * kDispatchUnroll + lane * 8;
    const T* x = static_cast<const T*>(a.x) + t * a.ldx;
    constexpr int emax = mx_emax<kE5m2>();
    float f[kDispatchUnroll][8];
#pragma unroll
    for (int u = 0; u < kDispatchUnroll; ++u) {
        if (h0 + 256 * u < a.hidden) {
            Vec<T, 8>::load(x + h0 + 256 * u, f[u]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[u][i] = 0.f;
        }
    }
    uint2 code[kDispatchUnroll];
    uint32_t word[kDispatchUnroll];
#pragma unroll
    for (int u = 0; u < kDispatchUnroll; ++u) {
        const float* x8 = f[u];
        float m = abs_max(abs_max(0.f, x8[0], x8[1]), x8[2], x8[3]);
        m = abs_max(abs_max(m, x8[4], x8[5]), x8[6], x8[7]);
        m = max_nan(m, __shfl_xor_sync(kLanes, m, 1));
        m = max_nan(m, __shfl_xor_sync(kLanes, m, 2));
        const uint32_t byte = mx_scale_byte(__float_as_uint(m), emax);
        const float inv = mx_inv_scale(byte);
        code[u] = make_uint2(mx_codes4<kE5m2>(make_float2(x8[0], x8[1]), make_float2(x8[2], x8[3]), inv),
                             mx_codes4<kE5m2>(make_float2(x8[4], x8[5]), make_float2(x8[6], x8[7]), inv));
        // the four blocks' bytes of the 16-lane group into one word
        uint32_t w = byte << (8 * ((lane >> 2) & 3));
        w |= __shfl_xor_sync(kLanes, w, 4);
        w |= __shfl_xor_sync(kLanes, w, 8);
        word[u] = w;
    }
    for (int j = 0; j < a.topk; ++j) {
        const long long r = a.pos[(long long)t * a.topk + j];
        if (r < 0 || r >= a.seg.rows) continue;
        uint8_t* o = static_cast<uint8_t*>(a.out) + r * a.hidden;
#pragma unroll
        for (int u = 0; u < kDispatchUnroll; ++u) {
            const int h = h0 + 256 * u;
            if (h < a.hidden) {
                *reinterpret_cast<uint2*>(o + h) = code[u];
                if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(a.out_scale + scale_word(h >> 7, r, rt)) = word[u];
            }
        }
    }
}

// Combine: out[t] = residual[t] + sum_j w[t][j] y[pos(t, j)], j in order, in
// fp32, rounded once.  Bound by the bytes of y read.  Two shapes of the same
// sum: with many tokens a warp takes 2 x 32 vectors of a row and one expert at
// a time (48 registers, the SM's warps keep enough loads in flight: 8192 tokens
// x 4 x 7168 105 us, against 153 us for the other); with few a warp takes 32
// vectors and has the loads of 8 experts in flight at once (8 tokens x 8 x 4096:
// 4.1 us against 7.5 us).
constexpr int kCombineGroup = 8;

template <typename T, int V, int U>
__global__ void __launch_bounds__(kRowThreads) moe_combine_kernel(MoeCombine a, int parts) {
    const unsigned t = blockIdx.x / parts;
    const int h0 = (int)((blockIdx.x - t * parts) * blockDim.x + threadIdx.x / 32 * 32) * U * V + (int)(threadIdx.x % 32) * V;
    grid_wait();
    grid_launch_next();
    float acc[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + 32 * V * u;
        if (a.residual && h < a.hidden) {
            Vec<T, V>::load(static_cast<const T*>(a.residual) + t * a.hidden + h, acc[u]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) acc[u][i] = 0.f;
        }
    }
    const int32_t* pos = a.pos + (long long)t * a.topk;
    const float* weight = a.weight + (long long)t * a.topk;
#pragma unroll 4
    for (int j = 0; j < a.topk; ++j) {
        const int r = pos[j];
        if (r < 0 || r >= a.rows) continue;
        const float w = a.weight ? weight[j] : 1.f;
        const T* y = static_cast<const T*>(a.y) + r * a.hidden;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + 32 * V * u;
            if (h < a.hidden) {
                float f[V];
                Vec<T, V>::load(y + h, f);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[u][i] = fmaf(w, f[i], acc[u][i]);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + 32 * V * u;
        if (h < a.hidden) Vec<T, V>::store(static_cast<T*>(a.out) + t * a.hidden + h, acc[u]);
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads) moe_combine_few_kernel(MoeCombine a, int parts) {
    const unsigned t = blockIdx.x / parts;
    const int h = (int)((blockIdx.x - t * parts) * blockDim.x + threadIdx.x) * V;
    grid_wait();
    grid_launch_next();
    if (h >= a.hidden) return;
    float acc[V];
    if (a.residual) {
        Vec<T, V>::load(static_cast<const T*>(a.residual) + t * a.hidden + h, acc);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
    }
    const int32_t* pos = a.pos + (long long)t * a.topk;
    const float* weight = a.weight + (long long)t * a.topk;
    for (int j0 = 0; j0 < a.topk; j0 += kCombineGroup) {
        typename Vec<T, V>::Raw piece[kCombineGroup];
        int row[kCombineGroup];
#pragma unroll
        for (int j = 0; j < kCombineGroup; ++j) {
            row[j] = j0 + j < a.topk ? pos[j0 + j] : -1;
            if (row[j] >= a.rows) row[j] = -1;
        }
#pragma unroll
        for (int j = 0; j < kCombineGroup; ++j)
            if (row[j] >= 0) piece[j] = Vec<T, V>::raw(static_cast<const T*>(a.y) + row[j] * a.hidden + h);
#pragma unroll
        for (int j = 0; j < kCombineGroup; ++j) {
            if (row[j] >= 0) {
                const float w = a.weight ? weight[j0 + j] : 1.f;
                float f[V];
                Vec<T, V>::values(piece[j], f);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = fmaf(w, f[i], acc[i]);
            }
        }
    }
    Vec<T, V>::store(static_cast<T*>(a.out) + t * a.hidden + h, acc);
}

// Gradient of the combine: dy[pos(t, j)] = w[t][j] dout[t], dw[t][j] = <dout[t],
// y[pos(t, j)]>.  A CTA takes a token: its warps walk the row in steps, each
// piece of dout read once for a group of 4 experts, whose loads are in flight
// together (56 registers: 32 warps to an SM; groups of 8 took 80 to 128 and
// measured 94 -> 121 us on 8192 tokens x 4 x 4096, the same on 509 x 8 x 2048);
// the products' sums are joined over lanes and then over warps in order.  Bound
// by y read and dy written: 8192 x 4 x 4096 in 94 us, 6.4 TB/s.
constexpr int kBwdGroup = 4;

template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads, 4) moe_combine_backward_kernel(MoeCombineBackward a) {
    grid_wait();
    grid_launch_next();
    if (blockIdx.x >= a.tokens) {
        const int b = (int)(blockIdx.x - a.tokens);
        zero_padding<false>(a.seg, b / kPadParts, b % kPadParts, kPadParts, a.dy, (size_t)a.hidden * sizeof(T), nullptr, 0, 0);
        return;
    }
    __shared__ float part[kRowThreads / 32][kBwdGroup];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, nw = blockDim.x / 32;
    const long long t = blockIdx.x;
    const T* d = static_cast<const T*>(a.dout) + t * a.hidden;
    for (int j0 = 0; j0 < a.topk; j0 += kBwdGroup) {
        int row[kBwdGroup];
        float w[kBwdGroup], sum[kBwdGroup];
#pragma unroll
        for (int j = 0; j < kBwdGroup; ++j) {
            row[j] = -1;
            sum[j] = w[j] = 0.f;
            if (j0 + j < a.topk) {
                const int r = a.pos[t * a.topk + j0 + j];
                if (r >= 0 && r < a.seg.rows) {
                    row[j] = r;
                    w[j] = a.weight ? a.weight[t * a.topk + j0 + j] : 1.f;
                }
            }
        }
        for (long long h = (long long)threadIdx.x * V; h < a.hidden; h += (long long)blockDim.x * V) {
            typename Vec<T, V>::Raw piece[kBwdGroup];
            const typename Vec<T, V>::Raw dpiece = Vec<T, V>::raw(d + h);
#pragma unroll
            for (int j = 0; j < kBwdGroup; ++j)
                if (row[j] >= 0) piece[j] = Vec<T, V>::raw(static_cast<const T*>(a.y) + row[j] * a.hidden + h);
            float df[V];
            Vec<T, V>::values(dpiece, df);
#pragma unroll
            for (int j = 0; j < kBwdGroup; ++j) {
                if (row[j] < 0) continue;
                float f[V];
                Vec<T, V>::values(piece[j], f);
#pragma unroll
                for (int i = 0; i < V; ++i) sum[j] = fmaf(df[i], f[i], sum[j]);
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] = w[j] * df[i];
                Vec<T, V>::store(static_cast<T*>(a.dy) + row[j] * a.hidden + h, f);
            }
        }
#pragma unroll
        for (int j = 0; j < kBwdGroup; ++j) {
#pragma unroll
            for (int s = 16; s; s >>= 1) sum[j] += __shfl_xor_sync(kLanes, sum[j], s);
            if (lane == 0) part[warp][j] = sum[j];
        }
        __syncthreads();
        if (threadIdx.x < kBwdGroup && j0 + (int)threadIdx.x < a.topk) {
            float s = 0.f;
            for (int w2 = 0; w2 < nw; ++w2) s += part[w2][threadIdx.x];
            a.dweight[t * a.topk + j0 + threadIdx.x] = s;
        }
        __syncthreads();
    }
}

// CTAs of a row kernel whose warps take `piece` elements each: as many warps as
// a row has pieces, at most 8
struct RowShape {
    unsigned threads, parts;
};
RowShape row_shape(long long hidden, int piece) {
    const long long pieces = (hidden + piece - 1) / piece, warps = std::min<long long>(pieces, kRowThreads / 32);
    return {(unsigned)warps * 32, (unsigned)((pieces + warps - 1) / warps)};
}

template <typename T>
bool aligned_rows(const void* p, long long ld) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (long long)sizeof(T) % 16 == 0);
}

template <typename W>
cudaError_t copy_words(MoeDispatch a, size_t row_bytes, size_t ld_bytes, cudaStream_t stream) {
    a.hidden = (long long)(row_bytes / sizeof(W));
    a.ldx = (long long)(ld_bytes / sizeof(W));
    const RowShape r = row_shape(a.hidden, 32 * kDispatchUnroll);
    const unsigned ctas = (unsigned)(a.tokens * r.parts);
    return launch(moe_dispatch_copy_kernel<W>, dim3(ctas + (unsigned)a.seg.experts * kPadParts), r.threads, 0, 1, stream, a, ctas,
                  (int)r.parts);
}

template <typename T>
cudaError_t dispatch_mx(const MoeDispatch& a, cudaStream_t stream) {
    const RowShape r = row_shape(a.hidden, 256 * kDispatchUnroll);
    const unsigned ctas = (unsigned)(a.tokens * r.parts);
    return launch(a.out_type == kTypeE5M2 ? moe_dispatch_mx_kernel<T, true> : moe_dispatch_mx_kernel<T, false>,
                  dim3(ctas + (unsigned)a.seg.experts * kPadParts), r.threads, 0, 1, stream, a, ctas, (int)r.parts);
}

template <typename T, int V>
cudaError_t combine_v(const MoeCombine& a, cudaStream_t stream) {
    constexpr int U = V == 1 ? 4 : 2;
    if (a.tokens * a.hidden <= 32ll * V * 16 * a.sms) {   // at most 16 warps to an SM in the few-token shape
        const RowShape r = row_shape(a.hidden, 32 * V);
        return launch(moe_combine_few_kernel<T, V>, dim3((unsigned)(a.tokens * r.parts)), r.threads, 0, 1, stream, a, (int)r.parts);
    }
    const RowShape r = row_shape(a.hidden, 32 * V * U);
    return launch(moe_combine_kernel<T, V, U>, dim3((unsigned)(a.tokens * r.parts)), r.threads, 0, 1, stream, a, (int)r.parts);
}
template <typename T>
cudaError_t combine_t(const MoeCombine& a, cudaStream_t stream) {
    if (aligned_rows<T>(a.y, a.hidden) && aligned_rows<T>(a.out, a.hidden) && aligned_rows<T>(a.residual, a.hidden))
        return combine_v<T, 16 / sizeof(T)>(a, stream);
    return combine_v<T, 1>(a, stream);
}

template <typename T, int V>
cudaError_t combine_backward_v(const MoeCombineBackward& a, cudaStream_t stream) {
    const dim3 ctas((unsigned)(a.tokens + (long long)a.seg.experts * kPadParts));
    // as many warps to a token as its row has pieces, at most 8 (more CTAs to an SM for narrow rows)
    return launch(moe_combine_backward_kernel<T, V>, ctas, row_shape(a.hidden, 32 * V).threads, 0, 1, stream, a);
}
template <typename T>
cudaError_t combine_backward_t(const MoeCombineBackward& a, cudaStream_t stream) {
    if (aligned_rows<T>(a.y, a.hidden) && aligned_rows<T>(a.dy, a.hidden) && aligned_rows<T>(a.dout, a.hidden))
        return combine_backward_v<T, 16 / sizeof(T)>(a, stream);
    return combine_backward_v<T, 1>(a, stream);
}

}  // namespace

cudaError_t launch_moe_sort(const MoeSort& a, cudaStream_t stream) {
    // one CTA while its 32 warps have at most four rounds of 32 ids each
    const int ctas = a.assignments <= 4096 ? 1 : kSortCtas;
    const long long per_cta = (a.assignments + ctas - 1) / ctas;
    const int warps = (int)std::min<long long>(32, std::max<long long>((per_cta + 31) / 32, (a.experts + 31) / 32));
    const size_t smem = ((size_t)warps * (a.experts | 1) + (size_t)(ctas + 1) * a.experts + 32) * sizeof(uint32_t);
    static unsigned long long allowed = 0;
    if (cudaError_t e = allow_smem(moe_sort_kernel, 176 * 1024, allowed)) return e;
    return launch(moe_sort_kernel, dim3(ctas), 32 * (unsigned)warps, smem, ctas, stream, a, ctas);
}

cudaError_t launch_moe_dispatch(const MoeDispatch& a, cudaStream_t stream) {
    if (a.out_type == kTypeE4M3 || a.out_type == kTypeE5M2) {
        if (a.x_type == kTypeBf16) return dispatch_mx<__nv_bfloat16>(a, stream);
        if (a.x_type == kTypeF16) return dispatch_mx<__half>(a, stream);
        return dispatch_mx<float>(a, stream);
    }
    const size_t es = a.x_type == kTypeF32 ? 4 : 2;
    const size_t row = (size_t)a.hidden * es, ld = (size_t)a.ldx * es;
    // the widest word that every row starts on
    const size_t any = row | ld | reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out);
    if (any % 16 == 0) return copy_words<uint4>(a, row, ld, stream);
    if (any % 4 == 0) return copy_words<uint32_t>(a, row, ld, stream);
    return copy_words<uint16_t>(a, row, ld, stream);
}

cudaError_t launch_moe_combine(const MoeCombine& a, cudaStream_t stream) {
    if (a.type == kTypeBf16) return combine_t<__nv_bfloat16>(a, stream);
    if (a.type == kTypeF16) return combine_t<__half>(a, stream);
    return combine_t<float>(a, stream);
}

cudaError_t launch_moe_combine_backward(const MoeCombineBackward& a, cudaStream_t stream) {
    if (a.type == kTypeBf16) return combine_backward_t<__nv_bfloat16>(a, stream);
    if (a.type == kTypeF16) return combine_backward_t<__half>(a, stream);
    return combine_backward_t<float>(a, stream);
}

}  // namespace mxa2a
