// Mixture-of-experts row movement: the stable sort of token assignments by
// expert, the rows' copy into that order (as they are, or quantised to MXFP8
// on the way), the weighted way back, and its gradient.
#include <algorithm>

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
// experts in shared memory; prefix sums over warps, then over the cluster's
// CTAs (distributed shared memory), then over experts (rounded up to the
// alignment) give every warp its first place per expert; a second walk over
// the range hands out the places in order, 32 assignments at a time, equal
// ids of a warp ranked by lane.  Bound by latency (ids are read twice from L2).
__device__ __forceinline__ int load_expert(const MoeSort& a, long long i, long long end) {
    if (i >= end) return -1;
    const int e = __ldg(a.expert + i);
    return (unsigned)e < (unsigned)a.experts ? e : -1;
}

__global__ void __launch_bounds__(1024) moe_sort_kernel(MoeSort a, int ctas) {
    extern __shared__ uint32_t sort_smem[];
    const int nw = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int E = a.experts;
    uint32_t* hist = sort_smem;              // [nw][E]: counts, then next places
    uint32_t* total = sort_smem + nw * E;    // [E]: this CTA's counts (read by the whole cluster)
    uint32_t* scan = total + E;              // [32]
    const int cta = (int)blockIdx.x;
    for (int i = threadIdx.x; i < nw * E; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    const long long per = ((a.assignments + (long long)ctas * nw - 1) / ((long long)ctas * nw) + 31) / 32 * 32;
    const long long lo = min(a.assignments, ((long long)cta * nw + warp) * per);
    const long long hi = min(a.assignments, lo + per);
    uint32_t* mine = hist + warp * E;
    for (long long i = lo + lane; i < hi; i += 32) {
        const int e = load_expert(a, i, hi);
        if (e >= 0) atomicAdd(&mine[e], 1u);   // counts only: their order does not matter
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        uint32_t run = 0;
        for (int w = 0; w < nw; ++w) {
            const uint32_t t = hist[w * E + e];
            hist[w * E + e] = run;
            run += t;
        }
        total[e] = run;
    }
    __syncthreads();
    if (ctas > 1) cluster_sync();
    // experts in chunks of blockDim: exclusive scan of the aligned totals
    uint32_t carry = 0;
    for (int e0 = 0; e0 < E; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x;
        uint32_t all = 0, before = 0;
        if (e < E) {
            for (int c = 0; c < ctas; ++c) {
                const uint32_t t = ctas == 1 ? total[e] : ld_shared_cluster_u32(mapa_shared(smem_u32(total + e), c));
                if (c < cta) before += t;
                all += t;
            }
        }
        const uint32_t seg = (all + a.align - 1) / a.align * a.align;
        uint32_t inc = seg;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t v = __shfl_up_sync(kLanes, inc, d);
            if (lane >= d) inc += v;
        }
        if (lane == 31) scan[warp] = inc;
        __syncthreads();
        uint32_t base = carry, block = 0;
        for (int w = 0; w < nw; ++w) {
            if (w < warp) base += scan[w];
            block += scan[w];
        }
        const uint32_t first = base + inc - seg;   // offsets[e]
        if (e < E) {
            for (int w = 0; w < nw; ++w) hist[w * E + e] += first + before;
            if (cta == 0) {
                a.offsets[e] = (int32_t)first;
                a.counts[e] = (int32_t)all;
            }
            // padding of segment e, split over the cluster's CTAs
            if (a.src)
                for (uint32_t r = first + all + cta; r < first + seg; r += ctas)
                    if (r < a.rows) a.src[r] = -1;
        }
        carry += block;
        __syncthreads();
    }
    if (cta == 0 && threadIdx.x == 0) a.offsets[E] = (int32_t)carry;
    if (a.src)
        for (long long r = carry + (long long)cta * blockDim.x + threadIdx.x; r < a.rows; r += (long long)ctas * blockDim.x)
            a.src[r] = -1;
    int e = load_expert(a, lo + lane, hi);
    for (long long i0 = lo; i0 < hi; i0 += 32) {
        const int next = load_expert(a, i0 + 32 + lane, hi);
        const long long i = i0 + lane;
        const uint32_t same = __match_any_sync(kLanes, e);
        const int rank = __popc(same & ((1u << lane) - 1));
        uint32_t place = 0;
        if (e >= 0) place = mine[e] + rank;
        __syncwarp();
        if (e >= 0 && rank == 0) mine[e] += __popc(same);
        __syncwarp();
        if (i < hi) {
            a.pos[i] = e >= 0 ? (int32_t)place : -1;
            if (e >= 0 && a.src && place < a.rows) a.src[place] = (int32_t)i;
        }
        e = next;
    }
    if (ctas > 1) cluster_sync();   // no CTA leaves while another may read its totals
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

// Dispatch: out[pos(t, j)] = x[t] for every expert j of token t.  A warp takes
// one piece of a token's row, reads it once and writes it to all its places
// (quantised once).  Bound by the bytes written (topk per byte read).
constexpr int kDispatchUnroll = 4;   // vectors of a lane in flight

template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads) moe_dispatch_copy_kernel(MoeDispatch a, long long row_ctas, int chunks) {
    if (blockIdx.x >= row_ctas) {
        const int b = (int)(blockIdx.x - row_ctas);
        zero_padding<false>(a.seg, b / kPadParts, b % kPadParts, kPadParts, a.out, (size_t)a.hidden * sizeof(T), nullptr, 0, 0);
        return;
    }
    // here T is an unsigned word of V elements' bytes: a plain copy
    const int lane = threadIdx.x % 32;
    const long long task = (long long)blockIdx.x * (kRowThreads / 32) + threadIdx.x / 32;
    const long long t = task / chunks;
    if (t >= a.tokens) return;
    const long long h0 = (task % chunks) * (32 * kDispatchUnroll) + lane;
    const T* x = static_cast<const T*>(a.x) + t * a.ldx;
    T v[kDispatchUnroll];
#pragma unroll
    for (int u = 0; u < kDispatchUnroll; ++u)
        if (h0 + 32 * u < a.hidden) v[u] = x[h0 + 32 * u];
    for (int j = 0; j < a.topk; ++j) {
        const long long r = __ldg(a.pos + t * a.topk + j);
        if (r < 0 || r >= a.seg.rows) continue;
        T* o = static_cast<T*>(a.out) + r * a.hidden;
#pragma unroll
        for (int u = 0; u < kDispatchUnroll; ++u)
            if (h0 + 32 * u < a.hidden) o[h0 + 32 * u] = v[u];
    }
}

// MX: 8 elements a lane and vector, 4 lanes a scale block, 16 lanes a scale word.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) moe_dispatch_mx_kernel(MoeDispatch a, long long row_ctas, int chunks) {
    const int kbs = (int)((a.hidden + 127) / 128), rt = (int)((a.seg.rows + 127) / 128);
    if (blockIdx.x >= row_ctas) {
        const int b = (int)(blockIdx.x - row_ctas);
        zero_padding<true>(a.seg, b / kPadParts, b % kPadParts, kPadParts, a.out, (size_t)a.hidden, a.out_scale, kbs, rt);
        return;
    }
    const int lane = threadIdx.x % 32;
    const long long task = (long long)blockIdx.x * (kRowThreads / 32) + threadIdx.x / 32;
    const long long t = task / chunks;
    if (t >= a.tokens) return;
    const int h0 = (int)(task % chunks) * (256 * kDispatchUnroll) + lane * 8;
    const T* x = static_cast<const T*>(a.x) + t * a.ldx;
    const bool e5m2 = a.out_type == kTypeE5M2;
    const int emax = mx_emax(e5m2);
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
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[u][i]) & 0x7fffffffu);
        m = max(m, __shfl_xor_sync(kLanes, m, 1));
        m = max(m, __shfl_xor_sync(kLanes, m, 2));
        const uint32_t byte = mx_scale_byte(m, emax);
        const float inv = mx_inv_scale(byte);
        code[u] = make_uint2(mx_codes4(f[u], inv, byte == 255, e5m2), mx_codes4(f[u] + 4, inv, byte == 255, e5m2));
        // the four blocks' bytes of the 16-lane group into one word
        uint32_t w = byte << (8 * ((lane >> 2) & 3));
        w |= __shfl_xor_sync(kLanes, w, 4);
        w |= __shfl_xor_sync(kLanes, w, 8);
        word[u] = w;
    }
    for (int j = 0; j < a.topk; ++j) {
        const long long r = __ldg(a.pos + t * a.topk + j);
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
// fp32, rounded once.  A warp takes one piece of a token's row.  Bound by the
// bytes of y read.
template <typename T, int V, int U>
__global__ void __launch_bounds__(kRowThreads) moe_combine_kernel(MoeCombine a, int chunks) {
    const int lane = threadIdx.x % 32;
    const long long task = (long long)blockIdx.x * (kRowThreads / 32) + threadIdx.x / 32;
    const long long t = task / chunks;
    if (t >= a.tokens) return;
    const long long h0 = (task % chunks) * (32 * V * U) + lane * V;
    float acc[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long h = h0 + 32 * V * u;
        if (a.residual && h < a.hidden) {
            Vec<T, V>::load(static_cast<const T*>(a.residual) + t * a.hidden + h, acc[u]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) acc[u][i] = 0.f;
        }
    }
#pragma unroll 4
    for (int j = 0; j < a.topk; ++j) {
        const long long r = __ldg(a.pos + t * a.topk + j);
        if (r < 0 || r >= a.rows) continue;
        const float w = a.weight ? __ldg(a.weight + t * a.topk + j) : 1.f;
        const T* y = static_cast<const T*>(a.y) + r * a.hidden;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long h = h0 + 32 * V * u;
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
        const long long h = h0 + 32 * V * u;
        if (h < a.hidden) Vec<T, V>::store(static_cast<T*>(a.out) + t * a.hidden + h, acc[u]);
    }
}

// Gradient of the combine: dy[pos(t, j)] = w[t][j] dout[t], dw[t][j] = <dout[t],
// y[pos(t, j)]>.  A CTA takes a token: its warps walk the row in steps, each
// piece of dout read once for a group of kBwdGroup experts; the products' sums
// are joined over lanes and then over warps in order.  Bound by y read and dy
// written.
constexpr int kBwdGroup = 8;

template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads) moe_combine_backward_kernel(MoeCombineBackward a) {
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
        long long row[kBwdGroup];
        float w[kBwdGroup], sum[kBwdGroup];
#pragma unroll
        for (int j = 0; j < kBwdGroup; ++j) {
            row[j] = -1;
            sum[j] = w[j] = 0.f;
            if (j0 + j < a.topk) {
                const long long r = __ldg(a.pos + t * a.topk + j0 + j);
                if (r >= 0 && r < a.seg.rows) {
                    row[j] = r * a.hidden;
                    w[j] = a.weight ? __ldg(a.weight + t * a.topk + j0 + j) : 1.f;
                }
            }
        }
        for (long long h = (long long)threadIdx.x * V; h < a.hidden; h += (long long)blockDim.x * V) {
            float df[V];
            Vec<T, V>::load(d + h, df);
#pragma unroll
            for (int j = 0; j < kBwdGroup; ++j) {
                if (row[j] < 0) continue;
                float f[V];
                Vec<T, V>::load(static_cast<const T*>(a.y) + row[j] + h, f);
#pragma unroll
                for (int i = 0; i < V; ++i) sum[j] = fmaf(df[i], f[i], sum[j]);
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] = w[j] * df[i];
                Vec<T, V>::store(static_cast<T*>(a.dy) + row[j] + h, f);
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

template <typename T>
bool aligned_rows(const void* p, long long ld) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (long long)sizeof(T) % 16 == 0);
}

template <typename W>
cudaError_t copy_words(MoeDispatch a, size_t row_bytes, size_t ld_bytes, cudaStream_t stream) {
    a.hidden = (long long)(row_bytes / sizeof(W));
    a.ldx = (long long)(ld_bytes / sizeof(W));
    const int chunks = (int)((a.hidden + 32 * kDispatchUnroll - 1) / (32 * kDispatchUnroll));
    const long long ctas = (a.tokens * chunks + kRowThreads / 32 - 1) / (kRowThreads / 32);
    moe_dispatch_copy_kernel<W, 1><<<(unsigned)(ctas + a.seg.experts * kPadParts), kRowThreads, 0, stream>>>(a, ctas, chunks);
    return cudaGetLastError();
}

template <typename T>
cudaError_t dispatch_mx(const MoeDispatch& a, cudaStream_t stream) {
    const int chunks = (int)((a.hidden + 256 * kDispatchUnroll - 1) / (256 * kDispatchUnroll));
    const long long ctas = (a.tokens * chunks + kRowThreads / 32 - 1) / (kRowThreads / 32);
    moe_dispatch_mx_kernel<T><<<(unsigned)(ctas + a.seg.experts * kPadParts), kRowThreads, 0, stream>>>(a, ctas, chunks);
    return cudaGetLastError();
}

template <typename T, int V, int U>
cudaError_t combine_v(const MoeCombine& a, cudaStream_t stream) {
    const int chunks = (int)((a.hidden + 32 * V * U - 1) / (32 * V * U));
    const long long ctas = (a.tokens * chunks + kRowThreads / 32 - 1) / (kRowThreads / 32);
    moe_combine_kernel<T, V, U><<<(unsigned)ctas, kRowThreads, 0, stream>>>(a, chunks);
    return cudaGetLastError();
}
template <typename T>
cudaError_t combine_t(const MoeCombine& a, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    if (aligned_rows<T>(a.y, a.hidden) && aligned_rows<T>(a.out, a.hidden) && aligned_rows<T>(a.residual, a.hidden))
        return combine_v<T, V, 2>(a, stream);
    return combine_v<T, 1, 4>(a, stream);
}

template <typename T>
cudaError_t combine_backward_t(const MoeCombineBackward& a, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const unsigned ctas = (unsigned)(a.tokens + (long long)a.seg.experts * kPadParts);
    if (aligned_rows<T>(a.y, a.hidden) && aligned_rows<T>(a.dy, a.hidden) && aligned_rows<T>(a.dout, a.hidden))
        moe_combine_backward_kernel<T, V><<<ctas, kRowThreads, 0, stream>>>(a);
    else
        moe_combine_backward_kernel<T, 1><<<ctas, kRowThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_moe_sort(const MoeSort& a, cudaStream_t stream) {
    const int ctas = a.assignments <= 4096 ? 1 : 8;
    const long long per_cta = (a.assignments + ctas - 1) / ctas;
    const int warps = (int)std::min<long long>(32, std::max<long long>((per_cta + 31) / 32, (std::min(a.experts, 1024) + 31) / 32));
    const int threads = 32 * std::max(1, warps);
    const size_t smem = ((size_t)(threads / 32) * a.experts + a.experts + 32) * sizeof(uint32_t);
    cudaError_t e = cudaFuncSetAttribute(moe_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 140 * 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {(unsigned)ctas, 1, 1};
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe_sort_kernel, a, ctas);
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
