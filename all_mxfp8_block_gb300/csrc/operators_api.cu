// C ABI of the mixture-of-experts row operators, the MX quantiser and the
// linear layer: argument checks, launch shapes, the layer's plan.  Host code
// only; the kernels are in moe.cu, quantize.cu and linear.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <new>

#include "../../include/mxa2a.h"
#include "kernels.cuh"
#include "linear.cuh"
#include "moe.cuh"
#include "mxquant.cuh"
#include "host.cuh"

using namespace mxa2a;

static_assert(MXA2A_TYPE_BF16 == kTypeBf16 && MXA2A_TYPE_F16 == kTypeF16 && MXA2A_TYPE_F32 == kTypeF32 &&
                  MXA2A_TYPE_E4M3 == kTypeE4M3 && MXA2A_TYPE_E5M2 == kTypeE5M2,
              "element types");
static_assert(MXA2A_ACT_NONE == kActNone && MXA2A_ACT_RELU == kActRelu && MXA2A_ACT_GELU == kActGelu &&
                  MXA2A_ACT_SILU == kActSilu,
              "activations");

namespace {

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool plain_type(int t) { return t == MXA2A_TYPE_BF16 || t == MXA2A_TYPE_F16 || t == MXA2A_TYPE_F32; }
bool mx_type(int t) { return t == MXA2A_TYPE_E4M3 || t == MXA2A_TYPE_E5M2; }
size_t type_bytes(int t) { return t == MXA2A_TYPE_F32 ? 4 : mx_type(t) ? 1 : 2; }
int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
int cuda_code(cudaError_t e) { return e == cudaSuccess ? MXA2A_OK : MXA2A_ERR_CUDA; }

// SM count of the current device, 0 if it is no compute capability 10.3 (looked up once per device)
int device_sms(int* dev_out = nullptr) {
    static int known[64];   // 0: not looked up; else SM count + 1 (1: unsupported)
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (dev_out) *dev_out = dev;
    int v = __atomic_load_n(&known[dev], __ATOMIC_RELAXED);
    if (!v) {
        int major = 0, minor = 0, sms = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return 0;
        v = (major == 10 && minor == 3 ? sms : 0) + 1;
        __atomic_store_n(&known[dev], v, __ATOMIC_RELAXED);
    }
    return v - 1;
}
int need_device() { return device_sms() ? MXA2A_OK : MXA2A_ERR_UNSUPPORTED_DEVICE; }

constexpr int64_t kMaxAssignments = int64_t(1) << 26;
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxHidden = int64_t(1) << 20;

// the size rules shared by the row operators
bool moe_shape(int64_t tokens, int topk, int experts, int64_t hidden, int64_t rows) {
    return tokens >= 0 && topk >= 1 && topk <= 64 && experts >= 1 && experts <= 1024 && tokens <= kMaxAssignments / topk &&
           hidden >= 1 && hidden <= kMaxHidden && rows >= 0 && rows <= kMaxRows &&
           // (a launch's blocks, at most one per 256 elements of a row, are counted in 32 bits)
           tokens * ((hidden + 255) / 256) <= kMaxRows - 8192;
}

}  // namespace

extern "C" {

int64_t mxa2a_moe_rows(int64_t tokens, int topk, int experts, int align) {
    if (align < 1 || align > 1024 || !moe_shape(tokens, topk, experts, 1, 0)) return -1;
    const int64_t a = tokens * topk;
    return up(a + std::min<int64_t>(experts, a) * (align - 1), align);
}

int mxa2a_moe_sort(int64_t tokens, int topk, int experts, int align, int64_t rows, const void* expert, void* offsets,
                   void* counts, void* pos, void* src, void* stream) {
    const int64_t need = mxa2a_moe_rows(tokens, topk, experts, align);
    if (need < 0 || rows < need || rows > kMaxRows) return MXA2A_ERR_INVALID_SHAPE;
    if (!offsets || !counts || (tokens && (!expert || !pos))) return MXA2A_ERR_NULL_PTR;
    if (!aligned(expert, 4) || !aligned(offsets, 4) || !aligned(counts, 4) || !aligned(pos, 4) || !aligned(src, 4))
        return MXA2A_ERR_MISALIGNED;
    if (int rc = need_device()) return rc;
    MoeSort a = {tokens * topk, rows, experts, align, static_cast<const int32_t*>(expert), static_cast<int32_t*>(offsets),
                 static_cast<int32_t*>(counts), static_cast<int32_t*>(pos), static_cast<int32_t*>(src)};
    return cuda_code(launch_moe_sort(a, static_cast<cudaStream_t>(stream)));
}

int mxa2a_moe_dispatch(int64_t tokens, int topk, int experts, int64_t hidden, int64_t rows, const void* x, int x_type,
                       int64_t ldx, const void* pos, const void* offsets, const void* counts, void* out, int out_type,
                       void* out_scale, void* stream) {
    if (!plain_type(x_type) || !(mx_type(out_type) || out_type == x_type)) return MXA2A_ERR_INVALID_OPTION;
    const bool mx = mx_type(out_type);
    if (!moe_shape(tokens, topk, experts, hidden, rows) || ldx < hidden || ldx > kMaxRows || (mx && hidden % 32))
        return MXA2A_ERR_INVALID_SHAPE;
    if (!offsets || !counts || (tokens && (!x || !pos)) || (rows && (!out || (mx && !out_scale)))) return MXA2A_ERR_NULL_PTR;
    const size_t es = type_bytes(x_type);
    if (!aligned(pos, 4) || !aligned(offsets, 4) || !aligned(counts, 4) || !aligned(x, es) || !aligned(out, mx ? 16 : es) ||
        (mx && (!aligned(x, 16) || ldx * es % 16 || !aligned(out_scale, 4))))
        return MXA2A_ERR_MISALIGNED;
    if (int rc = need_device()) return rc;
    if (!rows) return MXA2A_OK;
    MoeDispatch a = {};
    a.tokens = tokens;
    a.hidden = hidden;
    a.ldx = ldx;
    a.topk = topk;
    a.x = x;
    a.pos = static_cast<const int32_t*>(pos);
    a.seg = {static_cast<const int32_t*>(offsets), static_cast<const int32_t*>(counts), experts, rows};
    a.out = out;
    a.out_scale = static_cast<uint8_t*>(out_scale);
    a.x_type = x_type;
    a.out_type = out_type;
    return cuda_code(launch_moe_dispatch(a, static_cast<cudaStream_t>(stream)));
}

int mxa2a_moe_combine(int64_t tokens, int topk, int64_t hidden, int64_t rows, const void* y, int type, const void* pos,
                      const void* weight, const void* residual, void* out, void* stream) {
    if (!plain_type(type)) return MXA2A_ERR_INVALID_OPTION;
    if (!moe_shape(tokens, topk, 1, hidden, rows)) return MXA2A_ERR_INVALID_SHAPE;
    if (tokens && (!pos || !out || (rows && !y))) return MXA2A_ERR_NULL_PTR;
    const size_t es = type_bytes(type);
    if (!aligned(y, es) || !aligned(out, es) || !aligned(residual, es) || !aligned(pos, 4) || !aligned(weight, 4))
        return MXA2A_ERR_MISALIGNED;
    if (int rc = need_device()) return rc;
    if (!tokens) return MXA2A_OK;
    MoeCombine a = {tokens, hidden, rows, topk, y, static_cast<const int32_t*>(pos), static_cast<const float*>(weight),
                    residual, out, type, device_sms()};
    return cuda_code(launch_moe_combine(a, static_cast<cudaStream_t>(stream)));
}

int mxa2a_moe_combine_backward(int64_t tokens, int topk, int experts, int64_t hidden, int64_t rows, const void* dout,
                               int type, const void* y, const void* pos, const void* offsets, const void* counts,
                               const void* weight, void* dy, void* dweight, void* stream) {
    if (!plain_type(type)) return MXA2A_ERR_INVALID_OPTION;
    if (!moe_shape(tokens, topk, experts, hidden, rows)) return MXA2A_ERR_INVALID_SHAPE;
    if (!offsets || !counts || (tokens && (!dout || !pos || !dweight)) || (rows && (!y || !dy))) return MXA2A_ERR_NULL_PTR;
    const size_t es = type_bytes(type);
    if (!aligned(dout, es) || !aligned(y, es) || !aligned(dy, es) || !aligned(pos, 4) || !aligned(offsets, 4) ||
        !aligned(counts, 4) || !aligned(weight, 4) || !aligned(dweight, 4))
        return MXA2A_ERR_MISALIGNED;
    if (int rc = need_device()) return rc;
    MoeCombineBackward a = {};
    a.tokens = tokens;
    a.hidden = hidden;
    a.topk = topk;
    a.dout = dout;
    a.y = y;
    a.pos = static_cast<const int32_t*>(pos);
    a.weight = static_cast<const float*>(weight);
    a.seg = {static_cast<const int32_t*>(offsets), static_cast<const int32_t*>(counts), experts, rows};
    a.dy = dy;
    a.dweight = static_cast<float*>(dweight);
    a.type = type;
    return cuda_code(launch_moe_combine_backward(a, static_cast<cudaStream_t>(stream)));
}

int64_t mxa2a_scale_tiles_bytes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0 || rows > kMaxRows || cols > kMaxRows) return -1;
    return (rows + 127) / 128 * ((cols + 127) / 128) * 512;
}

int mxa2a_scale_tiles(const void* scale, int groups, int64_t rows, int64_t cols, void* tiles, void* stream) {
    if (groups < 0 || rows < 0 || cols < 0 || cols % 32 || rows > kMaxRows || cols > kMaxHidden || (int64_t)groups * rows > kMaxRows)
        return MXA2A_ERR_INVALID_SHAPE;
    const bool any = groups && rows && cols;
    if (any && (!scale || !tiles)) return MXA2A_ERR_NULL_PTR;
    if (!aligned(tiles, 4)) return MXA2A_ERR_MISALIGNED;
    if (int rc = need_device()) return rc;
    if (!any) return MXA2A_OK;
    return cuda_code(launch_scale_tiles(static_cast<const uint8_t*>(scale), groups, rows, cols / 32, static_cast<uint8_t*>(tiles),
                                        device_sms(), static_cast<cudaStream_t>(stream)));
}

int mxa2a_quantize(const void* x, int x_type, int64_t ldx, int groups, int64_t rows, int64_t cols, int format, void* codes,
                   void* scale, void* codes_t, void* scale_t, void* stream) {
    if (!plain_type(x_type) || !mx_type(format)) return MXA2A_ERR_INVALID_OPTION;
    // (columns in tiles of 64 are the launch's second dimension, row tiles of all groups its first)
    if (groups < 0 || rows < 0 || cols < 0 || cols % 32 || cols > kMaxHidden || ldx < cols || ldx > kMaxRows ||
        rows > kMaxRows || (int64_t)groups * (rows + 127) > kMaxRows)
        return MXA2A_ERR_INVALID_SHAPE;
    const bool any = groups && rows && cols;
    if (any && (!x || !codes != !scale || !codes_t != !scale_t || (!codes && !codes_t))) return MXA2A_ERR_NULL_PTR;
    if (!aligned(x, 16) || ldx * type_bytes(x_type) % 16 || !aligned(codes, 16) || !aligned(codes_t, 16) || !aligned(scale, 4) ||
        !aligned(scale_t, 4))
        return MXA2A_ERR_MISALIGNED;
    if (int rc = need_device()) return rc;
    if (!any) return MXA2A_OK;
    Quantize q = {};
    q.x = x;
    q.x_type = x_type;
    q.ldx = ldx;
    q.groups = groups;
    q.rows = rows;
    q.cols = cols;
    q.e5m2 = format == MXA2A_TYPE_E5M2;
    q.codes = static_cast<uint8_t*>(codes);
    q.scale = static_cast<uint8_t*>(scale);
    q.codes_t = static_cast<uint8_t*>(codes_t);
    q.scale_t = static_cast<uint8_t*>(scale_t);
    return cuda_code(launch_quantize(q, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ linear layer

struct mxa2a_linear {
    int groups;
    int64_t max_rows, N, K;
    int training;
    int device = 0, sms = 0;
    int64_t timeout_ns = 2000000000LL;
    int elem_types = 0;
    int launches = 0;
    unsigned long long launch_id = 0;
    // workspace: status | (training) dz codes, their scale tiles, the transpose's, the bias sums' blocks
    uint8_t* ws = nullptr;
    size_t ws_bytes = 0;
    DevStatus* status = nullptr;
    uint8_t *dz = nullptr, *dz_scale = nullptr, *dz_t = nullptr, *dz_t_scale = nullptr;
    float* colsum = nullptr;
};

int mxa2a_linear_validate(int groups, int64_t max_rows, int64_t N, int64_t K) {
    const int64_t lim = int64_t(1) << 20;
    if (groups < 1 || groups > 1024 || max_rows < 1 || max_rows > (int64_t(1) << 22) || N < 32 || K < 32 || N % 32 || K % 32 ||
        N > lim || K > lim || (int64_t)groups * N > kMaxRows || (int64_t)groups * K > kMaxRows)
        return MXA2A_ERR_INVALID_SHAPE;
    // tiles of any launch are counted in 32 bits
    const int64_t nt = (N + 127) / 128, kt = (K + 127) / 128, rt = max_rows / 32 + groups + 1;
    if (rt * std::max(nt, kt) > kMaxRows || (int64_t)groups * nt * kt * 4 > kMaxRows) return MXA2A_ERR_INVALID_SHAPE;
    return MXA2A_OK;
}

mxa2a_linear* mxa2a_linear_create(int groups, int64_t max_rows, int64_t N, int64_t K, int training) {
    if (int rc = mxa2a_linear_validate(groups, max_rows, N, K)) {
        set_last_error(rc);
        return nullptr;
    }
    int dev = 0;
    const int sms = device_sms(&dev);
    if (!sms) {
        set_last_error(MXA2A_ERR_UNSUPPORTED_DEVICE);
        return nullptr;
    }
    mxa2a_linear* l = new (std::nothrow) mxa2a_linear();
    if (!l) {
        set_last_error(MXA2A_ERR_CUDA);
        return nullptr;
    }
    l->groups = groups;
    l->max_rows = max_rows;
    l->N = N;
    l->K = K;
    l->training = training != 0;
    l->device = dev;
    l->sms = sms;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 1023) / 1024 * 1024;
        return at;
    };
    const size_t o_status = take(sizeof(DevStatus));
    const size_t rows32 = (size_t)up(max_rows, 32), tiles = (size_t)mxa2a_scale_tiles_bytes(max_rows, N);
    const size_t o_dz = take(training ? (size_t)max_rows * N : 0), o_dzs = take(training ? tiles : 0);
    const size_t o_dzt = take(training ? rows32 * N : 0), o_dzts = take(training ? tiles : 0);
    const size_t o_sum = take(training ? rows32 / 32 * N * sizeof(float) : 0);
    l->ws_bytes = off;
    if (cudaMalloc(&l->ws, l->ws_bytes) != cudaSuccess || cudaMemset(l->ws + o_status, 0, sizeof(DevStatus)) != cudaSuccess ||
        cudaDeviceSynchronize() != cudaSuccess) {
        cudaGetLastError();
        if (l->ws) cudaFree(l->ws);
        delete l;
        set_last_error(MXA2A_ERR_CUDA);
        return nullptr;
    }
    l->status = reinterpret_cast<DevStatus*>(l->ws + o_status);
    if (training) {
        l->dz = l->ws + o_dz;
        l->dz_scale = l->ws + o_dzs;
        l->dz_t = l->ws + o_dzt;
        l->dz_t_scale = l->ws + o_dzts;
        l->colsum = reinterpret_cast<float*>(l->ws + o_sum);
    }
    set_last_error(MXA2A_OK);
    return l;
}

}  // extern "C"

namespace {

int layer_device(const mxa2a_linear* l) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return MXA2A_ERR_CUDA;
    return dev == l->device ? MXA2A_OK : MXA2A_ERR_WRONG_DEVICE;
}

// Tile width, contraction split and grid of one product.
// rows: Q rows that a tile should hold; tiles(tq): tiles of the launch, at most.
// * The tile is the narrowest that holds a group's rows: columns past a group's
//   last row are multiplied for nothing, and a wider tile re-reads the P rows
//   less often.
// * Rows for 256-wide tiles go to the CTA-pair kernel once its tiles fill half
//   of the pairs (1024 x 4096 x 4096, 64 tiles: 18.6 us against 22.5 us on single
//   CTAs; 512 x 4096 x 4096, 32 tiles: 17.0 against 14.4), else to single CTAs on
//   128-wide tiles.
// * A launch with fewer tiles than CTAs splits the contraction over a cluster,
//   as far as every part keeps two 128-wide blocks (1 token x 7168 x 8192, 56
//   tiles: 18.6, 15.6, 20.9 us for 2, 4, 8 parts; 8 parts no longer fit at once).
struct Shape {
    int tq, splits, ctas;
};
template <typename Tiles>
Shape choose_shape(int sms, double rows, int kblocks, Tiles tiles) {
    Shape s;
    s.tq = rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256;
    if (s.tq == 256) {
        s.splits = 1;
        const int64_t pairs = std::min<int64_t>(tiles(256), sms / 2);
        if (pairs * 2 >= sms / 2) {
            s.ctas = (int)pairs * 2;
            return s;
        }
        s.tq = 128;
    }
    const int64_t slots = (int64_t)sms * linear_ctas_per_sm(s.tq), n = std::max<int64_t>(1, tiles(s.tq));
    s.splits = 1;
    while (s.splits < 8 && n * s.splits * 2 <= slots && kblocks / (s.splits * 2) >= 2) s.splits *= 2;
    s.ctas = (int)std::min<int64_t>(n * s.splits, slots / s.splits * s.splits);
    return s;
}

struct Product {
    const void *p, *p_scale, *q, *q_scale;
    int64_t p_rows, q_rows, cols;        // cols: extent of the contraction (a multiple of 32)
    int64_t p_groups;                    // matrices behind p
    int by_contraction;
    int groups;
    double tile_rows;                    // Q rows that a tile should hold
    LinParams params;                    // epilogue and segments; the rest is filled in here
};

// tiles of a product on tiles of tq Q rows, at most
int64_t product_tiles(const Product& d, int tq) {
    const int64_t whole = (d.q_rows + tq - 1) / tq, pt = (d.p_rows + linear_p_tile(tq) - 1) / linear_p_tile(tq);
    if (d.by_contraction) return d.groups * pt * whole;
    // (a group's last tile may be partly filled; a group without rows has none)
    return pt * (d.params.offsets ? std::min(d.q_rows / tq + std::min<int64_t>(d.groups, d.q_rows / 32), (d.q_rows + 31) / 32) : whole);
}
int product_blocks(const Product& d) {   // 128-wide blocks of one tile's contraction
    const int64_t kb = (d.cols + 127) / 128;
    return (int)(d.by_contraction ? std::max<int64_t>(1, kb / d.groups) : kb);
}

int launch_products(mxa2a_linear* l, const Product* d, int n, const Shape& shape, cudaStream_t stream) {
    LinPack k;
    k.n = n;
    for (int i = 0; i < n; ++i) {
        LinParams& p = k.p[i];
        p = d[i].params;
        p.groups = d[i].groups;
        p.by_contraction = d[i].by_contraction;
        p.p_rows = (int)d[i].p_rows;
        p.q_rows = (int)d[i].q_rows;
        p.blocks = (int)(d[i].cols / 32);
        p.p_row_tiles = (int)((d[i].p_rows + 127) / 128);
        p.q_row_tiles = (int)((d[i].q_rows + 127) / 128);
        p.p_scale = static_cast<const uint8_t*>(d[i].p_scale);
        p.q_scale = static_cast<const uint8_t*>(d[i].q_scale);
        p.p_scale_group = (size_t)mxa2a_scale_tiles_bytes(d[i].p_rows, d[i].cols);
        p.pt = (int)((d[i].p_rows + linear_p_tile(shape.tq) - 1) / linear_p_tile(shape.tq));
        p.qt = (int)((d[i].q_rows + shape.tq - 1) / shape.tq);
        p.splits = shape.splits;
        p.status = l->status;
        p.timeout_ns = l->timeout_ns;
        p.launch_id = l->launch_id + 1;
        LinMaps& m = k.maps[i];
        if (!encode_2d(&m.p, d[i].p, (uint64_t)d[i].cols, (uint64_t)(d[i].p_groups * d[i].p_rows), 128) ||
            !encode_2d(&m.q, d[i].q, (uint64_t)d[i].cols, (uint64_t)d[i].q_rows, (uint32_t)linear_q_box(shape.tq)) ||
            (shape.tq == 256 && !encode_2d(&m.q32, d[i].q, (uint64_t)d[i].cols, (uint64_t)d[i].q_rows, 32)))
            return MXA2A_ERR_CUDA;
        if (shape.tq != 256) m.q32 = m.q;
    }
    ++l->launch_id;
    ++l->launches;
    return cuda_code(launch_linear(k, shape.tq, shape.ctas, stream));
}
int launch_product(mxa2a_linear* l, const Product& d, cudaStream_t stream) {
    return launch_products(l, &d, 1, choose_shape(l->sms, d.tile_rows, product_blocks(d), [&](int tq) { return product_tiles(d, tq); }), stream);
}

// Rows of a tile: all of them without segments; else a group's mean and a fifth
// to spare, from the row capacity that the caller gave, in which every segment
// may hold up to 31 rows of padding.
double rows_per_group(int64_t rows, int groups, bool segs) {
    if (!segs) return (double)rows;
    const int64_t least = std::max<int64_t>(rows - 31ll * groups, rows / 32);
    return 1.2 * (double)least / groups;
}

}  // namespace

extern "C" {

int mxa2a_linear_run(mxa2a_linear* l, int64_t rows, const void* x, const void* x_scale, const void* w, const void* w_scale,
                     void* out, int out_type, void* out_scale, const void* offsets, const void* counts, const void* bias,
                     int activation, const void* residual, void* preact, void* stream) {
    if (!l) return MXA2A_ERR_NULL_PTR;
    const bool mx = mx_type(out_type);
    if (!(mx || out_type == MXA2A_TYPE_BF16 || out_type == MXA2A_TYPE_F32) || activation < MXA2A_ACT_NONE ||
        activation > MXA2A_ACT_SILU)
        return MXA2A_ERR_INVALID_OPTION;
    if (rows < 0 || rows > l->max_rows) return MXA2A_ERR_INVALID_SHAPE;
    if (!offsets != !counts || (!offsets && l->groups != 1)) return MXA2A_ERR_NULL_PTR;
    if (rows && (!x || !x_scale || !w || !w_scale || !out || (mx && !out_scale))) return MXA2A_ERR_NULL_PTR;
    if (!aligned(x, 16) || !aligned(x_scale, 16) || !aligned(w, 16) || !aligned(w_scale, 16) || !aligned(out, 16) ||
        !aligned(out_scale, 16) || !aligned(residual, 16) || !aligned(preact, 16) || !aligned(bias, 4) || !aligned(offsets, 4) ||
        !aligned(counts, 4))
        return MXA2A_ERR_MISALIGNED;
    if (int rc = layer_device(l)) return rc;
    l->launches = 0;
    if (!rows) return MXA2A_OK;
    LinParams p = {};
    p.fmt_q = l->elem_types & 1 ? 1 : 0;                             // x: E5M2 for 1 and 3
    p.fmt_p = l->elem_types == 1 || l->elem_types == 2 ? 1 : 0;      // w: E5M2 for 1 and 2
    p.offsets = static_cast<const int32_t*>(offsets);
    p.counts = static_cast<const int32_t*>(counts);
    p.bias = static_cast<const float*>(bias);
    p.act = activation;
    p.residual = static_cast<const uint16_t*>(residual);
    p.preact = static_cast<uint16_t*>(preact);
    p.out = out;
    p.out_type = out_type;
    p.out_scale = static_cast<uint8_t*>(out_scale);
    const Product d = {w, w_scale, x, x_scale, l->N, rows, l->K, l->groups, 0, l->groups,
                       rows_per_group(rows, l->groups, offsets != nullptr), p};
    return launch_product(l, d, static_cast<cudaStream_t>(stream));
}

int mxa2a_linear_backward(mxa2a_linear* l, int64_t rows, const void* dy, const void* preact, int activation, int grad_format,
                          const void* x_t, const void* x_t_scale, const void* w_t, const void* w_t_scale, void* dx, void* dw,
                          int dw_type, void* dbias, const void* offsets, const void* counts, void* stream) {
    if (!l) return MXA2A_ERR_NULL_PTR;
    if (!l->training || !mx_type(grad_format) || activation < MXA2A_ACT_NONE || activation > MXA2A_ACT_SILU ||
        (dw && dw_type != MXA2A_TYPE_BF16 && dw_type != MXA2A_TYPE_F32))
        return MXA2A_ERR_INVALID_OPTION;
    if (rows < 0 || rows > l->max_rows) return MXA2A_ERR_INVALID_SHAPE;
    if (!offsets != !counts || (!offsets && l->groups != 1)) return MXA2A_ERR_NULL_PTR;
    if (rows && (!dy || (activation != MXA2A_ACT_NONE && !preact) || (dx && (!w_t || !w_t_scale)) ||
                 (dw && (!x_t || !x_t_scale))))
        return MXA2A_ERR_NULL_PTR;
    if (!aligned(dy, 16) || !aligned(preact, 16) || !aligned(x_t, 16) || !aligned(x_t_scale, 16) || !aligned(w_t, 16) ||
        !aligned(w_t_scale, 16) || !aligned(dx, 16) || !aligned(dw, 16) || !aligned(dbias, 4) || !aligned(offsets, 4) ||
        !aligned(counts, 4))
        return MXA2A_ERR_MISALIGNED;
    if (int rc = layer_device(l)) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    l->launches = 0;
    if (!rows) {
        // no rows: the sums over them are zero
        if (dw && cudaMemsetAsync(dw, 0, (size_t)l->groups * l->N * l->K * type_bytes(dw_type), st) != cudaSuccess) return MXA2A_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, (size_t)l->groups * l->N * sizeof(float), st) != cudaSuccess) return MXA2A_ERR_CUDA;
        return MXA2A_OK;
    }
    if (!dx && !dw && !dbias) return MXA2A_OK;
    const Segments seg = {static_cast<const int32_t*>(offsets), static_cast<const int32_t*>(counts), l->groups, rows};
    Quantize q = {};
    q.x = dy;
    q.x_type = MXA2A_TYPE_BF16;
    q.ldx = l->N;
    q.groups = 1;
    q.rows = rows;
    q.cols = l->N;
    q.e5m2 = grad_format == MXA2A_TYPE_E5M2;
    if (dx) {
        q.codes = l->dz;
        q.scale = l->dz_scale;
    }
    if (dw) {
        q.codes_t = l->dz_t;
        q.scale_t = l->dz_t_scale;
    }
    if (activation != MXA2A_ACT_NONE) {
        q.preact = preact;
        q.act = activation;
    }
    q.seg = seg;
    if (dbias) q.colsum = l->colsum;
    if (launch_quantize(q, st) != cudaSuccess) return MXA2A_ERR_CUDA;
    ++l->launches;
    if (dbias) {
        if (launch_bias_sums(l->colsum, seg, l->N, static_cast<float*>(dbias), st) != cudaSuccess) return MXA2A_ERR_CUDA;
        ++l->launches;
    }
    const int fmt_x = l->elem_types & 1 ? 1 : 0, fmt_w = l->elem_types == 1 || l->elem_types == 2 ? 1 : 0;
    Product d[2];
    int n = 0;
    LinParams p = {};
    p.offsets = seg.offsets;
    p.counts = seg.counts;
    p.fmt_q = q.e5m2;
    if (dx) {
        p.fmt_p = fmt_w;
        p.out = dx;
        p.out_type = kTypeBf16;
        d[n++] = {w_t, w_t_scale, l->dz, l->dz_scale, l->K, rows, l->N, l->groups, 0, l->groups,
                  rows_per_group(rows, l->groups, offsets != nullptr), p};
    }
    if (dw) {
        p.fmt_p = fmt_x;
        p.out = dw;
        p.out_type = dw_type;
        d[n++] = {x_t, x_t_scale, l->dz_t, l->dz_t_scale, l->K, l->N, up(rows, 32), 1, 1, l->groups, (double)l->N, p};
    }
    if (n == 2) {
        // Both products in one launch where they want tiles of one width: no seam
        // between them (300 x 1056 x 1024: 20.9 -> 13.8 us).  On pairs only up to 8
        // tiles each: choosing the product per tile costs that kernel 1 to 3 %, which
        // outweighs the seam with many (16380 x 320 x 1120 over 10 experts, 6 tiles
        // each: 57.6 -> 49.7 us; 16384 x 4096 x 4096 over 8, 41 each: 503 -> 507 us).
        auto shape = [&](int i) { return choose_shape(l->sms, d[i].tile_rows, product_blocks(d[i]), [&](int tq) { return product_tiles(d[i], tq); }); };
        const Shape a = shape(0), b = shape(1);
        if (a.tq == b.tq) {
            const Shape both = choose_shape(l->sms, (double)a.tq, std::min(product_blocks(d[0]), product_blocks(d[1])),
                                            [&](int tq) { return product_tiles(d[0], tq) + product_tiles(d[1], tq); });
            const bool few = both.tq < 256 || product_tiles(d[0], 256) + product_tiles(d[1], 256) <= 8 * (l->sms / 2);
            if (both.tq == a.tq && few) return launch_products(l, d, 2, both, st);
        }
    }
    for (int i = 0; i < n; ++i)
        if (int rc = launch_product(l, d[i], st)) return rc;
    return MXA2A_OK;
}

int mxa2a_linear_get_status(mxa2a_linear* l, mxa2a_status* out) {
    if (!l || !out) return MXA2A_ERR_NULL_PTR;
    if (int rc = layer_device(l)) return rc;
    DevStatus st;
    if (cudaMemcpy(&st, l->status, sizeof st, cudaMemcpyDeviceToHost) != cudaSuccess) return MXA2A_ERR_CUDA;
    std::memset(out, 0, sizeof *out);
    out->step = out->segment = out->slot = -1;
    if ((st.key & 0xFF) == 0) return MXA2A_OK;
    out->code = (int)(st.key & 0xFF);
    out->role = st.role;
    out->block = st.block;
    out->observed = st.observed;
    out->expected = st.expected;
    out->launch = (int64_t)(st.key >> 8);
    // Read, so cleared on the device (and before the caller's next launch): replays of
    // a captured run share its launch index, which does not tell whether it was read.
    if (cudaMemset(&l->status->key, 0, sizeof st.key) != cudaSuccess || cudaStreamSynchronize(nullptr) != cudaSuccess)
        return MXA2A_ERR_CUDA;
    return MXA2A_OK;
}

int mxa2a_linear_set_option(mxa2a_linear* l, int key, int64_t v) {
    if (!l) return MXA2A_ERR_NULL_PTR;
    switch (key) {
        case MXA2A_OPT_TIMEOUT_NS:
            // (its waits are for this GPU's own work, microseconds: only a stall is to run out)
            if (v < 1000000) return MXA2A_ERR_INVALID_OPTION;
            l->timeout_ns = v;
            return MXA2A_OK;
        case MXA2A_OPT_ELEM_TYPES:
            if (v < 0 || v > 3) return MXA2A_ERR_INVALID_OPTION;
            l->elem_types = (int)v;
            return MXA2A_OK;
        default: return MXA2A_ERR_INVALID_OPTION;
    }
}

int mxa2a_linear_get_option(mxa2a_linear* l, int key, int64_t* v) {
    if (!l || !v) return MXA2A_ERR_NULL_PTR;
    switch (key) {
        case MXA2A_OPT_TIMEOUT_NS: *v = l->timeout_ns; return MXA2A_OK;
        case MXA2A_OPT_ELEM_TYPES: *v = l->elem_types; return MXA2A_OK;
        case MXA2A_INFO_LAUNCHES: *v = l->launches; return MXA2A_OK;
        case MXA2A_INFO_WORKSPACE_BYTES: *v = (int64_t)l->ws_bytes; return MXA2A_OK;
        default: return MXA2A_ERR_INVALID_OPTION;
    }
}

void mxa2a_linear_destroy(mxa2a_linear* l) {
    if (!l) return;
    int prev = -1;
    cudaGetDevice(&prev);
    if (prev != l->device) cudaSetDevice(l->device);
    cudaDeviceSynchronize();
    if (l->ws) cudaFree(l->ws);
    if (prev >= 0 && prev != l->device) cudaSetDevice(prev);
    delete l;
}

}  // extern "C"
