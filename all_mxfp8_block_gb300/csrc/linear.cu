// Grouped MXFP8 product with a fused epilogue (bias, activation, residual,
// BF16 / FP32 / MXFP8 output), for sm_103a.
//
//   out[q][p] = act( sum_c Q[q][c] P[p][c] + bias[p] ) + residual[q][p]
//
// One orientation serves every use: the P rows (weight rows) are the MMA's 128
// accumulator lanes, the Q rows (tokens) its columns, 32 to 256 of them.  A
// decode step's few tokens then cost a 32-column tile, the weights stream
// through once, and an output row is written by neighbouring lanes.
//
// CTA roles: warps 0, 2 and 3 issue the TMA loads (the stages in turn), warp 1 owns
// the tensor memory and issues the MMAs, warps 4-7 move the stages' scale bytes
// into tensor memory (one warp per lane quarter), the warps from 8 on are the
// epilogue.  A stage is one 128-wide block of the contraction: 128 P rows,
// tile_q Q rows (128-byte swizzled) and their scale tiles.  CTAs are
// persistent over tiles.  The widest tile is computed by CTA pairs: 256 P rows x
// 256 Q rows, the even CTA issuing the MMAs of both; a tile's MMAs are only as
// wide as its segment needs.  With few tiles a cluster of up to 8 CTAs shares a
// tile's contraction: each accumulates its part and writes every column's
// partial sums to the shared memory of the CTA that finishes the column, which
// adds them in rank order, in the same launch.
//
// Segments start at multiples of 32 rows, so a token tile may start inside a
// 128-row scale tile: the scale warps shift the columns while they copy.  A
// contraction range may start and end inside a 128-wide block: the MMA's
// 32-wide steps outside it are not issued.
//
// What bounds it: a few tokens, the weights' bytes and the launch's latency (1
// token x 7168 x 8192: 15.5 us, 3.9 TB/s; 8 tokens x 4 of 16 experts x 2048 x
// 7168: 36 us, 6.1 TB/s); wide tiles, the MMAs with the time of a stage around
// the ring close behind, and over longer runs the power limit (8192^3 on normally
// distributed operands: 310 us, 3.54 PFLOP/s, over seconds 358 us; on codes whose
// bits switch less 288, of which the MMAs alone are 256).  With an expert's weights
// read for 512 rows the loads come from HBM and are the slower side (32 experts x
// 512 x 2048 x 7168: 158 us, 138 us with one weight matrix).
//
// Every wait is bounded; after one ran out no role of the CTA starts another tile,
// a tile given up is not stored (the output is undefined then) and the status
// block tells.
#include <algorithm>

#include "launch.cuh"
#include "linear.cuh"
#include "mxquant.cuh"
#include "ptx.cuh"

namespace mxa2a {
using namespace ptx;

namespace {

constexpr int kMaxGroups = 1024;
constexpr int kLinMaxStages = 6;
constexpr int kEarly = 4;   // blocks of P fetched before the launch's turn (1 token x 7168 x 8192: 16.0 -> 15.3 us)
constexpr int kProd = 3;   // producer warps: 0, 2 and 3

// 32 lanes x 4 consecutive 32-bit columns
__device__ __forceinline__ void tmem_ld_32x32b_x4(uint32_t taddr, uint32_t (&r)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
}
__device__ __forceinline__ void st_shared_cluster_f32(uint32_t cluster_addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

template <int TQ>
struct LinCfg {
    // The CTA-pair kernel: two CTAs compute 256 P rows x 256 Q rows with one
    // MMA stream (cta_group::2), each holding its 128 P rows and half of the Q
    // rows, so a stage moves and reads a third less shared memory per MMA.
    static constexpr bool kPair = TQ == 256;
    // stages of the ring, and those of a launch whose CTAs share tiles: the others' part of the tile lands
    // behind them (all but this CTA's own share of at most 8: 7/8 of [TQ][128] fp32)
    static constexpr int kStages = kPair ? 5 : TQ == 128 ? 6 : TQ == 64 ? 4 : 5;
    static constexpr int kSplitStages = TQ == 64 ? 3 : 4;
    static constexpr int kCtasPerSm = TQ <= 64 ? 2 : 1;
    static constexpr int kEpiWarps = TQ >= 128 ? 8 : 4;
    static constexpr int kThreads = 256 + 32 * kEpiWarps;
    // Two accumulators.  Two of 256 columns would leave none for the scales, so
    // the pair kernel's overlap by 64 (columns 0..255 and 192..447): those are
    // moved to registers before the next tile's MMAs start, the others are read
    // while it runs.
    static constexpr int kAccStep = kPair ? 192 : TQ;
    static constexpr int kOverlap = TQ - kAccStep;
    static constexpr int kQAtoms = TQ == 32 ? 1 : TQ / 128 + (TQ == 64 ? 2 : 1);   // scale tiles a Q tile may touch
    static constexpr int kQCols = TQ / 32 < 4 ? 4 : TQ / 32;                        // TMEM columns of its scales
    static constexpr uint32_t kSfCol = kAccStep + TQ;
    static constexpr uint32_t kSfCols = 4 + kQCols;
    static constexpr uint32_t kTmem = TQ <= 32 ? 128 : (TQ == 64 ? 256 : 512);
    static constexpr int kQRows = kPair ? 128 : TQ;                                 // Q rows this CTA holds of a tile
    static constexpr int kQBytes = kQRows * 128;
    static constexpr int kColsPerWarp = TQ / (kEpiWarps / 4);
    static constexpr int kStageBytes = kAStageBytes + kQBytes;
    static constexpr size_t oPart = (size_t)kSplitStages * kStageBytes;
    static constexpr size_t kPartBytes = kPair ? 0 : (size_t)TQ * 512 / 8 * 7;
    static constexpr size_t oSfp = (size_t)kStages * kStageBytes > oPart + kPartBytes ? (size_t)kStages * kStageBytes : oPart + kPartBytes;
    static constexpr size_t oSfq = oSfp + (size_t)kStages * 512;
    static constexpr size_t oCtl = oSfq + (size_t)kStages * kQAtoms * 512;
    static constexpr size_t ctl_bytes();
    static_assert(kSfCol + kStages * kSfCols <= kTmem, "tensor memory columns");
};

struct __align__(8) LinCtl {
    uint64_t full[kLinMaxStages];      // operands landed and scales in tensor memory
    uint64_t empty[kLinMaxStages];     // the stage's MMAs are done
    uint64_t sf_full[kLinMaxStages];   // scale tiles landed in shared memory
    uint64_t acc_full[2], acc_empty[2];   // accumulator: a tile's sums are there / all read
    uint64_t acc_part[2];                 // its columns that the other accumulator shares are read
    uint32_t tmem;
    volatile int abort;
    volatile int issued[3];           // stages issued by each producer
    int total, rows_total;            // tiles of the launch; of its first product
    int start[kMaxGroups + 1];        // first tile of each group (grouped Q rows)
};
template <int TQ>
constexpr size_t LinCfg<TQ>::ctl_bytes() { return oCtl + sizeof(LinCtl) + 1024; }

__device__ __forceinline__ void lin_report(const LinParams& p, int role, long long parity) {
    DevStatus* st = p.status;
    const unsigned long long mine = (p.launch_id << 8) | (unsigned long long)kErrTimeout;
    unsigned long long cur = atomicAdd(&st->key, 0ull);
    for (;;) {
        if ((cur >> 8) == p.launch_id) return;   // this launch already reported
        const unsigned long long prev = atomicCAS(&st->key, cur, mine);
        if (prev == cur) break;
        cur = prev;
    }
    st->role = role;
    st->block = blockIdx.x;
    st->step = st->segment = st->slot = -1;
    st->observed = -1;
    st->expected = parity;
    __threadfence();
}

// kCluster: the phase is completed by arrivals from the other CTA of a pair.
template <bool kCluster = false>
__device__ __forceinline__ bool lin_try(uint64_t* bar, uint32_t parity) {
    return kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
}
// Bounded wait of a whole warp for an mbarrier phase, with one answer for all its
// lanes; false once the CTA gave up.  After a time-out every later wait that would
// block returns at once and no role starts another tile, so that all reach the
// end together.
template <bool kCluster = false>
__device__ __forceinline__ bool lin_wait(const LinParams& p, LinCtl* ctl, uint64_t* bar, uint32_t parity, int role) {
    if (__all_sync(kLanes, lin_try<kCluster>(bar, parity))) return true;
    const uint64_t t0 = globaltimer();
    for (uint32_t n = 1;; ++n) {
        if (__all_sync(kLanes, lin_try<kCluster>(bar, parity))) return true;
        if (__any_sync(kLanes, ctl->abort)) return false;
        if ((n & 63) == 0 && __any_sync(kLanes, globaltimer() - t0 > (uint64_t)p.timeout_ns)) {
            if (threadIdx.x % 32 == 0) lin_report(p, role, (long long)parity);
            ctl->abort = 1;
            return false;
        }
    }
}

struct LinItem {
    int which;           // product of the launch
    int group;
    int p0;              // this CTA's first P row inside the group
    int q0;              // first Q row
    int nq;              // Q rows multiplied: up to the segment's end, a multiple of 32
    int q_end;           // Q rows past this are not this tile's (segment end)
    int q_live;          // Q rows past this are padding: zeros are written
    int b0, b1;          // 32-blocks of the contraction
    int kb0, kb1;        // 128-blocks this CTA reads
};

__device__ __forceinline__ int seg_start(const LinParams& p, int g, int limit) {
    // 32-row granular and inside the buffers, whatever the array holds
    return max(0, min(*(p.offsets + g), limit)) & ~31;
}

// Q tiles of a group of Q rows
template <int TQ>
__device__ __forceinline__ int q_tiles(const LinParams& p, int g) {
    int len = p.q_rows;
    if (p.offsets) len = max(0, min(*(p.offsets + g + 1), p.q_rows) - seg_start(p, g, p.q_rows));
    return (len + TQ - 1) / TQ;
}

// a launch's one product, or its two
struct LinOne {
    static constexpr bool kTwo = false;
    const LinParams& p0;
    const CUtensorMap &mp, &mq, &mq32;
    __device__ __forceinline__ const LinParams& p(int) const { return p0; }
    __device__ __forceinline__ const CUtensorMap& map_p(int) const { return mp; }
    __device__ __forceinline__ const CUtensorMap& map_q(int) const { return mq; }
    __device__ __forceinline__ const CUtensorMap& map_q32(int) const { return mq32; }
};
struct LinTwo {
    static constexpr bool kTwo = true;
    const LinPack& k;
    __device__ __forceinline__ const LinParams& p(int i) const { return k.p[i]; }
    __device__ __forceinline__ const CUtensorMap& map_p(int i) const { return k.maps[i].p; }
    __device__ __forceinline__ const CUtensorMap& map_q(int i) const { return k.maps[i].q; }
    __device__ __forceinline__ const CUtensorMap& map_q32(int i) const { return k.maps[i].q32; }
};

template <int TQ, typename K>
__device__ __forceinline__ LinItem lin_item(const K& k, const LinCtl* ctl, int tile, int rank) {
    LinItem it;
    it.which = K::kTwo && tile >= ctl->rows_total ? 1 : 0;
    if (it.which) tile -= ctl->rows_total;
    const LinParams& p = k.p(it.which);
    // (Every role works this out for every tile: three divisions less are half a
    // percent of 16384 x 4096 x 4096.)
    int r, qt;   // tile inside the group; the group's Q tiles
    if (p.by_contraction) {
        const int per = p.pt * p.qt;
        it.group = tile / per;
        r = tile - it.group * per;
        qt = p.qt;
        it.q0 = 0;
        it.q_end = it.q_live = p.q_rows;
        it.b0 = 0;
        it.b1 = p.blocks;
        if (p.offsets) {
            it.b0 = seg_start(p, it.group, p.blocks * 32) / 32;
            it.b1 = max(it.b0, seg_start(p, it.group + 1, p.blocks * 32) / 32);
        }
    } else {
        int lo = 0, hi = p.groups - 1;   // the last group that starts at or before this tile
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (ctl->start[mid] <= tile) lo = mid; else hi = mid - 1;
        }
        it.group = lo;
        r = tile - ctl->start[lo];
        it.q0 = 0;
        it.q_end = it.q_live = p.q_rows;
        qt = q_tiles<TQ>(p, lo);
        if (p.offsets) {
            it.q0 = seg_start(p, lo, p.q_rows);
            it.q_end = lo + 1 == p.groups ? min(*(p.offsets + lo + 1), p.q_rows) : seg_start(p, lo + 1, p.q_rows);
            it.q_live = it.q0 + min(max(0, it.q_end - it.q0), max(0, *(p.counts + lo)));
        }
        it.b0 = 0;
        it.b1 = p.blocks;
    }
    // bands of 2048 P rows, all Q tiles of a band before the next: the CTAs in
    // flight share P and Q tiles in L2
    constexpr int kBand = LinCfg<TQ>::kPair ? 8 : 16;
    const int band = p.pt <= kBand ? 0 : r / (kBand * qt), np = min(kBand, p.pt - band * kBand), rb = r - band * kBand * qt;
    const int q_tile = np == kBand ? rb / kBand : rb / np;
    const int p_tile = band * kBand + rb - q_tile * np;
    // the segment's tiles are equally wide, in 32-row steps (none is empty: the
    // width is at most TQ): no narrow last tile that costs a stage's latency for
    // little work
    const int steps = (it.q_end - it.q0 + 31) >> 5;
    int width = 32;
#pragma unroll
    for (int i = 1; i < TQ / 32; ++i) width += steps > i * qt ? 32 : 0;
    it.q0 += q_tile * width;
    it.q_end = min(it.q_end, it.q0 + width);
    it.p0 = p_tile * (LinCfg<TQ>::kPair ? 256 : 128) + (LinCfg<TQ>::kPair ? rank * 128 : 0);
    it.nq = max(32, min(TQ, (it.q_end - it.q0 + 31) & ~31));   // (a tile past its segment's end, which only foreign offsets make: nothing is stored)
    const int lo = it.b0 / 4, hi = it.b1 > it.b0 ? (it.b1 + 3) / 4 : lo;
    if (LinCfg<TQ>::kPair) {
        it.kb0 = lo;
        it.kb1 = hi;
    } else {
        const int per = (hi - lo + p.splits - 1) / p.splits;
        it.kb0 = min(hi, lo + rank * per);
        it.kb1 = min(hi, it.kb0 + per);
    }
    return it;
}

// ------------------------------------------------------------------ epilogue
// A warp's share of a tile: lanes are 32 consecutive features (P rows), columns
// consecutive tokens (Q rows).
struct LinShare {
    long long row;   // output row of the share's first column
    int end, live;   // columns from the first one on that are written / that hold tokens (the others are zeros)
    int f;           // this lane's feature
    float bias;
};
__device__ __forceinline__ LinShare lin_share(const LinParams& p, const LinItem& it, int f, int col0) {
    LinShare e;
    const int q = it.q0 + col0;
    e.row = (p.by_contraction ? (long long)it.group * p.q_rows : 0) + q;
    e.end = max(0, it.q_end - q);
    e.live = max(0, min(it.q_live - q, e.end));
    e.f = f;
    e.bias = p.bias && f < p.p_rows ? p.bias[(size_t)it.group * p.p_rows + f] : 0.f;
    return e;
}

// BF16 values of two tokens and this lane's feature <-> one token and two
// features (even lanes the first token): one exchange with the neighbouring lane
__device__ __forceinline__ uint32_t lin_swap(uint32_t w, int lane) {
    return __byte_perm(w, __shfl_xor_sync(kLanes, w, 1), lane & 1 ? 0x3276 : 0x5410);
}
// (A piece inside the segment takes the path without a comparison per store,
// its addresses by addition: the products and comparisons of the other path are
// most of its instructions, 1.7 us against 0.7 us for 32 columns.)
template <int NC>
__device__ __forceinline__ void lin_store_bf16(uint16_t* out, int ld, const LinShare& e, int j0, int lane, const float (&v)[NC]) {
    const int odd = lane & 1;
    char* o = reinterpret_cast<char*>(out + (e.row + j0 + odd) * ld + (e.f & ~1));
    const size_t step = (size_t)ld * 4;   // two rows
    if (j0 + NC <= e.end) {
#pragma unroll
        for (int j = 0; j < NC; j += 2, o += step)
            *reinterpret_cast<uint32_t*>(o) = lin_swap(bf16x2_bits(v[j], v[j + 1]), lane);
    } else {
        const int left = e.end - j0 - odd;
#pragma unroll
        for (int j = 0; j < NC; j += 2, o += step) {
            const uint32_t w = lin_swap(bf16x2_bits(v[j], v[j + 1]), lane);
            if (j < left) *reinterpret_cast<uint32_t*>(o) = w;
        }
    }
}

// max |v| over the warp's lanes, keeping a NaN
__device__ __forceinline__ float lin_warp_amax(float v) {
    float r;
    asm("redux.sync.max.abs.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// MXFP8 output: the warp's 32 features are one block of every token.  The
// blocks' largest values come as one reduction per column; lane j then works
// out column j's scale byte and factor for all, and stores the byte.
template <int NC, bool kE5m2>
__device__ __forceinline__ void lin_store_mx(const LinParams& p, const LinShare& e, int j0, int lane, const float (&v)[NC]) {
    const int ld = p.p_rows, i3 = lane & 3;
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const float m = lin_warp_amax(v[j]);
        if (lane == j) amax = m;
    }
    const uint32_t byte = mx_scale_byte(__float_as_uint(amax), mx_emax<kE5m2>());
    const float inv = mx_inv_scale(byte);
    if (lane < NC && j0 + lane < e.end)
        p.out_scale[scale_word(e.f >> 7, e.row + j0 + lane, p.q_row_tiles) + ((e.f >> 5) & 3)] = (uint8_t)byte;
    uint8_t* o = static_cast<uint8_t*>(p.out) + (e.row + j0 + i3) * ld + (e.f & ~3);
    const size_t step = 4 * (size_t)ld;
#pragma unroll
    for (int j = 0; j < NC; j += 4, o += step) {
        float s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = v[j + i] * __shfl_sync(kLanes, inv, j + i);
        uint32_t w = __byte_perm(fp8x2<kE5m2>(s[0], s[1]), fp8x2<kE5m2>(s[2], s[3]), 0x5410);
        // 4 x 4 byte transpose over four lanes: lane 4 a + i then holds features 4 a .. 4 a + 3 of token j + i
        w = __byte_perm(w, __shfl_xor_sync(kLanes, w, 1), lane & 1 ? 0x3715 : 0x6240);
        w = __byte_perm(w, __shfl_xor_sync(kLanes, w, 2), lane & 2 ? 0x3276 : 0x5410);
        if (j0 + j + i3 < e.end) *reinterpret_cast<uint32_t*>(o) = w;
    }
}

// Finish columns j0 .. j0 + NC - 1 of the share: v[j] are their sums.
template <int NC>
__device__ __forceinline__ void lin_store(const LinParams& p, const LinShare& e, int j0, int lane, float (&v)[NC]) {
    static_assert(NC % 4 == 0, "columns");
    if (j0 >= e.end) return;   // (uniform over the warp)
    const int ld = p.p_rows;
#pragma unroll
    for (int j = 0; j < NC; ++j) v[j] += e.bias;   // (0 without one: a branch here spills registers)
    if (j0 + NC > e.live) {
#pragma unroll
        for (int j = 0; j < NC; ++j) v[j] = j0 + j < e.live ? v[j] : 0.f;
    }
    if (p.preact) lin_store_bf16<NC>(p.preact, ld, e, j0, lane, v);
    // (0 stays 0 on padding rows)
    if (p.act == kActGelu) {
#pragma unroll
        for (int j = 0; j < NC; ++j) v[j] = act_value<kActGelu>(v[j]);
    } else if (p.act == kActSilu) {
#pragma unroll
        for (int j = 0; j < NC; ++j) v[j] = act_value<kActSilu>(v[j]);
    } else if (p.act == kActRelu) {
#pragma unroll
        for (int j = 0; j < NC; ++j) v[j] = act_value<kActRelu>(v[j]);
    }
    if (p.residual) {
        const int odd = lane & 1, left = e.live - j0 - odd;
        const char* r = reinterpret_cast<const char*>(p.residual + (e.row + j0 + odd) * ld + (e.f & ~1));
        const size_t step = (size_t)ld * 4;
        uint32_t w[NC / 2];
        if (j0 + NC <= e.live) {
#pragma unroll
            for (int j = 0; j < NC; j += 2, r += step) w[j / 2] = ld_nc_u32(r);
        } else {
#pragma unroll
            for (int j = 0; j < NC; j += 2, r += step)
                w[j / 2] = j < left ? ld_nc_u32(r) : 0u;
        }
#pragma unroll
        for (int j = 0; j < NC; j += 2) {
            const uint32_t t = lin_swap(w[j / 2], lane);
            v[j] += bf16_lo(t);
            v[j + 1] += bf16_hi(t);
        }
    }
    if (p.out_type == kTypeBf16) {
        lin_store_bf16<NC>(static_cast<uint16_t*>(p.out), ld, e, j0, lane, v);
    } else if (p.out_type == kTypeF32) {
        float* o = static_cast<float*>(p.out) + (e.row + j0) * ld + e.f;
        if (j0 + NC <= e.end) {
#pragma unroll
            for (int j = 0; j < NC; ++j, o += ld) *o = v[j];
        } else {
#pragma unroll
            for (int j = 0; j < NC; ++j, o += ld)
                if (j0 + j < e.end) *o = v[j];
        }
    } else {
        if (p.out_type == kTypeE5M2)
            lin_store_mx<NC, true>(p, e, j0, lane, v);
        else
            lin_store_mx<NC, false>(p, e, j0, lane, v);
    }
}

// Zeros for a whole tile of the by-contraction output (BF16 or FP32): rows in
// turn over the warps, 16 bytes a lane.
template <int TQ>
__device__ __forceinline__ void lin_store_zeros(const LinParams& p, const LinItem& it, int warp, int warps, int lane) {
    const int size = p.out_type == kTypeF32 ? 4 : 2, units = min(128, p.p_rows - it.p0) * size / 16;   // (of 8 or 4 columns)
    uint8_t* out = static_cast<uint8_t*>(p.out) + (((long long)it.group * p.q_rows + it.q0) * p.p_rows + it.p0) * size;
    const int rows = it.q_end - it.q0;
    if (size == 2) {   // two rows at a time
        for (int r = 2 * warp + (lane >> 4); r < rows; r += 2 * warps)
            if ((lane & 15) < units) reinterpret_cast<uint4*>(out + (long long)r * p.p_rows * 2)[lane & 15] = make_uint4(0, 0, 0, 0);
    } else {
        for (int r = warp; r < rows; r += warps)
            if (lane < units) reinterpret_cast<uint4*>(out + (long long)r * p.p_rows * 4)[lane] = make_uint4(0, 0, 0, 0);
    }
}

// The pair kernel's registers: its epilogue holds 64 columns beside the piece in
// work; 8 warps x 192 + 8 x 64 are the launch's 16 x 128.  (No function calls in
// that kernel: the split is then not allocated.)
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// fetch a box into L2
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x),
                 "r"(y)
                 : "memory");
}
// arrive on a barrier of another CTA without ordering earlier memory accesses (a
// release waits for every earlier global store, about 1 us; what the barrier
// hands over is tensor memory, whose accesses are complete: tcgen05.wait::st / ::ld)
__device__ __forceinline__ void mbar_arrive_remote_relaxed(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// The cluster barriers of a shared tile: the parts have been written to their
// owners; before the next tile's, they have been read.
__device__ __forceinline__ void lin_tile_end(bool more) {
    cluster_sync();
    if (more) cluster_sync();
}

// The launch's one product (LinOne) or two (LinTwo); kernels of their own, since
// choosing a product per tile costs the pair kernel 3 %.
template <int TQ, typename K>
__device__ __forceinline__ void linear_body(const K& k) {
    using C = LinCfg<TQ>;
    constexpr bool kPair = C::kPair, kTwo = K::kTwo;
    extern __shared__ uint8_t lin_smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(lin_smem_raw) + 1023) & ~uintptr_t(1023));
    LinCtl* ctl = reinterpret_cast<LinCtl*>(smem + C::oCtl);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const bool split = !kPair && k.p(0).splits > 1;
    const int stages = split ? C::kSplitStages : C::kStages;
    const int share = kPair ? 2 : k.p(0).splits;   // CTAs to a tile
    const int rank = kPair || split ? (int)cluster_ctarank() : 0;
    const int first = (int)blockIdx.x / share, stride = (int)gridDim.x / share;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            // the producer's arming and one arrival per scale warp
            mbar_init(&ctl->full[s], 1 + (kPair ? 8 : 4));
            mbar_init(&ctl->empty[s], 1);
            mbar_init(&ctl->sf_full[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl->acc_full[b], 1);
            mbar_init(&ctl->acc_empty[b], kPair ? 2 * C::kEpiWarps : C::kEpiWarps);
            mbar_init(&ctl->acc_part[b], C::kEpiWarps);   // (half of either CTA's epilogue warps)
        }
        ctl->abort = 0;
        ctl->issued[0] = ctl->issued[1] = ctl->issued[2] = 0;
        fence_mbarrier_init();
        prefetch_tensormap(&k.map_p(0));
        prefetch_tensormap(&k.map_q(0));
    }
    if (warp == 1) {
        if (kPair) {
            tmem_alloc_pair(&ctl->tmem, C::kTmem);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(&ctl->tmem, C::kTmem);
            tmem_relinquish();
        }
    }
    const LinParams& p0 = k.p(0);
    if (!kPair && !kTwo && threadIdx.x == 0 && !p0.offsets && !p0.by_contraction && p0.q_rows <= TQ && first < p0.pt) {
        // One tile of Q rows (a decode step): the first weights on their way to L2
        // while the kernel before this one ends.  (A prefetch orders nothing and L2
        // holds what that kernel writes, so weights that it still writes are read
        // as written.)
        const int hi = (p0.blocks + 3) / 4, per = (hi + p0.splits - 1) / p0.splits, lo = rank * per;
        for (int kb = lo; kb < min(min(hi, lo + per), lo + kEarly); ++kb) tma_prefetch_2d(&k.map_p(0), kb * 128, first * 128);
    }
    // (everything above touches this CTA's own memory only)
    grid_wait();
    if (warp == 3) {
        // tiles of the launch; first tile of every group of Q rows
        int sum = 0;
        if (p0.by_contraction) {
            sum = p0.groups * p0.pt * p0.qt;
        } else {
            for (int g0 = 0; g0 < p0.groups; g0 += 32) {
                const int g = g0 + lane;
                int n = 0;
                if (g < p0.groups) n = q_tiles<TQ>(p0, g) * p0.pt;
                int inc = n;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int v = __shfl_up_sync(kLanes, inc, d);
                    if (lane >= d) inc += v;
                }
                if (g < p0.groups) ctl->start[g] = sum + inc - n;
                sum += __shfl_sync(kLanes, inc, 31);
            }
            if (lane == 0) ctl->start[p0.groups] = sum;
        }
        if (lane == 0) {
            ctl->rows_total = sum;
            ctl->total = sum + (kTwo ? k.p(1).groups * k.p(1).pt * k.p(1).qt : 0);
        }
    }
    __syncthreads();
    grid_launch_next();   // (tensor memory is allocated: the next kernel's CTAs cannot take it first)
    tc_fence_after();
    const uint32_t tmem = ctl->tmem;
    const int total = ctl->total;

    if (kPair || split) cluster_sync();   // every CTA of the cluster runs before any touches its shared memory

    // (whole warpgroups take each side; each side's code follows its register count)
    if (warp < 8) {
    if constexpr (kPair) regs_down<64>();
    if (warp == 0 || (warp >= 2 && warp <= kProd)) {
        // ---------------------------------------------------------- TMA producers: the stages in turn
        const bool leader = elect_one();
        const int pid = warp ? warp - 1 : 0;
        int turn = pid;
        int n = 0, stage = 0;
        uint32_t ph = 0;
        // (pair: both CTAs' loads of a stage complete on the even CTA's barrier,
        // which its P producer arms for the bytes of both)
        const uint32_t full0 = kPair ? mapa_shared(smem_u32(&ctl->full[0]), 0) : 0u;
        const uint64_t keep = l2_policy_evict_last();
        for (int tile = first; tile < total; tile += stride) {
            if (__any_sync(kLanes, ctl->abort)) {
                if (split) lin_tile_end(tile + stride < total);
                continue;
            }
            const LinItem it = lin_item<TQ>(k, ctl, tile, rank);
            const LinParams& p = k.p(it.which);
            const int qa = it.q0 >> 7;                                          // first scale tile of the Q rows
            const int atoms = min(((it.q0 & 127) + TQ + 127) >> 7, p.q_row_tiles - qa);
            const int pa = min(it.p0 >> 7, p.p_row_tiles - 1);                  // (a pair's second half may lie past P)
            const int py = (p.by_contraction ? 0 : it.group * p.p_rows) + it.p0;
            const int half = it.nq / 2, boxes = (half + 31) / 32;               // pair: Q rows of each CTA, in boxes of 32
            const bool whole = !kPair || it.nq == TQ;
            const uint32_t bytes = kAStageBytes + (whole ? C::kQBytes : boxes * 32 * 128);
            const int qy = it.q0 + (kPair ? rank * half : 0);
            const uint8_t* sfp = p.p_scale + (p.by_contraction ? 0 : (size_t)it.group * p.p_scale_group) + (size_t)pa * 512;
            const uint8_t* sfq = p.q_scale + (size_t)qa * 512;
            for (int kb = it.kb0; kb < it.kb1; ++kb, ++n) {
                if (turn == 0) {
                    if (!lin_wait<kPair>(k.p(0), ctl, &ctl->empty[stage], ph ^ 1, kRoleTma)) break;
                    if (leader) {
                        uint8_t* pd = smem + (size_t)stage * C::kStageBytes;
                        uint8_t* qd = pd + kAStageBytes;
                        mbar_arrive_expect_tx(&ctl->sf_full[stage], 512 * (1 + atoms));
                        bulk_load(smem + C::oSfp + stage * 512, sfp + (size_t)kb * p.p_row_tiles * 512, 512, &ctl->sf_full[stage]);
                        bulk_load(smem + C::oSfq + (size_t)stage * C::kQAtoms * 512, sfq + (size_t)kb * p.q_row_tiles * 512, 512 * atoms,
                                  &ctl->sf_full[stage]);
                        if constexpr (kPair) {
                            const uint32_t bar = full0 + (uint32_t)stage * sizeof(uint64_t);
                            if (rank == 0) mbar_arrive_expect_tx(&ctl->full[stage], 2 * bytes);
                            tma_load_2d_pair(pd, &k.map_p(it.which), bar, kb * 128, py, keep);
                            if (whole)
                                tma_load_2d_pair(qd, &k.map_q(it.which), bar, kb * 128, qy, keep);
                            else
                                for (int b = 0; b < boxes; ++b)
                                    tma_load_2d_pair(qd + b * 4096, &k.map_q32(it.which), bar, kb * 128, qy + b * 32, keep);
                        } else {
                            mbar_arrive_expect_tx(&ctl->full[stage], bytes);
                            tma_load_2d(pd, &k.map_p(it.which), &ctl->full[stage], kb * 128, py);
                            tma_load_2d(qd, &k.map_q(it.which), &ctl->full[stage], kb * 128, qy);
                        }
                        ctl->issued[pid] = n + 1;
                    }
                    __syncwarp();
                    turn = kProd;
                }
                --turn;
                if (++stage == stages) {
                    stage = 0;
                    ph ^= 1;
                }
            }
            __syncwarp();
            if (split) lin_tile_end(tile + stride < total);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMA issuer (pair: the even CTA's, for both)
        // Its time from one stage to the next is what bounds the product (every
        // instruction here counts once per stage): one wait, no other shared-memory
        // access, the descriptors by addition.
        const uint32_t idesc0 = (kTwo ? 0u : ((uint32_t)p0.fmt_p << 7) | ((uint32_t)p0.fmt_q << 10)) | (1u << 23) |
                                ((kPair ? 16u : 8u) << 24);
        const uint64_t ad0 = smem_desc(smem_u32(smem), 16, 1024, kLayoutSw128);
        const uint64_t bd0 = smem_desc(smem_u32(smem + kAStageBytes), 16, 1024, kLayoutSw128);
        // The whole warp walks the loop (the descriptors stay in uniform registers),
        // one elected lane issues.
        const bool leader = elect_one();
        int stage = 0, acc = 0;
        uint32_t ph = 0;
        for (int tile = first; tile < total; tile += stride) {
            if (kPair && rank != 0) break;
            if (__any_sync(kLanes, ctl->abort)) {
                if (split) lin_tile_end(tile + stride < total);
                continue;
            }
            const LinItem it = lin_item<TQ>(k, ctl, tile, rank);
            if (it.kb1 > it.kb0) {
                const int buf = acc & 1;
                bool ready = lin_wait<kPair>(k.p(0), ctl, &ctl->acc_empty[buf], ((acc >> 1) & 1) ^ 1, kRoleMma);
                if (C::kOverlap && acc) ready &= lin_wait<kPair>(k.p(0), ctl, &ctl->acc_part[buf ^ 1], ((acc - 1) >> 1) & 1, kRoleMma);
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(buf * C::kAccStep);
                uint32_t idesc1 = idesc0 | ((uint32_t)(it.nq >> 3) << 17);
                if (kTwo) idesc1 |= ((uint32_t)k.p(it.which).fmt_p << 7) | ((uint32_t)k.p(it.which).fmt_q << 10);
                int kb = ready ? it.kb0 : it.kb1 + 1;   // (a tile given up ends elsewhere than at kb1)
                for (; kb < it.kb1; ++kb) {
                    if (!lin_wait<kPair>(k.p(0), ctl, &ctl->full[stage], ph, kRoleMma)) break;
                    tc_fence_after();
                    const uint32_t sf = tmem + C::kSfCol + (uint32_t)stage * C::kSfCols;
                    const uint64_t ad = ad0 + (uint32_t)(stage * (C::kStageBytes >> 4));
                    const uint64_t bd = bd0 + (uint32_t)(stage * (C::kStageBytes >> 4));
                    const int k0 = max(0, it.b0 - kb * 4), k1 = min(4, it.b1 - kb * 4);
                    if (leader) {
                        auto step = [&](int k, uint32_t add) {   // 32 of the contraction: +32 bytes inside the swizzled 128, scale byte k
                            const uint32_t idesc = idesc1 | ((uint32_t)k << 4) | ((uint32_t)k << 29);
                            if constexpr (kPair)
                                mma_mxf8f6f4_pair(d, ad + 2ull * k, bd + 2ull * k, idesc, sf, sf + 4, add);
                            else
                                mma_mxf8f6f4(d, ad + 2ull * k, bd + 2ull * k, idesc, sf, sf + 4, add);
                        };
                        const uint32_t later = kb != it.kb0;
                        if (k1 - k0 == 4) {
                            step(0, later);
                            step(1, 1);
                            step(2, 1);
                            step(3, 1);
                        } else {   // a range that starts or ends inside the block
                            for (int k = k0; k < k1; ++k) step(k, later | (uint32_t)(k > k0));
                        }
                        if constexpr (kPair)
                            tc_commit_pair_multicast(&ctl->empty[stage], 0x3);
                        else
                            tc_commit(&ctl->empty[stage]);
                    }
                    __syncwarp();
                    if (++stage == stages) {
                        stage = 0;
                        ph ^= 1;
                    }
                }
                if (leader && kb == it.kb1) {   // (sums of a tile given up are handed to nobody)
                    if constexpr (kPair)
                        tc_commit_pair_multicast(&ctl->acc_full[buf], 0x3);
                    else
                        tc_commit(&ctl->acc_full[buf]);
                }
                ++acc;
            }
            __syncwarp();
            if (split) lin_tile_end(tile + stride < total);
        }
    } else if (warp >= 4 && warp < 8) {
        // ---------------------------------------------------------- scale warps
        const int quarter = warp & 3;
        const uint32_t full0 = kPair ? mapa_shared(smem_u32(&ctl->full[0]), 0) : 0u;
        int stage = 0;
        uint32_t ph = 0;
        for (int tile = first; tile < total; tile += stride) {
            if (__any_sync(kLanes, ctl->abort)) {
                if (split) lin_tile_end(tile + stride < total);
                continue;
            }
            const LinItem it = lin_item<TQ>(k, ctl, tile, rank);
            const int shift = (it.q0 & 127) >> 5;   // 32-row groups before the tile in its first scale tile
            for (int kb = it.kb0; kb < it.kb1; ++kb) {
                if (!lin_wait(k.p(0), ctl, &ctl->sf_full[stage], ph, kRoleScale)) break;
                tc_fence_after();
                // (as many places as stages: the producer filled this stage after the
                // last MMAs that read its place; a wait of its own for them cost 6 %)
                const uint32_t t = tmem + ((uint32_t)(quarter * 32) << 16) + C::kSfCol + (uint32_t)stage * C::kSfCols;
                tmem_st_32x32b_x4(t, reinterpret_cast<const uint4*>(smem + C::oSfp + stage * 512)[lane]);
                const uint8_t* sq = smem + C::oSfq + (size_t)stage * C::kQAtoms * 512;
                // words 4 a + shift .. of the tiles' concatenated columns
                if (shift == 0) {
#pragma unroll
                    for (int a = 0; a < C::kQCols / 4; ++a)
                        tmem_st_32x32b_x4(t + 4 + 4 * a, reinterpret_cast<const uint4*>(sq + a * 512)[lane]);
                } else {
                    uint4 x = reinterpret_cast<const uint4*>(sq)[lane];
#pragma unroll
                    for (int a = 0; a < C::kQCols / 4; ++a) {
                        const uint4 y = a + 1 < C::kQAtoms ? reinterpret_cast<const uint4*>(sq + (a + 1) * 512)[lane] : x;
                        tmem_st_32x32b_x4(t + 4 + 4 * a, shift == 1   ? make_uint4(x.y, x.z, x.w, y.x)
                                                         : shift == 2 ? make_uint4(x.z, x.w, y.x, y.y)
                                                                      : make_uint4(x.w, y.x, y.y, y.z));
                        x = y;
                    }
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (!kPair || rank == 0)
                        mbar_arrive(&ctl->full[stage]);
                    else
                        mbar_arrive_remote_relaxed(full0 + (uint32_t)stage * sizeof(uint64_t));
                }
                if (++stage == stages) {
                    stage = 0;
                    ph ^= 1;
                }
            }
            __syncwarp();
            if (split) lin_tile_end(tile + stride < total);
        }
    }
    } else {
        // ---------------------------------------------------------- epilogue
        if constexpr (kPair) regs_up<192>();
        const int quarter = warp & 3, part = (warp - 8) >> 2;
        // shared tiles: the others' parts of this CTA's columns, [splits - 1][TQ / splits][128] fp32
        const float* parts_in = reinterpret_cast<const float*>(smem + C::oPart);
        const int own = split ? TQ / k.p(0).splits : TQ;
        int acc = 0;
        for (int tile = first; tile < total; tile += stride) {
            if (__any_sync(kLanes, ctl->abort)) {
                if (split) lin_tile_end(tile + stride < total);
                continue;
            }
            const LinItem it = lin_item<TQ>(k, ctl, tile, rank);
            const bool live = it.kb1 > it.kb0;
            const int buf = acc & 1;
            const int f = it.p0 + quarter * 32 + lane;
            const LinParams& p = k.p(it.which);
            const bool in_p = it.p0 + quarter * 32 < p.p_rows;   // (P rows come in blocks of 32: uniform over the warp)
            const uint32_t t = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(buf * C::kAccStep + part * C::kColsPerWarp);
            if (live) {
                if (!lin_wait<kPair>(k.p(0), ctl, &ctl->acc_full[buf], (acc >> 1) & 1, kRoleEpi)) {   // no sums: nothing is stored
                    if (split) lin_tile_end(tile + stride < total);
                    continue;
                }
                tc_fence_after();
            }
            if (p.by_contraction && it.b1 <= it.b0) {   // a group without tokens
                const int warps = split ? C::kEpiWarps * p.splits : C::kEpiWarps;
                lin_store_zeros<TQ>(p, it, (split ? rank * C::kEpiWarps : 0) + warp - 8, warps, lane);
                if (split) lin_tile_end(tile + stride < total);
                continue;
            }
            const LinShare e = lin_share(p, it, f, part * C::kColsPerWarp);
            if constexpr (kPair) {
                // The 64 columns that the next tile's accumulator takes over (the
                // tile's last in the first accumulator, its first in the second)
                // go to registers first and are handed over; 32 columns at a time
                // then come from there or from tensor memory (loading a piece while
                // another is finished measured slower: 35.1 -> 41.3 us on 4096 x 8192
                // x 512).
                const int over = buf == 0 ? C::kColsPerWarp - C::kOverlap : 0;
                const bool mine = live && part == (buf ^ 1);
                constexpr int NC = 32;
                float v[C::kOverlap];
                if (mine) {
#pragma unroll
                    for (int i = 0; i < C::kOverlap; i += NC)
                        tmem_ld_32x32b_x32(t + (uint32_t)(over + i), *reinterpret_cast<uint32_t(*)[32]>(v + i));
                    tc_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (rank == 0)
                            mbar_arrive(&ctl->acc_part[buf]);
                        else
                            mbar_arrive_remote_relaxed(mapa_shared(smem_u32(&ctl->acc_part[buf]), 0));
                    }
                }
#pragma unroll 1
                for (int c = 0; c < C::kColsPerWarp; c += NC) {
                    float u[NC];
                    if (mine && c >= over && c < over + C::kOverlap) {
#pragma unroll
                        for (int j = 0; j < NC; ++j) u[j] = v[j];
#pragma unroll
                        for (int j = 0; j < C::kOverlap - NC; ++j) v[j] = v[j + NC];
                    } else if (live) {
                        tmem_ld_32x32b_x32(t + (uint32_t)c, *reinterpret_cast<uint32_t(*)[32]>(u));
                        tc_wait_ld();
                    } else {
#pragma unroll
                        for (int j = 0; j < NC; ++j) u[j] = 0.f;
                    }
                    if (in_p) lin_store<NC>(p, e, c, lane, u);
                }
                if (live) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (rank == 0)
                            mbar_arrive(&ctl->acc_empty[buf]);
                        else
                            mbar_arrive_remote_relaxed(mapa_shared(smem_u32(&ctl->acc_empty[buf]), 0));
                    }
                    ++acc;
                }
            } else {
                if (!split) {
#pragma unroll 1
                    for (int c = 0; c < C::kColsPerWarp; c += 16) {
                        float v[16];
                        if (live) {
                            tmem_ld_32x32b_x16(t + (uint32_t)c, *reinterpret_cast<uint32_t(*)[16]>(v));
                            tc_wait_ld();
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] = 0.f;
                        }
                        if (in_p) lin_store<16>(p, e, c, lane, v);
                    }
                } else {
                    // every 4 columns to the CTA that finishes them
#pragma unroll 1
                    for (int c0 = part * C::kColsPerWarp; c0 < (part + 1) * C::kColsPerWarp; c0 += 32) {
                        float v[32];
                        if (live) {
                            tmem_ld_32x32b_x32(t + (uint32_t)(c0 - part * C::kColsPerWarp), *reinterpret_cast<uint32_t(*)[32]>(v));
                            tc_wait_ld();
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = 0.f;
                        }
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const int c = c0 + j, to = c / own;
                            if (to == rank) continue;
                            const int slot = rank < to ? rank : rank - 1;
                            const uint32_t at = mapa_shared(smem_u32(parts_in + (slot * own + c - to * own) * 128 + quarter * 32 + lane), to);
#pragma unroll
                            for (int i = 0; i < 4; ++i) st_shared_cluster_f32(at + i * 512, v[j + i]);
                        }
                    }
                    __syncwarp();
                    cluster_sync();
                    // this CTA's columns, the parts added in rank order
                    const LinShare whole = lin_share(p, it, f, 0);
                    for (int c = rank * own + part * 4; c < (rank + 1) * own; c += 4 * (C::kEpiWarps / 4)) {
                        float mine[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
                        if (live) {
                            tmem_ld_32x32b_x4(t + (uint32_t)(c - part * C::kColsPerWarp), *reinterpret_cast<uint32_t(*)[4]>(mine));
                            tc_wait_ld();
                        }
                        const float* in = parts_in + (c - rank * own) * 128 + quarter * 32 + lane;
                        for (int s = 0; s < p.splits; ++s) {
                            if (s == rank) {
#pragma unroll
                                for (int j = 0; j < 4; ++j) v[j] += mine[j];
                            } else {
#pragma unroll
                                for (int j = 0; j < 4; ++j) v[j] += in[j * 128];
                                in += own * 128;
                            }
                        }
                        if (in_p) lin_store<4>(p, whole, c, lane, v);
                    }
                    __syncwarp();
                    if (tile + stride < total) cluster_sync();
                }
                if (live) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->acc_empty[buf]);
                    ++acc;
                }
            }
        }
    }
    __syncthreads();
    if (ctl->abort && threadIdx.x == 0) {
        // loads and MMAs may still be in flight on this CTA's memory: they end
        // within microseconds (pair: the even CTA's barrier counts both CTAs'
        // loads, and both end together below); 1 ms at least, 10 at most
        const uint64_t t0 = globaltimer();
        const int last = max(max(ctl->issued[0], ctl->issued[1]), ctl->issued[2]) - 1;
        for (int i = 0; i < 2 * stages; ++i) {   // operands, then scale tiles
            const int s = i % stages, n = last - ((last - s) % stages + stages) % stages;   // stage s's last use
            if (n < 0 || (i < stages && kPair && rank != 0)) continue;
            while (!lin_try<kPair>(i < stages ? &ctl->full[s] : &ctl->sf_full[s], (n / stages) & 1))
                if (globaltimer() - t0 > 10000000) break;
        }
        while (globaltimer() - t0 < 1000000) {
        }
    }
    __syncthreads();
    if (kPair) cluster_sync();   // both CTAs are done with each other's barriers and tensor memory
    if (warp == 1) {
        tc_fence_after();
        if (kPair)
            tmem_dealloc_pair(tmem, C::kTmem);
        else
            tmem_dealloc(tmem, C::kTmem);
    }
}

template <int TQ>
__global__ void __launch_bounds__(LinCfg<TQ>::kThreads, LinCfg<TQ>::kCtasPerSm)
    linear_kernel(const __grid_constant__ LinParams p, const __grid_constant__ CUtensorMap map_p,
                  const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_q32) {
    linear_body<TQ>(LinOne{p, map_p, map_q, map_q32});
}
template <int TQ>
__global__ void __launch_bounds__(LinCfg<TQ>::kThreads, LinCfg<TQ>::kCtasPerSm)
    linear2_kernel(const __grid_constant__ LinPack k) {
    linear_body<TQ>(LinTwo{k});
}

template <int TQ>
cudaError_t launch_n(const LinPack& k, int ctas, cudaStream_t stream) {
    using C = LinCfg<TQ>;
    static unsigned long long allowed[2] = {};
    const int cluster = C::kPair ? 2 : k.p[0].splits;
    if (k.n > 1) {
        if (cudaError_t e = allow_smem(linear2_kernel<TQ>, C::ctl_bytes(), allowed[1])) return e;
        return launch(linear2_kernel<TQ>, dim3((unsigned)ctas), C::kThreads, C::ctl_bytes(), cluster, stream, k);
    }
    if (cudaError_t e = allow_smem(linear_kernel<TQ>, C::ctl_bytes(), allowed[0])) return e;
    return launch(linear_kernel<TQ>, dim3((unsigned)ctas), C::kThreads, C::ctl_bytes(), cluster, stream, k.p[0], k.maps[0].p,
                  k.maps[0].q, k.maps[0].q32);
}

}  // namespace

cudaError_t launch_linear(const LinPack& k, int tile_q, int ctas, cudaStream_t stream) {
    switch (tile_q) {
        case 32: return launch_n<32>(k, ctas, stream);
        case 64: return launch_n<64>(k, ctas, stream);
        case 128: return launch_n<128>(k, ctas, stream);
        default: return launch_n<256>(k, ctas, stream);
    }
}

int linear_ctas_per_sm(int tile_q) { return tile_q <= 64 ? 2 : 1; }

}  // namespace mxa2a
