// What the grouped GEMMs share: the control block with its barriers and segment table, the tile
// schedule, the drain after an abort, and the host side's tensor maps.
#pragma once

#include <mutex>

#include "internal.h"

namespace moe {

constexpr int kMaxG = 1024;      // segment table capacity (weight rows)
constexpr int kMaxStages = 16;
constexpr int kCtrlBytes = 12288;
constexpr int kSmemLimit = 232448;
constexpr int kSmemBudget = kSmemLimit - 1024 - kCtrlBytes;

__host__ __device__ constexpr int round1024(int b) { return (b + 1023) & ~1023; }
__host__ __device__ constexpr int cmin(int a, int b) { return a < b ? a : b; }
__host__ __device__ constexpr int tmem_cols_pow2(int c) {
    return c <= 32 ? 32 : c <= 64 ? 64 : c <= 128 ? 128 : c <= 256 ? 256 : 512;
}

struct CtrlBlock {
    uint64_t full[kMaxStages], empty[kMaxStages];          // operand ring (smem or TMEM)
    uint64_t raw_full[kMaxStages], raw_empty[kMaxStages];  // raw ring (FP4)
    uint64_t tfull[2], tempty[2], drain[6];
    uint32_t tmem_slot;
    int abort;
    int cu[kMaxG];
    int tpre[kMaxG + 1];
};
static_assert(sizeof(CtrlBlock) <= kCtrlBytes, "control block");

// ------------------------------------------------------------------ shared pieces

template <int BT>
__device__ __forceinline__ void decode_tile(int L, const CtrlBlock* c, int G, int NT, int& g, int& nt,
                                            int& row0, int& rows) {
    int lo = 0, hi = G - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (c->tpre[mid] <= L) lo = mid;
        else hi = mid - 1;
    }
    g = lo;
    const int mcount = (c->tpre[g + 1] - c->tpre[g]) / NT;
    const int r = L - c->tpre[g];
    nt = r / mcount;
    const int mt = r - nt * mcount;
    const int start = g ? c->cu[g - 1] : 0;
    // the segment's mcount = ceil(len / BT) token tiles share its rows evenly (in multiples of
    // 16, at most BT each), so that the tiles of one weight block take about the same time and
    // read the weight tile from L2 together; (mcount - 1) * rs < len keeps every tile non-empty
    const int len = c->cu[g] - start;
    const int rs = min(BT, ((len + mcount - 1) / mcount + 15) & ~15);
    row0 = start + mt * rs;
    rows = min(rs, c->cu[g] - row0);
}

// One warp: the segment table (cu, the running maximum of the ends clamped to [0, M_alloc], and the
// running tile count tpre). A segment whose end lies before an earlier one is empty, and the next begins
// where the longest so far ended: every tile has rows, inside the buffers, and no two share one. (Taken
// from the given end before it, a segment after one that fell could get more tiles than rows, and an MMA
// of width 0 with them.)
template <int BT, typename Args>
__device__ __forceinline__ void build_segment_table(const Args& a, CtrlBlock* ctl, int lane) {
    const int G = a.G, NT = a.NT;
    int carry = 0, before = 0;  // tiles, and the running maximum, up to this chunk of 32 segments
    for (int base = 0; base < G; base += 32) {
        const int g = base + lane;
        const int raw = g < G ? a.cu[g] : 0;
        const int own = min(max(raw, 0), a.M_alloc);
        int end = max(own, before);
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, end, off);
            if (lane >= off) end = max(end, n);
        }
        int prev = __shfl_up_sync(0xffffffffu, end, 1);
        if (lane == 0) prev = before;
        if (g < G && (raw != own || own < prev)) report_error(a.err, MOE_ERR_DEVICE, 1000000 + g);
        const int tiles = ((end - prev + BT - 1) / BT) * NT;  // 0 past the last segment, whose own end is 0
        int incl = tiles;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += n;
        }
        if (g < G) {
            ctl->cu[g] = end;
            ctl->tpre[g + 1] = carry + incl;
        }
        carry += __shfl_sync(0xffffffffu, incl, 31);
        before = __shfl_sync(0xffffffffu, end, 31);
    }
    if (lane == 0) ctl->tpre[0] = 0;
}

// What one thread has in flight: the producer's stages (and the parity of each one's last
// issue), or whether a tcgen05 issuer (MMA or scale copies) issued anything.
struct Issued {
    uint32_t mask = 0, par = 0;
    bool tc = false;
};

// After an abort, before the CTA's shared and tensor memory are released: the producer
// waits for its copies to land, a tcgen05 issuer commits to its own drain barrier and waits
// for it. An abort can come after a role left its loop normally, so this runs for every
// role once all have stopped. These waits take the default limit; nothing aborts them.
__device__ __forceinline__ void drain_in_flight(const Issued& is, uint64_t* full, int stages, uint64_t* drain) {
    int never = 0;
    for (int q = 0; q < stages; ++q)
        if (is.mask >> q & 1u) mbar_wait(&full[q], is.par >> q & 1u, &never);
    if (is.tc && drain) {
        mma_commit(drain);
        mbar_wait(drain, 0, &never);
    }
}

// The pipeline-wait limit of a launch (gemm.cu), and the L2 policies of the weight and token copies.
long long wait_limit_cycles();
void l2_policies(int* w, int* t);

// ============================================================ host side

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encode() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// 2-D map over rows of bytes: [rows, cols] with rows `stride` bytes apart; box = box_cols
// bytes x box_rows. Rows and columns past the ends read as zero.
bool make_map_u8(CUtensorMap* m, const void* ptr, uint64_t cols, uint64_t rows, uint64_t stride,
                 uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle sw) {
    EncodeTiledFn enc = get_encode();
    if (!enc) return false;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {stride};
    const cuuint32_t box[2] = {box_cols, box_rows};
    const cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// `done` belongs to the caller's instantiation: kernels of one signature share a
// function-pointer type, so the flag cannot live in a template on that type.
template <typename Kern>
cudaError_t set_smem_once(Kern kern, int bytes, int (&done)[64]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        done[dev] = 1;
    }
    return cudaSuccess;
}

// Pairs that can be resident at once (clusters of two CTAs, one CTA per SM), per device.
template <typename Kern>
int max_pairs_once(Kern kern, int smem, int threads, int (&cache)[64]) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (!cache[dev]) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * (num_sms() / 2));
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) return 0;
        cache[dev] = n;
    }
    return cache[dev];
}

}  // namespace

}  // namespace moe
