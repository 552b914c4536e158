// S3/S5 — the grouped GEMM of MXFP4 activations and MXFP4 weights (W4A4).
//
//   out[r, n] = alpha_g * sum_k a[i(r), k] * W[g][n, k],   i(r) = row_idx[r] or r,
//
// both operands e2m1 with one e8m0 scale per 32 values along K, on the block-scaled tensor-core
// instruction kind::mxf4 (K = 64 per instruction, two scales per row). Products and scales are
// exact; the sum is fp32. Tiling as in the other grouped GEMMs ("swap AB"): a tile is 128 weight
// rows (M) by up to BT token rows (N) of one segment, the MMA as wide as the tile's rows.
//
// A pipeline stage is 256 values of K: 128 bytes of packed codes per row on either side, in the
// 128-byte swizzle, and the stage's scales as 512-byte blocks in tensor-memory copy order. The
// weights come by TMA, and so do token rows in segment order. Token rows that row_idx gathers come
// by cp.async from the gather warps: the four-row TMA gather took about 80 cycles a copy, 1.15 ms
// against 0.30 ms in segment order for 8192 rows x 4096 into 14336. The weights' scales are
// prepared blocks; the tokens' [rows, K/32] bytes may sit at any alignment, which no TMA copy
// takes, so the scale warps load them through registers.
//
// PAIR: two SMs per tile (a cluster of two CTAs, cta_group::2). A pair tile is 256 weight rows, 128
// from each CTA's shared memory, by up to BT tokens, half of them from each, so an SM moves half the
// token operand per product. The leader (rank 0) issues MMAs and scale copies for both. Pairs take token
// rows in segment order only; a kernel of its own brings them into it first.
//
// The scales run ahead of the codes in a ring of their own, so that their way through registers,
// shared and tensor memory is not in line with the codes' copies. Warp roles, each run by whole warps
// with one lane elected to issue:
//   producer   the codes of both sides into the stages (tokens only in segment order)
//   MMA        a stage's four instructions at most
//   copier     scale blocks from the scale ring into tensor-memory slots (PAIR: two, taking the stages in turn)
//   epilogue   four warps: tensor memory -> alpha, bf16 -> out
//   scales     four or eight warps, taking the stages in turn: both sides' scale blocks into the scale ring
//   gather     four warps, in turn too (with row_idx): the token rows' codes by cp.async
// Barriers, all with bounded waits as in the other GEMMs (s stage, d scale-ring entry, b buffer):
//   full[s]      the TMA copies of stage s landed and its scales are in tensor memory (PAIR: on the
//                leader, both CTAs' copies)
//   gfull[s]     the gathered rows of stage s landed
//   empty[s]     the MMAs that read stage s, and its slot of scales, completed (both CTAs)
//   sf_ready[d]  this CTA's scale blocks are in the ring; psf[d], on the leader: the peer's
//   sf_free[d]   they were copied (both CTAs)
//   tfull[b]     accumulator b holds a finished tile (both CTAs);  tempty[b]  it was read (leader)
#include <cmath>

#include "gemm_common.cuh"

namespace moe {

namespace {

constexpr int kStageK = 256;
constexpr int kGatherWarps = 4;
constexpr int kSfRing = 8;

// Tiles whose rows the producer may have written and the MMA warp not yet read: it is at most
// kMaxStages stages, so at most as many tiles, ahead.
constexpr int kTileRing = 32;

// The control block with what only this kernel has.
struct Mxf4Ctl {
    CtrlBlock c;
    int rows[kTileRing];  // rows of this CTA's tiles, written by the producer before the tile's first stage
    uint64_t gfull[kMaxStages], sf_ready[kSfRing], psf[kSfRing], sf_free[kSfRing];
};

// A position in a ring of n entries and the parity of the current turn.
struct Ring {
    int i = 0;
    uint32_t ph = 0;
    MOE_DEV void next(int n) {
        if (++i == n) {
            i = 0;
            ph ^= 1u;
        }
    }
};

struct Mxf4Args {
    const int32_t* cu;
    int G, N, K, KB, NT, NT1, M_alloc;  // NT1: 128-row weight blocks
    __nv_bfloat16* out;
    const float* alpha;
    const uint8_t* w_sf;     // [G, NT1, KS] blocks of 512 bytes, KS = blocks of 128 values
    int KS;
    const uint8_t* a_codes;  // [a_rows, K/2]
    const uint8_t* a_sf;     // [a_rows, K/32]
    int a_rows;
    const int32_t* row_idx;
    DevError* err;
    long long wait_limit;
    int l2_w, l2_t;
};

template <int BT, bool GATHER, bool PAIR>
struct Mxf4Cfg {
    static constexpr int A_BYTES = kTileN * kStageK / 2;
    static constexpr int B_ROWS = PAIR ? BT / 2 : BT;           // this CTA's token rows
    static constexpr int B_BYTES = B_ROWS * kStageK / 2;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int RG = (BT + 127) / 128;                 // 128-row groups of the token side
    static constexpr int SF_ENTRY = 1024 + 2 * RG * 512;        // weights' two blocks, tokens' [128-K half][row group]
    static constexpr int SF_SLOT = 8 + 8 * RG;                  // TMEM columns of a stage's scales
    static constexpr int SF_BASE = 2 * BT;                      // after two accumulators
    // behind the stages: the scale ring, the control block, the gather warps' row tables, the epilogue's staging
    static constexpr int TAB_OFF = (sizeof(Mxf4Ctl) + 15) / 16 * 16;
    static constexpr int STAGING_OFF = (TAB_OFF + (GATHER ? kGatherWarps * B_ROWS * 4 : 0) + 127) / 128 * 128;
    static constexpr int TAIL_BYTES = kSfRing * SF_ENTRY + STAGING_OFF + 4 * 2048;
    static constexpr int STAGES = cmin(kMaxStages, (kSmemLimit - 1024 - TAIL_BYTES) / STAGE);
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE + TAIL_BYTES;
    // Slots in tensor memory, no more than stages: when the copier takes a slot up again, the MMAs of the
    // stage that had it have completed, and with them those of the turn of full[s] before its own.
    static constexpr int SLOTS = cmin(cmin(kSfRing, STAGES), (512 - SF_BASE) / SF_SLOT);
    static constexpr int TMEM_COLS = tmem_cols_pow2(SF_BASE + SLOTS * SF_SLOT);
    // A copier's three waits, copies and commits of a stage are about 600 cycles on a pair, where a stage's
    // MMAs take 350: two take the stages in turn.
    static constexpr int COPIERS = PAIR ? 2 : 1;
    static constexpr int COPIER_WARP0 = 2;
    static constexpr int EPI_WARP0 = COPIER_WARP0 + COPIERS;
    static constexpr int SCALE_WARP0 = EPI_WARP0 + 4;
    // A scale warp spends about 2400 cycles on a stage, most of them on its loads' way; with four warps that
    // was 630 (pairs) and 540 cycles a stage, the pace of the whole kernel (128 experts x 2880 x 2880 with 64
    // rows each: 118 us, with eight warps 104). Smaller tiles wait for the weights from memory, and four are
    // better there (with 32 rows each 98 us against 101).
    static constexpr int SCALE_WARPS = GATHER || BT < 128 ? 4 : 8;
    static constexpr int GATHER_WARP0 = SCALE_WARP0 + SCALE_WARPS;
    static constexpr int THREADS = (GATHER_WARP0 + (GATHER ? kGatherWarps : 0)) * 32;
    static_assert(BT % 16 == 0 && BT >= 16 && BT <= 240, "token tile");
    static_assert(!PAIR || (BT % 32 == 0 && !GATHER), "pair MMA N: a multiple of 32; tokens by TMA");
    static_assert(STAGES >= 3 && SLOTS >= 2 && SMEM_BYTES <= kSmemLimit && SF_BASE + SLOTS * SF_SLOT <= 512, "MXFP4 GEMM config");
    static_assert(B_BYTES % 1024 == 0, "operand alignment");
    // a warp that takes every n-th turn of a ring finds the turn of an entry before its own finished (a wait
    // by parity a whole turn ahead of its barrier would pass at once); a copier that waits for the MMAs of
    // SLOTS stages ago knows those of COPIERS stages before to be done, which has to be a turn of empty[]
    static_assert((!GATHER || STAGES >= kGatherWarps) && kSfRing % SCALE_WARPS == 0 && kSfRing % COPIERS == 0 &&
                      COPIERS <= STAGES, "turns of the rings");
};

MOE_DEV uint4 ld_shared16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// The eight scale bytes of a row's stage, read at whatever alignment the row has; bytes past the
// row's end are 0 (2^-127: their codes are zero).
MOE_DEV uint2 load_scales8(const uint8_t* p, int n) {
    if (n >= 8) {
        const uintptr_t al = reinterpret_cast<uintptr_t>(p);
        if ((al & 7) == 0) return __ldg(reinterpret_cast<const uint2*>(p));
        if ((al & 3) == 0) {
            const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
            return make_uint2(__ldg(q), __ldg(q + 1));
        }
        if ((al & 1) == 0) {
            const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
            return make_uint2((uint32_t)__ldg(q) | (uint32_t)__ldg(q + 1) << 16,
                              (uint32_t)__ldg(q + 2) | (uint32_t)__ldg(q + 3) << 16);
        }
    }
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) w[i >> 2] |= (uint32_t)__ldg(p + i) << (8 * (i & 3));
    return make_uint2(w[0], w[1]);
}

template <int BT, bool GATHER, bool PAIR>
__global__ void __launch_bounds__(Mxf4Cfg<BT, GATHER, PAIR>::THREADS, 1)
    grouped_gemm_mxf4_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                             const Mxf4Args a) {
    using C = Mxf4Cfg<BT, GATHER, PAIR>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* sf_ring = smem + C::STAGES * C::STAGE;
    Mxf4Ctl* mc = reinterpret_cast<Mxf4Ctl*>(sf_ring + kSfRing * C::SF_ENTRY);
    CtrlBlock* ctl = &mc->c;
    volatile int* abort_flag = &ctl->abort;
    Issued is;
    auto opA = [&](int s) { return smem + s * C::STAGE; };
    auto opB = [&](int s) { return smem + s * C::STAGE + C::A_BYTES; };
    auto sfA = [&](int d) { return sf_ring + d * C::SF_ENTRY; };
    auto sfB = [&](int d, int h, int rg) { return sf_ring + d * C::SF_ENTRY + 1024 + (h * C::RG + rg) * 512; };
    const int warp = __shfl_sync(0xffffffffu, warp_id(), 0), lane = lane_id();
    const int G = a.G, NT = a.NT, KB = a.KB;  // NT: blocks of 128 weight rows, or of 256 (PAIR)
    const int rank = PAIR ? (int)cluster_ctarank() : 0;
    const bool leader = rank == 0;
    const int first_tile = PAIR ? blockIdx.x >> 1 : blockIdx.x, tile_step = PAIR ? gridDim.x >> 1 : gridDim.x;
    // the MMA's width for a tile's rows, and the first row of this CTA's part of the token operand
    auto mma_n = [](int rows) { return PAIR ? (rows + 31) & ~31 : (rows + 15) & ~15; };
    auto part0 = [&](int rows) { return rank * (mma_n(rows) / 2); };
    // A whole warp's wait; wait_peer where threads of the pair's other CTA arrive.
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.wait_limit));
    };
    auto wait_peer = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait_relaxed(bar, parity, abort_flag, a.wait_limit));
    };
    auto commit = [](uint64_t* bar) {  // in both CTAs of a pair
        if (PAIR) mma_commit_pair(bar, 0x3);
        else mma_commit(bar);
    };
    auto commit_here = [](uint64_t* bar) {
        if (PAIR) mma_commit_pair_here(bar);
        else mma_commit(bar);
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&ctl->full[s], 2);  // the producer and the copier
            mbar_init(&ctl->empty[s], 1);
            mbar_init(&mc->gfull[s], 32);  // the lanes of the gather warp that copied the stage's rows
        }
        for (int d = 0; d < kSfRing; ++d) {
            mbar_init(&mc->sf_ready[d], 2);  // the weights' copy and the tokens' scale warp
            mbar_init(&mc->psf[d], 1);
            mbar_init(&mc->sf_free[d], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl->tfull[b], 1);
            mbar_init(&ctl->tempty[b], PAIR ? 8 : 4);
        }
        for (int i = 0; i < 1 + C::COPIERS; ++i) mbar_init(&ctl->drain[i], 1);
        ctl->abort = 0;
        fence_barrier_init();
    }
    if (threadIdx.x == 32) {
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_w);
    }
    if (warp == 1) {
        if (PAIR) {
            tmem_alloc_pair(&ctl->tmem_slot, C::TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(&ctl->tmem_slot, C::TMEM_COLS);
            tmem_relinquish();
        }
    }
    pdl_wait();
    if (warp == 0) build_segment_table<BT>(a, ctl, lane);
    tc_fence_before();
    if (PAIR) cluster_sync();  // both CTAs' barriers initialised and tensor memory allocated
    else __syncthreads();
    tc_fence_after();
    pdl_launch();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, ctl->tmem_slot, 0);
    const int total = __shfl_sync(0xffffffffu, ctl->tpre[G], 0);
    // A tile's segment, weight block and rows, the same in every lane.
    auto tile = [&](int L, int& g, int& nt, int& row0, int& rows) {
        decode_tile<BT>(L, ctl, G, NT, g, nt, row0, rows);
        g = __shfl_sync(0xffffffffu, g, 0);
        nt = __shfl_sync(0xffffffffu, nt, 0);
        row0 = __shfl_sync(0xffffffffu, row0, 0);
        rows = __shfl_sync(0xffffffffu, rows, 0);
    };
    auto give_up = [&](int site) {  // this warp's wait ran out, or another's did
        if (lane == 0) {
            report_error(a.err, MOE_ERR_TIMEOUT, site);
            ctl->abort = 1;
        }
    };

    if (warp == 0) {
        // ---------------- producer
        const uint64_t pol_w = l2_policy(a.l2_w), pol_t = l2_policy(a.l2_t);
        constexpr uint32_t BYTES = C::A_BYTES + (GATHER ? 0 : C::B_BYTES);
        Ring st;
        int n = 0;
        bool ok = true;
        for (int L = first_tile; L < total && ok; L += tile_step, ++n) {
            int g, nt, row0, rows;
            tile(L, g, nt, row0, rows);
            const int wrow = (PAIR ? 2 * nt + rank : nt) * kTileN;  // a block past the last reads as zeros
            const int trow = row0 + part0(rows);
            for (int kb = 0; kb < KB; ++kb) {
                if (!wait(&ctl->empty[st.i], st.ph ^ 1u)) {
                    ok = false;
                    break;
                }
                const int s = st.i, x = kb * (kStageK / 2);
                if (elect_one()) {
                    if (kb == 0) mc->rows[n % kTileRing] = rows;  // the arrival below publishes it
                    if (PAIR) {
                        const uint32_t bar = mapa_shared(smem_u32(&ctl->full[s]), 0);  // the leader's
                        if (leader) mbar_arrive_expect_tx(&ctl->full[s], 2 * BYTES);
                        tma_load_3d_pair(opA(s), &tm_w, bar, x, wrow, g);
                        if (!GATHER) tma_load_2d_pair(opB(s), &tm_a, bar, x, trow);
                    } else {
                        mbar_arrive_expect_tx(&ctl->full[s], BYTES);
                        tma_load_3d_p(opA(s), &tm_w, &ctl->full[s], x, wrow, g, pol_w);
                        if (!GATHER) tma_load_2d_p(opB(s), &tm_a, &ctl->full[s], x, trow, pol_t);
                    }
                }
                is.mask |= 1u << s;
                is.par = (is.par & ~(1u << s)) | (st.ph << s);
                st.next(C::STAGES);
            }
        }
        if (!ok) give_up(1);
    } else if (warp == 1) {
        // ---------------- MMAs
        if (leader) {
            const uint64_t a0 = sw128_kmajor_desc(smem_u32(opA(0))), b0 = sw128_kmajor_desc(smem_u32(opB(0)));
            constexpr uint32_t id2 = idesc_mxf4(0, 0, 2) ^ idesc_mxf4(0, 0, 0), at2 = 2u << 30;
            Ring st, sl;
            int b = 0, n = 0;
            uint32_t bph = 0, idesc = 0;
            bool ok = true, next_full = false, next_g = !GATHER;
            for (int L = first_tile; L < total && ok; L += tile_step, ++n) {
                if (!(PAIR ? wait_peer(&ctl->tempty[b], bph ^ 1u) : wait(&ctl->tempty[b], bph ^ 1u))) {
                    ok = false;
                    break;
                }
                const uint32_t d = tmem_base + (uint32_t)(b * BT);
                for (int kb = 0; kb < KB; ++kb) {
                    if ((!next_full && !wait(&ctl->full[st.i], st.ph)) || (!next_g && !wait(&mc->gfull[st.i], st.ph))) {
                        ok = false;
                        break;
                    }
                    if (GATHER) fence_proxy_async_smem();  // the gathered rows came by the generic proxy
                    tc_fence_after();
                    if (kb == 0)
                        idesc = idesc_mxf4(PAIR ? 2 * kTileN : kTileN,
                                           mma_n(__shfl_sync(0xffffffffu, mc->rows[n % kTileRing], 0)), 0);
                    const int s = st.i, t = sl.i;
                    st.next(C::STAGES);
                    sl.next(C::SLOTS);
                    // a look at the next stage's barriers, whose answers come while the MMAs are issued
                    next_full = mbar_test(&ctl->full[st.i], st.ph);
                    if (GATHER) next_g = mbar_test(&mc->gfull[st.i], st.ph);
                    const uint64_t as = a0 + (uint64_t)(s * (C::STAGE >> 4)), bs = b0 + (uint64_t)(s * (C::STAGE >> 4));
                    const uint32_t sfa = tmem_base + (uint32_t)(C::SF_BASE + t * C::SF_SLOT);
                    const int steps = (a.K - kb * kStageK + 63) >> 6;
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (j < steps) {
                                const uint32_t id = j & 1 ? idesc | id2 : idesc, at = j & 1 ? at2 : 0u;
                                const uint32_t fa = (sfa + 4 * (j >> 1)) | at, fb = (sfa + 8 + 4 * C::RG * (j >> 1)) | at;
                                const uint32_t acc = j ? 1u : (uint32_t)(kb != 0);
                                if (PAIR) mma_mxf4_ss_pair(d, as + 2 * j, bs + 2 * j, id, fa, fb, acc);
                                else mma_mxf4_ss(d, as + 2 * j, bs + 2 * j, id, fa, fb, acc);
                            }
                        }
                        is.tc = true;
                        commit(&ctl->empty[s]);
                    }
                    next_full = __all_sync(0xffffffffu, next_full);
                    if (GATHER) next_g = __all_sync(0xffffffffu, next_g);
                }
                if (!ok) break;
                if (elect_one()) commit(&ctl->tfull[b]);
                b ^= 1;
                if (b == 0) bph ^= 1u;
            }
            if (!ok) give_up(2);
        }
    } else if (warp < C::EPI_WARP0) {
        // ---------------- scale blocks: ring -> tensor memory (peer: tells the leader they are in its ring),
        // every COPIERS-th stage
        const int mine = warp - C::COPIER_WARP0;
        const uint64_t ring0 = sf_block_desc(smem_u32(sf_ring));
        // st: the stage that the scales are of; last: the stage that had the slot before, SLOTS ago
        Ring rg, sl, st, last;
        int it = 0;
        bool ok = true;
        for (int L = first_tile; L < total && ok; L += tile_step) {
            int g, nt, row0, rows;
            tile(L, g, nt, row0, rows);
            const bool wide = C::RG > 1 && mma_n(rows) > 128;  // the second 128-row group is in use
            for (int kb = 0; kb < KB; ++kb, ++it) {
                if (C::COPIERS == 1 || it % C::COPIERS == mine) {
                    if (!wait(&mc->sf_ready[rg.i], rg.ph) ||
                        (leader && ((PAIR && !wait_peer(&mc->psf[rg.i], rg.ph)) ||
                                    (it >= C::SLOTS && !wait(&ctl->empty[last.i], last.ph))))) {
                        ok = false;
                        break;
                    }
                    if (PAIR && leader) fence_acquire_smem_cluster();
                    tc_fence_after();
                    const uint64_t src = ring0 + (uint64_t)(rg.i * (C::SF_ENTRY >> 4));
                    const uint32_t sfa = tmem_base + (uint32_t)(C::SF_BASE + sl.i * C::SF_SLOT), sfb = sfa + 8;
                    const bool both = a.KS - 2 * kb > 1;  // both 128-K halves
                    auto copy = [](uint32_t t, uint64_t desc) {
                        if (PAIR) tmem_cp_32x128b_x4_pair(t, desc);
                        else tmem_cp_32x128b_x4(t, desc);
                    };
                    if (elect_one()) {
                        if (!leader) {
                            fence_release_smem_cluster();  // both sides' blocks, which this warp has waited for
                            mbar_arrive_remote(mapa_shared(smem_u32(&mc->psf[rg.i]), 0));
                        } else {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                if (h == 0 || both) {
                                    copy(sfa + 4 * h, src + 32 * h);
                                    copy(sfb + 4 * h * C::RG, src + 64 + 32 * h * C::RG);
                                    if (wide) copy(sfb + 4 * (h * C::RG + 1), src + 64 + 32 * (h * C::RG + 1));
                                }
                            }
                            is.tc = true;
                            commit_here(&ctl->full[st.i]);
                            commit(&mc->sf_free[rg.i]);
                        }
                    }
                }
                rg.next(kSfRing);
                sl.next(C::SLOTS);
                st.next(C::STAGES);
                if (it >= C::SLOTS) last.next(C::STAGES);
            }
        }
        if (!ok) give_up(4);
    } else if (warp < C::SCALE_WARP0) {
        // ---------------- epilogue (four warps): lane = weight row, columns = tokens
        // A warp's 32 weight rows of 32 tokens are transposed through its own 2 KB of shared memory (64
        // bytes a token, the 16-byte pieces of token t at c ^ (t / 2 % 4) against bank conflicts), so that
        // a store writes 64 contiguous bytes of eight tokens. Stores of two bytes a lane straight from
        // the registers held the kernel at 228 us in the 14336 x 4096 case without any loads or MMAs.
        const int q = warp & 3;
        const uint32_t stage = smem_u32(mc) + C::STAGING_OFF + q * 2048;
        // stmatrix: lane 8 i + k addresses token k + 8 (i / 2), 16-byte piece (i % 2) + 2 (row half)
        const int st_t = (lane & 7) + 8 * (lane >> 4), st_c = (lane >> 3) & 1;
        const uint32_t st0 = st_t * 64 + ((st_c ^ (st_t >> 1 & 3)) << 4), st1 = st_t * 64 + (((st_c + 2) ^ (st_t >> 1 & 3)) << 4);
        const uint32_t ld0 = (lane >> 2) * 64 + (((lane & 3) ^ (lane >> 3 & 3)) << 4);  // token 8 i + lane / 4, piece lane % 4
        int b = 0;
        uint32_t bph = 0;
        for (int L = first_tile; L < total; L += tile_step) {
            int g, nt, row0, rows;
            tile(L, g, nt, row0, rows);
            if (!wait(&ctl->tfull[b], bph)) {
                give_up(3);
                break;
            }
            tc_fence_after();
            const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * BT);
            const int n0 = (PAIR ? 2 * nt + rank : nt) * kTileN + q * 32;
            const float al = a.alpha ? a.alpha[g] : 1.0f;
#pragma unroll 1
            for (int c0 = 0; c0 < rows; c0 += 32) {
                const bool more = c0 + 16 < rows;  // the MMA wrote rows rounded up to 16
                uint32_t r[4][8];                  // [16-token half][16-row half]
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < 2 || more) tmem_ld_16x16(tb + c0 + 16 * (i >> 1) + ((uint32_t)(16 * (i & 1)) << 16), r[i]);
                tmem_ld_wait();
                __syncwarp();  // the previous chunk has been read
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t d[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(r[i][2 * j]) * al,
                                                                       __uint_as_float(r[i][2 * j + 1]) * al);
                        d[j] = *reinterpret_cast<const uint32_t*>(&v);
                    }
                    if (i < 2 || more) stmatrix_x4_trans(stage + 1024 * (i >> 1) + (i & 1 ? st1 : st0), d[0], d[1], d[2], d[3]);
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 8 * i + (lane >> 2), n = n0 + 8 * (lane & 3);
                    const uint4 v = ld_shared16(stage + 512 * i + ld0);
                    if (c0 + t < rows && n < a.N)
                        *reinterpret_cast<uint4*>(a.out + (size_t)(row0 + c0 + t) * a.N + n) = v;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) mbar_arrive_remote(mapa_shared(smem_u32(&ctl->tempty[b]), 0));
                else mbar_arrive(&ctl->tempty[b]);
            }
            b ^= 1;
            if (b == 0) bph ^= 1u;
        }
        // rows past the last segment are zero
        const int start = ctl->cu[G - 1];
        const long long n8 = (long long)(a.M_alloc - start) * (a.N / 8);
        uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)start * a.N);
        for (long long i = (long long)blockIdx.x * 128 + threadIdx.x - 32 * C::EPI_WARP0; i < n8; i += (long long)gridDim.x * 128)
            o[i] = make_uint4(0u, 0u, 0u, 0u);
    } else if (warp < C::GATHER_WARP0) {
        // ---------------- scale warp: every SCALE_WARPS-th stage
        constexpr int NR = (BT + 31) / 32;  // rows per lane: lane, lane + 32, ...
        const int mine = warp - C::SCALE_WARP0;
        const int row_bytes = a.K / 32;
        const uint64_t pol_w = l2_policy(a.l2_w);
        int it = 0;
        Ring rg;
        bool ok = true;
        for (int L = first_tile; L < total && ok; L += tile_step) {
            int g, nt, row0, rows;
            tile(L, g, nt, row0, rows);
            // a pair's second block past the last one repeats the last block's scales (its codes are zeros)
            const int wb = min(PAIR ? 2 * nt + rank : nt, a.NT1 - 1);
            const uint8_t* wsf = a.w_sf + ((size_t)g * a.NT1 + wb) * a.KS * 512;
            const uint8_t* src[NR];
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int r = 32 * i + lane;
                src[i] = nullptr;
                if (r < rows) {
                    const int v = GATHER ? a.row_idx[row0 + r] : row0 + r;
                    if (!GATHER || (v >= 0 && v < a.a_rows)) src[i] = a.a_sf + (size_t)v * row_bytes;
                }
            }
            for (int kb = 0; kb < KB; ++kb, ++it) {
                if (it % C::SCALE_WARPS == mine) {
                    const int d = rg.i;
                    uint2 v[4 * C::RG];
#pragma unroll
                    for (int i = 0; i < 4 * C::RG; ++i) {
                        v[i] = make_uint2(0u, 0u);
                        if (i < NR && src[i < NR ? i : 0]) v[i] = load_scales8(src[i < NR ? i : 0] + kb * 8, row_bytes - kb * 8);
                    }
                    if (!wait(&mc->sf_free[d], rg.ph ^ 1u)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        const uint32_t bytes = min(1024, (a.KS - 2 * kb) * 512);
                        mbar_arrive_expect_tx(&mc->sf_ready[d], bytes);
                        bulk_load_p(sfA(d), wsf + (size_t)kb * 1024, bytes, &mc->sf_ready[d], pol_w);
                    }
                    is.mask |= 1u << d;
                    is.par = (is.par & ~(1u << d)) | (rg.ph << d);
#pragma unroll
                    for (int r = 0; r < C::RG; ++r) {
                        reinterpret_cast<uint4*>(sfB(d, 0, r))[lane] =
                            make_uint4(v[4 * r].x, v[4 * r + 1].x, v[4 * r + 2].x, v[4 * r + 3].x);
                        reinterpret_cast<uint4*>(sfB(d, 1, r))[lane] =
                            make_uint4(v[4 * r].y, v[4 * r + 1].y, v[4 * r + 2].y, v[4 * r + 3].y);
                    }
                    fence_proxy_async_smem();  // the copies read these bytes through the async proxy
                    __syncwarp();
                    if (elect_one()) mbar_arrive(&mc->sf_ready[d]);
                }
                rg.next(kSfRing);
            }
        }
        if (!ok) give_up(5);
    } else {
        // ---------------- gather warp: the token rows of every kGatherWarps-th stage by cp.async. Lane
        // 8 rr + c copies chunk c (16 bytes) of rows 4 i + rr, so that one instruction reads four whole
        // 128-byte row pieces; chunk c of row r lands at c ^ (r % 8), the 128-byte swizzle. Rows past
        // the tile's, without a source, and chunks past K are zeros.
        const int mine = warp - C::GATHER_WARP0;
        const int rr = lane >> 3, c = lane & 7;
        int* tab = reinterpret_cast<int*>(reinterpret_cast<char*>(mc) + C::TAB_OFF) + mine * C::B_ROWS;
        const uint64_t pol_t = l2_policy(a.l2_t);
        const int row_bytes = a.K / 2;
        // rows 4 i + rr with even and odd i differ in bit 2 of the swizzle's row
        const uint32_t sw0 = (uint32_t)(rr * 128 + ((c ^ rr) << 4)), sw1 = (uint32_t)(rr * 128 + ((c ^ (rr + 4)) << 4));
        int it = 0;
        Ring st;
        bool ok = true;
        for (int L = first_tile; L < total && ok; L += tile_step) {
            int g, nt, row0, rows;
            tile(L, g, nt, row0, rows);
            const int part = mma_n(rows);
            __syncwarp();
            for (int i = lane; i < part; i += 32) {
                int v = -1;
                if (i < rows) {
                    v = a.row_idx[row0 + i];
                    if (v < 0 || v >= a.a_rows) {  // counts as a row of zeros
                        report_error(a.err, MOE_ERR_DEVICE, row0 + i);
                        v = -1;
                    }
                }
                tab[i] = v;
            }
            __syncwarp();
            for (int kb = 0; kb < KB; ++kb, ++it) {
                if (it % kGatherWarps == mine) {
                    if (!wait(&ctl->empty[st.i], st.ph ^ 1u)) {
                        ok = false;
                        break;
                    }
                    const int off = kb * (kStageK / 2) + c * 16;
                    const bool in = off < row_bytes;
                    const uint8_t* base = a.a_codes + (in ? off : 0);
                    const uint32_t dst = smem_u32(opB(st.i));
#pragma unroll 4
                    for (int i = 0; i < part / 4; i += 2) {
                        const int r0 = tab[4 * i + rr], r1 = tab[4 * i + 4 + rr];
                        cp_async16_p(dst + i * 512 + sw0, base + (size_t)max(r0, 0) * row_bytes, in && r0 >= 0 ? 16u : 0u, pol_t);
                        cp_async16_p(dst + i * 512 + 512 + sw1, base + (size_t)max(r1, 0) * row_bytes, in && r1 >= 0 ? 16u : 0u, pol_t);
                    }
                    cp_async_arrive_noinc(&mc->gfull[st.i]);
                }
                st.next(C::STAGES);
            }
        }
        cp_async_wait_all();
        if (!ok) give_up(6);
    }

    // After an abort (PAIR: always; in a normal run these waits return at once) every role lets what
    // it has in flight finish, so that no memory is released, or left by a CTA of the pair, in use.
    // Copies get about 100 microseconds a stage, far longer than one takes: after an abort the leader's
    // barriers may wait for copies that the peer never issued.
    tc_fence_before();
    __syncthreads();
    if (PAIR || *abort_flag) {
        int never = 0;
        constexpr long long COPY_LIMIT = 200000;
        const bool scale = warp >= C::SCALE_WARP0 && warp < C::GATHER_WARP0;
        if (scale) {  // entry d is always the same warp's: its latest copy is the one to wait for
            for (int d = 0; d < kSfRing; ++d)
                if (is.mask >> d & 1u) mbar_wait(&mc->sf_ready[d], is.par >> d & 1u, &never, COPY_LIMIT);
        } else if (warp == 0 && leader) {
            for (int q = 0; q < C::STAGES; ++q)
                if (is.mask >> q & 1u) mbar_wait(&ctl->full[q], is.par >> q & 1u, &never, COPY_LIMIT);
        } else if (warp == 0 && is.mask && *abort_flag) {
            // the peer's copies complete on the leader's barriers, which it cannot watch
            const long long t0 = clock64();
            while (clock64() - t0 < COPY_LIMIT) {
            }
        }
        if (is.tc) {
            uint64_t* drain = &ctl->drain[warp - 1];
            commit_here(drain);
            mbar_wait(drain, 0, &never);
        }
        tc_fence_before();
    }
    if (PAIR) cluster_sync();
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        if (PAIR) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
        else tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

// Packed codes as bytes: [rows, K/2] tokens, or [G, N, Kp/2] weights in boxes of 128 bytes.
bool make_map_codes(CUtensorMap* m, const void* ptr, uint64_t bytes, uint64_t N, uint64_t G) {
    EncodeTiledFn enc = get_encode();
    if (!enc) return false;
    const cuuint64_t dims[3] = {bytes, N, G};
    const cuuint64_t strides[2] = {bytes, N * bytes};
    const cuuint32_t box[3] = {kStageK / 2, kTileN, 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kPairTile = 192, kOrderedTile = 64;  // kOrderedTile: from here on rows are gathered first

template <int BT, bool GATHER, bool PAIR>
cudaError_t set_attributes() {
    return cudaFuncSetAttribute(grouped_gemm_mxf4_kernel<BT, GATHER, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Mxf4Cfg<BT, GATHER, PAIR>::SMEM_BYTES);
}
template <int BT>
cudaError_t set_attributes_of_tile() {
    const cudaError_t e = set_attributes<BT, false, false>();
    return e == cudaSuccess ? set_attributes<BT, true, false>() : e;
}

// What the first call on a device sets up, for every tile: a later call of another size has nothing left to
// do before its launches, in a stream capture too. pairs: how many CTA pairs run at once, 0 where none can.
struct DeviceSetup {
    std::once_flag once;
    cudaError_t status = cudaSuccess;
    int pairs = 0;
};
cudaError_t device_setup(int* pairs) {
    static DeviceSetup setups[64];
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    DeviceSetup& d = setups[dev];
    std::call_once(d.once, [&d] {
        cudaError_t (*const all[])() = {set_attributes_of_tile<16>, set_attributes_of_tile<32>, set_attributes_of_tile<64>,
                                        set_attributes_of_tile<128>, set_attributes<kPairTile, false, true>};
        for (auto set : all)
            if (d.status == cudaSuccess) d.status = set();
        if (d.status != cudaSuccess) return;
        using C = Mxf4Cfg<kPairTile, false, true>;
        int cache[64] = {0};
        d.pairs = max_pairs_once(grouped_gemm_mxf4_kernel<kPairTile, false, true>, C::SMEM_BYTES, C::THREADS, cache);
        if (d.pairs < 1) cudaGetLastError();  // no error of the call's: it takes one-SM tiles
    });
    *pairs = d.pairs;
    return d.status;
}

template <int BT, bool GATHER, bool PAIR>
cudaError_t run_mxf4(const CUtensorMap& ta, const CUtensorMap& tw, Mxf4Args a, int maxp, cudaStream_t st, bool pdl) {
    using C = Mxf4Cfg<BT, GATHER, PAIR>;
    auto kern = grouped_gemm_mxf4_kernel<BT, GATHER, PAIR>;
    if (PAIR) {
        a.NT = (a.NT1 + 1) / 2;
        const long long tiles = ((long long)(a.M_alloc + BT - 1) / BT + a.G) * a.NT;
        const int pairs = (int)std::min<long long>(maxp, tiles);
        return launch_k_pairs(kern, dim3(2 * pairs), dim3(C::THREADS), (size_t)C::SMEM_BYTES, st, pdl, ta, tw, a);
    }
    a.NT = a.NT1;
    const long long tiles = ((long long)(a.M_alloc + BT - 1) / BT + a.G) * a.NT;
    const int grid = (int)std::min<long long>(num_sms(), tiles);
    return launch_k(kern, dim3(grid), dim3(C::THREADS), (size_t)C::SMEM_BYTES, st, pdl, ta, tw, a);
}

template <int BT, bool PAIR = false>
cudaError_t run_mxf4_bt(const Mxf4Problem& p, const CUtensorMap& tw, const Mxf4Args& a, int maxp, cudaStream_t st, bool pdl) {
    CUtensorMap ta;
    if (!make_map_u8(&ta, p.a_codes, (uint64_t)p.K / 2, p.a_rows, p.K / 2, kStageK / 2, PAIR ? BT / 2 : BT,
                     CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    return p.row_idx ? run_mxf4<BT, !PAIR, PAIR>(ta, tw, a, maxp, st, pdl) : run_mxf4<BT, false, PAIR>(ta, tw, a, maxp, st, pdl);
}

// The rows that row_idx names, copied into segment order, a warp to a row: a product in tiles of 64 tokens
// and more gains more from rows in order than the copy takes, which is about 3 us (8192 rows x 4096 into
// 14336: 239 us on pairs, 266 in 128-token tiles of one SM, 368 when those gather. 128 experts x 2880 x 2880
// with 64 rows each 106 and 138, with 32 rows 103 and 102, with 8 rows 100 and 94). Rows behind the
// segments are left out: their row_idx may be anything.
__global__ void __launch_bounds__(256) gather_mxfp4_rows_kernel(const uint8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, int a_rows,
                                                                const int32_t* __restrict__ row_idx,
                                                                const int32_t* __restrict__ cu, int G, int M, int K,
                                                                uint8_t* codes_out, uint8_t* scales_out, DevError* err) {
    pdl_wait();
    const int lane = lane_id();
    const long long r = (long long)blockIdx.x * 8 + warp_id();
    int end = 0;
    for (int g = lane; g < G; g += 32) end = max(end, cu[g]);
    end = min(__reduce_max_sync(0xffffffffu, end), M);
    if (r < end) {
        const int v = row_idx[r];
        const bool ok = v >= 0 && v < a_rows;
        if (!ok && lane == 0) report_error(err, MOE_ERR_DEVICE, (int)r);  // counts as a row of zeros
        const int nc = K / 32;  // 16 codes bytes and one scale byte per 32 values
        const uint4* s = reinterpret_cast<const uint4*>(codes) + (size_t)(ok ? v : 0) * nc;
        uint4* d = reinterpret_cast<uint4*>(codes_out) + (size_t)r * nc;
        const uint8_t* ss = scales + (size_t)(ok ? v : 0) * nc;
        uint8_t* ds = scales_out + (size_t)r * nc;
#pragma unroll 4
        for (int i = lane; i < nc; i += 32) {
            d[i] = ok ? __ldg(s + i) : make_uint4(0u, 0u, 0u, 0u);
            ds[i] = ok ? __ldg(ss + i) : (uint8_t)0;
        }
    }
    pdl_launch();
}

}  // namespace

// Token tile: a tile costs a stage per 256 K whatever its width, so it should hold a whole segment;
// mean + 2 sqrt(mean) covers nearly every one. Longer segments go to CTA pairs, where there is a
// tile for each pair of SMs: 8 experts x 14336 x 4096 with 1024 rows each took 239 us on pairs and 266 in
// 128-token tiles (in runs of 2 s, at the power limit, 275 and 308), with 128 rows 57 and 55, with 64 rows 54
// and, in 64-token tiles, 50. The mean alone decides: with half of 16384 rows on one of 32 experts 2880 x 2880
// took 112 us, with as many rows on each 107.
// MOE_TOKEN_TILE=16|32|64|128 and MOE_GEMM_PAIRS=0|1 override the choice (tests, tuning).
// Returns 16, 32, 64 or 128, or, where rows are in segment order or can be brought into it, kPairTile.
int gemm_mxf4_tile(int G, int N, int M_alloc, bool pairs) {
    const long long segs = std::max<long long>(1, std::min<long long>(G, M_alloc));
    const double avg = (double)M_alloc / (double)segs;
    const char* env = getenv("MOE_TOKEN_TILE");
    const int v = env ? atoi(env) : 0;
    const bool forced = v == 16 || v == 32 || v == 64 || v == 128;
    const double want = forced ? v : avg + 2.0 * std::sqrt(avg);
    const char* pe = getenv("MOE_GEMM_PAIRS");
    const int mode = pe && (pe[0] == '0' || pe[0] == '1') && pe[1] == '\0' ? pe[0] - '0' : 2;
    const int nt1 = (N + kTileN - 1) / kTileN;
    const long long pair_tiles = ((long long)M_alloc + kPairTile - 1) / kPairTile * ((nt1 + 1) / 2);
    if (pairs && (mode == 1 || (mode == 2 && want > 128 && pair_tiles >= num_sms() / 2))) return kPairTile;
    return want <= 16 ? 16 : want <= 32 ? 32 : want <= 64 ? 64 : 128;
}

size_t gemm_mxf4_rows_bytes(int tile, int K, int M_alloc) {
    return tile >= kOrderedTile ? (size_t)M_alloc * (K / 2 + K / 32) : 0;
}

cudaError_t launch_gemm_mxf4(const Mxf4Problem& problem, cudaStream_t st, bool pdl) {
    Mxf4Problem p = problem;
    int maxp = 0;
    const cudaError_t ready = device_setup(&maxp);
    if (ready != cudaSuccess) return ready;
    const int bt = p.tile == kPairTile && maxp < 1 ? 128 : p.tile;  // no clusters of two here: one SM a tile
    if (bt >= kOrderedTile && p.row_idx && p.rows) {
        uint8_t* codes = static_cast<uint8_t*>(p.rows);
        uint8_t* scales = codes + (size_t)p.M_alloc * (p.K / 2);
        const cudaError_t e = launch_k(gather_mxfp4_rows_kernel, dim3((p.M_alloc - 1) / 8 + 1), dim3(256), 0, st, pdl, p.a_codes,
                                       p.a_scales, p.a_rows, p.row_idx, p.cu_seqlens, p.G, p.M_alloc, p.K, codes, scales, p.err);
        if (e != cudaSuccess) return e;
        p.a_codes = codes;
        p.a_scales = scales;
        p.a_rows = p.M_alloc;
        p.row_idx = nullptr;
        pdl = true;
    }
    const int Kp = mx8_kpad(p.K);
    Mxf4Args a{};
    a.cu = p.cu_seqlens;
    a.G = p.G;
    a.N = p.N;
    a.K = p.K;
    a.KB = (p.K + kStageK - 1) / kStageK;
    a.NT1 = (p.N + kTileN - 1) / kTileN;
    a.M_alloc = p.M_alloc;
    a.out = static_cast<__nv_bfloat16*>(p.out);
    a.alpha = p.alpha;
    a.w_sf = static_cast<const uint8_t*>(p.kscale);
    a.KS = Kp / kMx8StageK;
    a.a_codes = p.a_codes;
    a.a_sf = p.a_scales;
    a.a_rows = p.a_rows;
    a.row_idx = p.row_idx;
    a.err = p.err;
    a.wait_limit = wait_limit_cycles();
    l2_policies(&a.l2_w, &a.l2_t);
    CUtensorMap tw;
    if (!make_map_codes(&tw, p.kdata, (uint64_t)Kp / 2, p.N, p.G)) return cudaErrorInvalidValue;
    if (bt == kPairTile) return run_mxf4_bt<kPairTile, true>(p, tw, a, maxp, st, pdl);
    if (bt == 16) return run_mxf4_bt<16>(p, tw, a, maxp, st, pdl);
    if (bt == 32) return run_mxf4_bt<32>(p, tw, a, maxp, st, pdl);
    if (bt == 64) return run_mxf4_bt<64>(p, tw, a, maxp, st, pdl);
    return run_mxf4_bt<128>(p, tw, a, maxp, st, pdl);
}

}  // namespace moe
