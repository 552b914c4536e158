// S3/S5 — the grouped GEMM of MXFP4 activations and MXFP4 weights (W4A4).
//
//   out[r, n] = alpha_g * sum_k a[i(r), k] * W[g][n, k],   i(r) = row_idx[r] or r,
//
// both operands e2m1 with one e8m0 scale per 32 values along K, on the block-scaled tensor-core
// instruction kind::mxf4 (K = 64 per instruction, two scales per row). Products and scales are
// exact; the sum is fp32. Tiling as in the other grouped GEMMs ("swap AB"): a tile is 128 weight
// rows (M) by up to BT token rows (N) of one segment, the MMA as wide as the tile's rows.
//
// A pipeline stage is 256 values of K: 128 bytes of packed codes per row on either side, loaded by
// TMA with the 128-byte swizzle (the token rows by a gather of four rows per copy when row_idx is
// given), and the stage's scales as 512-byte blocks in tensor-memory copy order. The weights' are
// prepared so; the tokens' [rows, K/32] bytes may sit at any alignment, which no TMA copy takes, so
// scale warps load them a stage of their own ahead, through registers.
//
// Warp roles: 0 producer, 1 MMA issuer, 2..5 epilogue, then the scale warps, which also issue the
// copies of both sides' scales into the stage's tensor-memory slot. Waits are bounded as in the
// other GEMMs.
#include <cmath>

#include "gemm_common.cuh"

namespace moe {

namespace {

constexpr int kStageK = 256;
constexpr int kScaleWarps = 4;

struct Mxf4Args {
    const int32_t* cu;
    int G, N, K, KB, NT, M_alloc;
    __nv_bfloat16* out;
    const float* alpha;
    const uint8_t* w_sf;     // [G, NT, KS] blocks of 512 bytes, KS = blocks of 128 values
    int KS;
    const uint8_t* a_sf;     // [a_rows, K/32]
    int a_rows;
    const int32_t* row_idx;
    DevError* err;
    long long wait_limit;
    int l2_w, l2_t;
};

template <int BT>
struct Mxf4Cfg {
    static constexpr int A_BYTES = kTileN * kStageK / 2;
    static constexpr int B_OFF = A_BYTES;
    static constexpr int B_BYTES = BT * kStageK / 2;
    static constexpr int SFA_OFF = B_OFF + B_BYTES;             // two 512-byte blocks
    static constexpr int RG = (BT + 127) / 128;                 // 128-row groups of the token side
    static constexpr int SFB_OFF = SFA_OFF + 1024;              // [128-K half][row group] blocks
    static constexpr int STAGE = round1024(SFB_OFF + 2 * RG * 512);
    static constexpr int SF_SLOT = 8 + 8 * RG;                  // TMEM columns of a stage's scales
    static constexpr int SF_BASE = 2 * BT;                      // after two accumulators
    static constexpr int STAGES = cmin(cmin(kMaxStages, kSmemBudget / STAGE), (512 - SF_BASE) / SF_SLOT);
    static constexpr int TMEM_COLS = tmem_cols_pow2(SF_BASE + STAGES * SF_SLOT);
    static constexpr int SCALE_WARP0 = 6;
    static constexpr int THREADS = (SCALE_WARP0 + kScaleWarps) * 32;
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE + kCtrlBytes;
    static_assert(BT % 16 == 0 && BT >= 16 && BT <= 240, "token tile");
    static_assert(STAGES >= 3 && SMEM_BYTES <= kSmemLimit && SF_BASE + STAGES * SF_SLOT <= 512, "MXFP4 GEMM config");
    static_assert(B_OFF % 1024 == 0 && SFA_OFF % 512 == 0, "operand alignment");
};

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

template <int BT, bool GATHER>
__global__ void __launch_bounds__(Mxf4Cfg<BT>::THREADS, 1)
    grouped_gemm_mxf4_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                             const Mxf4Args a) {
    using C = Mxf4Cfg<BT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    CtrlBlock* ctl = reinterpret_cast<CtrlBlock*>(smem + C::STAGES * C::STAGE);
    volatile int* abort_flag = &ctl->abort;
    Issued is;
    auto opA = [&](int s) { return smem + s * C::STAGE; };
    auto opB = [&](int s) { return smem + s * C::STAGE + C::B_OFF; };
    auto sfA = [&](int s) { return smem + s * C::STAGE + C::SFA_OFF; };
    auto sfB = [&](int s, int h, int rg) { return smem + s * C::STAGE + C::SFB_OFF + (h * C::RG + rg) * 512; };
    uint64_t* sf_full = ctl->raw_full;  // the scales of stage s are in tensor memory
    const int warp = warp_id(), lane = lane_id();
    const int G = a.G, NT = a.NT, KB = a.KB;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
            mbar_init(&sf_full[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl->tfull[b], 1);
            mbar_init(&ctl->tempty[b], 4);
        }
        for (int i = 0; i <= kScaleWarps; ++i) mbar_init(&ctl->drain[i], 1);
        ctl->abort = 0;
        fence_barrier_init();
    }
    if (threadIdx.x == 32) {
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_w);
    }
    if (warp == 1) {
        tmem_alloc(&ctl->tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    pdl_wait();
    if (warp == 0) build_segment_table<BT>(a, ctl, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch();
    const uint32_t tmem_base = ctl->tmem_slot;
    const int total = ctl->tpre[G];

    if (warp == 0) {
        // ---------------- producer: lane 0 the tiled copies, all lanes the gathered token rows
        const uint64_t pol_w = l2_policy(a.l2_w), pol_t = l2_policy(a.l2_t);
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int L = blockIdx.x; L < total && ok; L += gridDim.x) {
            int g, nt, row0, rows;
            decode_tile<BT>(L, ctl, G, NT, g, nt, row0, rows);
            const uint8_t* wsf = a.w_sf + ((size_t)g * NT + nt) * a.KS * 512;
            constexpr int Q = (BT / 4 + 31) / 32;  // gathers of four rows per lane
            int idx[Q][4];
            if (GATHER) {
#pragma unroll
                for (int q = 0; q < Q; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = (q * 32 + lane) * 4 + i;
                        int v = r < rows ? a.row_idx[row0 + r] : a.a_rows;
                        if (v < 0 || v > a.a_rows || (v == a.a_rows && r < rows)) {
                            report_error(a.err, MOE_ERR_DEVICE, row0 + r);
                            v = a.a_rows;  // past the last row: reads as zeros
                        }
                        idx[q][i] = v;
                    }
            }
            for (int kb = 0; kb < KB; ++kb) {
                if (!__all_sync(0xffffffffu, mbar_wait(&ctl->empty[s], ph ^ 1u, abort_flag, a.wait_limit))) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    const uint32_t sfn = min(1024, (a.KS - 2 * kb) * 512);
                    mbar_arrive_expect_tx(&ctl->full[s], C::A_BYTES + C::B_BYTES + sfn);
                    tma_load_3d_p(opA(s), &tm_w, &ctl->full[s], kb * (kStageK / 2), nt * kTileN, g, pol_w);
                    bulk_load_p(sfA(s), wsf + (size_t)kb * 1024, sfn, &ctl->full[s], pol_w);
                    if (!GATHER) tma_load_2d_p(opB(s), &tm_a, &ctl->full[s], kb * (kStageK / 2), row0, pol_t);
                    is.mask |= 1u << s;
                    is.par = (is.par & ~(1u << s)) | (ph << s);
                }
                __syncwarp();
                if (GATHER) {
#pragma unroll
                    for (int q = 0; q < Q; ++q)
                        if ((q * 32 + lane) * 4 < BT)
                            tma_gather4(opB(s) + (q * 32 + lane) * 512, &tm_a, &ctl->full[s], kb * (kStageK / 2),
                                        idx[q][0], idx[q][1], idx[q][2], idx[q][3]);
                }
                if (++s == C::STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!ok && lane == 0) {
            report_error(a.err, MOE_ERR_TIMEOUT, 1);
            ctl->abort = 1;
        }
    } else if (warp == 1) {
        if (lane == 0) {  // ---------------- MMAs
            int s = 0, b = 0;
            uint32_t ph = 0, bph = 0;
            bool ok = true;
            for (int L = blockIdx.x; L < total && ok; L += gridDim.x) {
                int g, nt, row0, rows;
                decode_tile<BT>(L, ctl, G, NT, g, nt, row0, rows);
                const int n_mma = (rows + 15) & ~15;
                if (!mbar_wait(&ctl->tempty[b], bph ^ 1u, abort_flag, a.wait_limit)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(b * BT);
                for (int kb = 0; kb < KB; ++kb) {
                    if (!mbar_wait(&ctl->full[s], ph, abort_flag, a.wait_limit) ||
                        !mbar_wait(&sf_full[s], ph, abort_flag, a.wait_limit)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sfa = tmem_base + (uint32_t)(C::SF_BASE + s * C::SF_SLOT), sfb = sfa + 8;
                    const int steps = min(4, (a.K - kb * kStageK + 63) >> 6);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j < steps) {
                            const uint32_t id = (uint32_t)(j & 1) * 2, at = id << 30;
                            mma_mxf4_ss(d, sw128_kmajor_desc(smem_u32(opA(s)) + 32 * j),
                                        sw128_kmajor_desc(smem_u32(opB(s)) + 32 * j), idesc_mxf4(kTileN, n_mma, id),
                                        (sfa + 4 * (j >> 1)) | at, (sfb + 4 * C::RG * (j >> 1)) | at, (kb | j) != 0);
                        }
                    }
                    is.tc = true;
                    mma_commit(&ctl->empty[s]);
                    if (++s == C::STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
                mma_commit(&ctl->tfull[b]);
                b ^= 1;
                if (b == 0) bph ^= 1u;
            }
            if (!ok) {
                report_error(a.err, MOE_ERR_TIMEOUT, 2);
                ctl->abort = 1;
            }
        }
    } else if (warp >= C::SCALE_WARP0) {
        // ---------------- scale warp i: the token scales of stages i, i + kScaleWarps, ...
        constexpr int NR = (BT + 31) / 32;  // rows per lane: lane, lane + 32, ...
        const int mine = warp - C::SCALE_WARP0;
        const int row_bytes = a.K / 32;
        int it = 0, s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int L = blockIdx.x; L < total && ok; L += gridDim.x) {
            int g, nt, row0, rows;
            decode_tile<BT>(L, ctl, G, NT, g, nt, row0, rows);
            const uint8_t* src[NR];
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int r = 32 * i + lane;
                src[i] = nullptr;
                if (r < rows) {
                    const int v = GATHER ? a.row_idx[row0 + r] : row0 + r;
                    if (v >= 0 && v < a.a_rows) src[i] = a.a_sf + (size_t)v * row_bytes;
                }
            }
            for (int kb = 0; kb < KB; ++kb, ++it) {
                if (it % kScaleWarps == mine) {
                    uint2 v[4 * C::RG];
#pragma unroll
                    for (int i = 0; i < 4 * C::RG; ++i) {
                        v[i] = make_uint2(0u, 0u);
                        if (i < NR && src[i < NR ? i : 0]) v[i] = load_scales8(src[i < NR ? i : 0] + kb * 8, row_bytes - kb * 8);
                    }
                    if (!__all_sync(0xffffffffu, mbar_wait(&ctl->empty[s], ph ^ 1u, abort_flag, a.wait_limit))) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int rg = 0; rg < C::RG; ++rg) {
                        reinterpret_cast<uint4*>(sfB(s, 0, rg))[lane] =
                            make_uint4(v[4 * rg].x, v[4 * rg + 1].x, v[4 * rg + 2].x, v[4 * rg + 3].x);
                        reinterpret_cast<uint4*>(sfB(s, 1, rg))[lane] =
                            make_uint4(v[4 * rg].y, v[4 * rg + 1].y, v[4 * rg + 2].y, v[4 * rg + 3].y);
                    }
                    fence_proxy_async_smem();  // the copies read these bytes through the async proxy
                    if (!__all_sync(0xffffffffu, mbar_wait(&ctl->full[s], ph, abort_flag, a.wait_limit))) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        tc_fence_after();
                        const uint32_t sfa = tmem_base + (uint32_t)(C::SF_BASE + s * C::SF_SLOT), sfb = sfa + 8;
                        const int halves = min(2, a.KS - 2 * kb);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (h < halves) {
                                tmem_cp_32x128b_x4(sfa + 4 * h, sf_block_desc(smem_u32(sfA(s)) + 512 * h));
#pragma unroll
                                for (int rg = 0; rg < C::RG; ++rg)
                                    tmem_cp_32x128b_x4(sfb + 4 * (h * C::RG + rg),
                                                       sf_block_desc(smem_u32(sfB(s, h, rg))));
                            }
                        }
                        mma_commit(&sf_full[s]);
                    }
                    is.tc = true;
                    __syncwarp();
                }
                if (++s == C::STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!ok && lane == 0) {
            report_error(a.err, MOE_ERR_TIMEOUT, 5);
            ctl->abort = 1;
        }
    } else {
        // ---------------- epilogue (warps 2..5): lane = weight row, columns = tokens
        const int q = warp & 3;
        int b = 0;
        uint32_t bph = 0;
        for (int L = blockIdx.x; L < total; L += gridDim.x) {
            int g, nt, row0, rows;
            decode_tile<BT>(L, ctl, G, NT, g, nt, row0, rows);
            if (!mbar_wait(&ctl->tfull[b], bph, abort_flag, a.wait_limit)) {
                if (lane == 0) report_error(a.err, MOE_ERR_TIMEOUT, 3);
                ctl->abort = 1;
                break;
            }
            tc_fence_after();
            const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * BT);
            const int n = nt * kTileN + q * 32 + lane;
            const float al = a.alpha ? a.alpha[g] : 1.0f;
            for (int c0 = 0; c0 < rows; c0 += 16) {
                uint32_t r[16];
                tmem_ld16(tb + c0, r);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (n < a.N && c0 + j < rows)
                        a.out[(size_t)(row0 + c0 + j) * a.N + n] = __float2bfloat16_rn(__uint_as_float(r[j]) * al);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->tempty[b]);
            b ^= 1;
            if (b == 0) bph ^= 1u;
        }
        // rows past the last segment are zero
        const int start = ctl->cu[G - 1];
        const long long n8 = (long long)(a.M_alloc - start) * (a.N / 8);
        uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)start * a.N);
        for (long long i = (long long)blockIdx.x * 128 + threadIdx.x - 64; i < n8; i += (long long)gridDim.x * 128)
            o[i] = make_uint4(0u, 0u, 0u, 0u);
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        drain_in_flight(is, ctl->full, C::STAGES,
                        lane != 0                  ? nullptr
                        : warp == 1                ? &ctl->drain[0]
                        : warp >= C::SCALE_WARP0 ? &ctl->drain[1 + warp - C::SCALE_WARP0]
                                                   : nullptr);
        tc_fence_before();
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::TMEM_COLS);
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

template <int BT, bool GATHER>
cudaError_t run_mxf4(const CUtensorMap& ta, const CUtensorMap& tw, const Mxf4Args& a, cudaStream_t st, bool pdl) {
    using C = Mxf4Cfg<BT>;
    auto kern = grouped_gemm_mxf4_kernel<BT, GATHER>;
    static int done[64] = {0};
    cudaError_t e = set_smem_once(kern, C::SMEM_BYTES, done);
    if (e != cudaSuccess) return e;
    const long long tiles = ((long long)(a.M_alloc + BT - 1) / BT + a.G) * a.NT;
    const int grid = (int)std::min<long long>(num_sms(), tiles);
    return launch_k(kern, dim3(grid), dim3(C::THREADS), (size_t)C::SMEM_BYTES, st, pdl, ta, tw, a);
}

template <int BT>
cudaError_t run_mxf4_bt(const Mxf4Problem& p, const CUtensorMap& tw, const Mxf4Args& a, cudaStream_t st, bool pdl) {
    CUtensorMap ta;
    if (!make_map_u8(&ta, p.a_codes, (uint64_t)p.K / 2, p.a_rows, p.K / 2, kStageK / 2, p.row_idx ? 1 : BT,
                     CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    return p.row_idx ? run_mxf4<BT, true>(ta, tw, a, st, pdl) : run_mxf4<BT, false>(ta, tw, a, st, pdl);
}

}  // namespace

cudaError_t launch_gemm_mxf4(const Mxf4Problem& p, cudaStream_t st, bool pdl) {
    const int Kp = mx8_kpad(p.K);
    Mxf4Args a{};
    a.cu = p.cu_seqlens;
    a.G = p.G;
    a.N = p.N;
    a.K = p.K;
    a.KB = (p.K + kStageK - 1) / kStageK;
    a.NT = (p.N + kTileN - 1) / kTileN;
    a.M_alloc = p.M_alloc;
    a.out = static_cast<__nv_bfloat16*>(p.out);
    a.alpha = p.alpha;
    a.w_sf = static_cast<const uint8_t*>(p.kscale);
    a.KS = Kp / kMx8StageK;
    a.a_sf = p.a_scales;
    a.a_rows = p.a_rows;
    a.row_idx = p.row_idx;
    a.err = p.err;
    a.wait_limit = wait_limit_cycles();
    l2_policies(&a.l2_w, &a.l2_t);
    CUtensorMap tw;
    if (!make_map_codes(&tw, p.kdata, (uint64_t)Kp / 2, p.N, p.G)) return cudaErrorInvalidValue;
    const long long segs = std::max<long long>(1, std::min<long long>(p.G, p.M_alloc));
    const double avg = (double)p.M_alloc / (double)segs;
    // MOE_TOKEN_TILE=16|32|64|128|192 overrides the token-tile choice (tests, tuning)
    const char* env = getenv("MOE_TOKEN_TILE");
    const int v = env ? atoi(env) : 0;
    const double want = v == 16 || v == 32 || v == 64 || v == 128 || v == 192 ? v : avg + 2.0 * std::sqrt(avg);
    if (want <= 16) return run_mxf4_bt<16>(p, tw, a, st, pdl);
    if (want <= 32) return run_mxf4_bt<32>(p, tw, a, st, pdl);
    if (want <= 64) return run_mxf4_bt<64>(p, tw, a, st, pdl);
    if (want <= 128) return run_mxf4_bt<128>(p, tw, a, st, pdl);
    return run_mxf4_bt<192>(p, tw, a, st, pdl);
}

}  // namespace moe
