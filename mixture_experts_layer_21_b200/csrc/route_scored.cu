// S1 routing by scores: softmax or sigmoid scores s, a selection bias (c = s + bias), groups kept
// by their best or two best c, the top-k of c in the kept groups, weights from s, renormalised or
// raw. One warp per token; lane l holds experts l, l + 32, ...
//
// A masked expert (logit -inf or NaN) has s = 0 and ranks below every live one of the kept
// groups, by id among its like, so that the ids a row gets are always valid and distinct.
#include "internal.h"

namespace moe {

namespace {

constexpr int kNone = 0x7fffffff;

template <bool BF16>
MOE_DEV float load_logit(const void* row, int e) {
    if (BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(row)[e]);
    return static_cast<const float*>(row)[e];
}

// One token with every decision in fp64.
template <int EPL>
__device__ void route_exact(const RouteScored& a, const float (&l)[EPL], int t) {
    const double ninf = -(double)INFINITY;
    const int lane = lane_id(), E = a.E, gs = E / a.n_group;
    double s[EPL], c[EPL];
    if (a.scoring == MOE_SCORE_SOFTMAX) {
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) mx = fmaxf(mx, l[i]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            // the largest logit's term is 1 whether it is finite or +inf
            s[i] = l[i] == -INFINITY ? 0.0 : l[i] == mx ? 1.0 : exp((double)l[i] - (double)mx);
            sum += s[i];
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
#pragma unroll
        for (int i = 0; i < EPL; ++i) s[i] = sum > 0.0 ? s[i] / sum : 0.0;
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) s[i] = l[i] == -INFINITY ? 0.0 : 1.0 / (1.0 + exp(-(double)l[i]));
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = i * 32 + lane;
        c[i] = ninf;
        if (e < E && l[i] != -INFINITY) c[i] = s[i] + (a.bias ? (double)a.bias[e] : 0.0);
    }
    uint32_t taken = 0;  // bit i: entry i of this lane is chosen, absent or outside the kept groups
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (i * 32 + lane >= E) taken |= 1u << i;
    if (a.topk_group < a.n_group) {
        // each group's two largest c (or, ranked by its best expert without a bias, its largest
        // logit); lane g keeps group g's score
        const bool by_logit = a.group_score == MOE_GROUP_MAX && !a.bias;
        double my_gs = ninf;
        for (int g = 0; g < a.n_group; ++g) {
            double a1 = ninf, a2 = ninf;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = i * 32 + lane;
                if (e < E && e / gs == g) {
                    const double v = by_logit ? (double)l[i] : c[i];
                    a2 = fmax(a2, fmin(a1, v));
                    a1 = fmax(a1, v);
                }
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                const double b1 = __shfl_xor_sync(0xffffffffu, a1, off);
                const double b2 = __shfl_xor_sync(0xffffffffu, a2, off);
                a2 = fmax(fmin(a1, b1), fmax(a2, b2));
                a1 = fmax(a1, b1);
            }
            if (lane == g) my_gs = a1 + (a.group_score == MOE_GROUP_TOP2 && a2 != ninf ? a2 : 0.0);
        }
        uint32_t keep = 0;
        for (int j = 0; j < a.topk_group; ++j) {
            double bv = my_gs;
            int bg = (lane < a.n_group && !(keep >> lane & 1u)) ? lane : kNone;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                const double ov = __shfl_xor_sync(0xffffffffu, bv, off);
                const int og = __shfl_xor_sync(0xffffffffu, bg, off);
                if (og != kNone && (bg == kNone || ov > bv || (ov == bv && og < bg))) {
                    bv = ov;
                    bg = og;
                }
            }
            keep |= 1u << bg;  // bg is valid: topk_group <= n_group
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = i * 32 + lane;
            if (e < E && !(keep >> (e / gs) & 1u)) taken |= 1u << i;
        }
    }
    double my_s = 0.0;
    int my_id = 0;
    for (int j = 0; j < a.topk; ++j) {
        double bv = 0.0, bs = 0.0;
        int bid = kNone;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const double v = a.bias ? c[i] : (double)l[i];
            if (!(taken >> i & 1u) && (bid == kNone || v > bv)) {
                bv = v;
                bs = s[i];
                bid = i * 32 + lane;
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const double ov = __shfl_xor_sync(0xffffffffu, bv, off);
            const double os = __shfl_xor_sync(0xffffffffu, bs, off);
            const int oid = __shfl_xor_sync(0xffffffffu, bid, off);
            if (oid != kNone && (bid == kNone || ov > bv || (ov == bv && oid < bid))) {
                bv = ov;
                bs = os;
                bid = oid;
            }
        }
        // bid is valid: the kept groups hold at least topk experts
        if ((bid & 31) == lane) taken |= 1u << (bid >> 5);
        if (lane == j) {
            my_s = bs;
            my_id = bid;
        }
    }
    double sum = lane < a.topk ? my_s : 0.0;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane < a.topk) {
        const double w = a.renorm ? (sum > 0.0 ? my_s / sum : 0.0) : my_s;
        a.ids[(size_t)t * a.topk + lane] = my_id;
        a.w[(size_t)t * a.topk + lane] = (float)((double)a.scale * w);
    }
}

template <int EPL, bool BF16>
__global__ void __launch_bounds__(128) route_scored_kernel(const RouteScored a) {
    pdl_wait();
    const int t = blockIdx.x * (blockDim.x >> 5) + warp_id();
    if (t < a.T) {
        const void* row = static_cast<const char*>(a.logits) + (size_t)t * a.stride * (BF16 ? 2 : 4);
        float l[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = i * 32 + lane_id();
            l[i] = e < a.E ? load_logit<BF16>(row, e) : -INFINITY;
            if (isnan(l[i])) l[i] = -INFINITY;
        }
        route_exact<EPL>(a, l, t);
    }
    pdl_launch();
}

template <int EPL>
cudaError_t run_route(const RouteScored& r, cudaStream_t st, bool pdl) {
    const dim3 grid((r.T + 3) / 4), block(128);
    if (r.bf16) return launch_k(route_scored_kernel<EPL, true>, grid, block, 0, st, pdl, r);
    return launch_k(route_scored_kernel<EPL, false>, grid, block, 0, st, pdl, r);
}

}  // namespace

cudaError_t launch_route_scored(const RouteScored& r, cudaStream_t st, bool pdl) {
    const int epl = (r.E + 31) / 32;
    if (epl <= 1) return run_route<1>(r, st, pdl);
    if (epl <= 2) return run_route<2>(r, st, pdl);
    if (epl <= 4) return run_route<4>(r, st, pdl);
    if (epl <= 8) return run_route<8>(r, st, pdl);
    if (epl <= 16) return run_route<16>(r, st, pdl);
    return run_route<32>(r, st, pdl);
}

}  // namespace moe
