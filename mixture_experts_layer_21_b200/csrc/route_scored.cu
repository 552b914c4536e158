// S1 routing by scores: softmax or sigmoid scores s, a selection bias (c = s + bias), groups kept
// by their best or two best c, the top-k of c in the kept groups, weights from s, renormalised or
// raw. One warp per token; lane l holds the experts l EPL .. l EPL + EPL - 1, so that a lower lane
// has lower ids, a group of a multiple of EPL experts has lanes of its own, and a lane's logits
// are one wide load.
//
// A masked expert (logit -inf or NaN) has s = 0 and ranks below every live one of the kept
// groups, by id among its like, so that the ids a row gets are always valid and distinct.
//
// The decisions are those of fp64. The scores are computed in fp32 first, with a bound on their
// error, and where every comparison that decides is wider than it (but for a token in some
// hundreds), that is the answer; else fp64 decides among the candidates that are too close. In fp64
// throughout 16384 tokens x 256 experts in 8 groups took 158 us.
#include "internal.h"

namespace moe {

namespace {

constexpr int kNone = 0x7fffffff;

template <bool BF16>
MOE_DEV float load_logit(const void* row, int e) {
    if (BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(row)[e]);
    return static_cast<const float*>(row)[e];
}

// ----------------------------------------------------------------- fp64
// What one warp needs of a token in fp64, from the logits in memory (in the cache by then). The
// functions are called for few tokens and stay out of line: the registers of their loops would cost
// the other tokens occupancy.
template <bool BF16>
struct Token64 {
    const moe_route_args_t& a;
    const void* row;
    float mx;     // softmax: the largest logit
    double norm;  // softmax: the sum of the scores' numerators

    MOE_DEV Token64(const moe_route_args_t& r, int t, float largest)
        : a(r), row(static_cast<const char*>(r.logits) + (size_t)t * r.row_stride * (BF16 ? 2 : 4)), mx(largest), norm(1.0) {}
    MOE_DEV float logit(int e) const {
        const float x = load_logit<BF16>(row, e);
        return isnan(x) ? -INFINITY : x;
    }
    // the score, softmax's without its denominator: the largest logit's is 1 whether it is finite or +inf
    MOE_DEV double part(float l) const {
        const double x = a.scoring == MOE_SCORE_SIGMOID ? -(double)l : l == mx ? 0.0 : (double)l - (double)mx;
        const double z = exp(x);
        return l == -INFINITY ? 0.0 : a.scoring == MOE_SCORE_SIGMOID ? 1.0 / (1.0 + z) : z;
    }
    MOE_DEV void set_norm(double sum) {  // sum: this lane's
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        norm = a.scoring == MOE_SCORE_SIGMOID || !(sum > 0.0) ? 1.0 : sum;
    }
    MOE_DEV double value(int e, float l, double p) const {  // c, -inf where masked
        return l == -INFINITY ? -(double)INFINITY : p / norm + (a.bias ? (double)a.bias[e] : 0.0);
    }
};

// c of every expert into c[E] (shared memory of the warp's own).
template <bool BF16>
__device__ __forceinline__ void values64(Token64<BF16>& k, double* c) {
    const int lane = lane_id(), E = k.a.E;
    double sum = 0.0;
    __syncwarp();
#pragma unroll 4
    for (int e = lane; e < E; e += 32) {
        const double p = k.part(k.logit(e));
        c[e] = p;
        sum += p;
    }
    k.set_norm(sum);
#pragma unroll 4
    for (int e = lane; e < E; e += 32) c[e] = k.value(e, k.logit(e), c[e]);
    __syncwarp();
}

// The kept groups of a token whose c are in c[E], as bits.
template <bool BF16>
__device__ __forceinline__ uint32_t keep64(const Token64<BF16>& k, const double* c) {
    const moe_route_args_t& a = k.a;
    const double ninf = -(double)INFINITY;
    // each group's largest c or the sum of its two largest (ranked by its best expert without a
    // bias, its largest logit): a power of two of lanes to a group, then lane g has group g's
    const bool by_logit = a.group_score == MOE_GROUP_MAX && !a.bias;
    const int lane = lane_id(), gs = a.E / a.n_group;
    const int lanes = 1 << (31 - __clz(32 / a.n_group)), g = lane / lanes;
    double a1 = ninf, a2 = ninf;
    if (g < a.n_group) {
#pragma unroll 4
        for (int e = g * gs + lane % lanes; e < (g + 1) * gs; e += lanes) {
            const double v = by_logit ? (double)k.logit(e) : c[e];
            a2 = fmax(a2, fmin(a1, v));
            a1 = fmax(a1, v);
        }
    }
    for (int off = 1; off < lanes; off <<= 1) {
        const double b1 = __shfl_xor_sync(0xffffffffu, a1, off), b2 = __shfl_xor_sync(0xffffffffu, a2, off);
        a2 = fmax(fmin(a1, b1), fmax(a2, b2));
        a1 = fmax(a1, b1);
    }
    const double my = __shfl_sync(0xffffffffu, a1 + (a.group_score == MOE_GROUP_TOP2 && a2 != ninf ? a2 : 0.0),
                                  min(lane * lanes, 31));
    int rank = 0;  // how many groups come before this lane's
    for (int h = 0; h < a.n_group; ++h) {
        const double o = __shfl_sync(0xffffffffu, my, h);
        rank += o > my || (o == my && h < lane);
    }
    return __ballot_sync(0xffffffffu, lane < a.n_group && rank < a.topk_group);
}

// The kept groups alone.
template <bool BF16>
__device__ __noinline__ uint32_t groups64(const moe_route_args_t& a, int t, float mx, double* c) {
    Token64<BF16> k(a, t, mx);
    values64(k, c);
    return keep64(k, c);
}

// The topk best of `count` <= 32 candidates, lane i's being expert id: lane j gets the j-th.
template <bool BF16>
__device__ __noinline__ int order64(const moe_route_args_t& a, int t, float mx, int id, int count) {
    const int lane = lane_id();
    Token64<BF16> k(a, t, mx);
    if (a.scoring == MOE_SCORE_SOFTMAX) {
        double sum = 0.0;
#pragma unroll 4
        for (int e = lane; e < a.E; e += 32) sum += k.part(k.logit(e));
        k.set_norm(sum);
    }
    double c = 0.0;
    if (lane < count) {
        const float l = k.logit(id);
        c = k.value(id, l, k.part(l));
    }
    int rank = 0, best = 0;
    for (int h = 0; h < count; ++h) {
        const double o = __shfl_sync(0xffffffffu, c, h);
        const int oid = __shfl_sync(0xffffffffu, id, h);
        rank += o > c || (o == c && oid < id);
    }
    for (int h = 0; h < count; ++h) {
        const int r = __shfl_sync(0xffffffffu, rank, h), oid = __shfl_sync(0xffffffffu, id, h);
        if (r == lane) best = oid;
    }
    return best;
}

// A whole token.
template <bool BF16>
__device__ __noinline__ void route64(const moe_route_args_t& a, int t, double* c) {
    const int lane = lane_id(), E = a.E, gs = E / a.n_group;
    Token64<BF16> k(a, t, -INFINITY);
    if (a.scoring == MOE_SCORE_SOFTMAX) {
        for (int e = lane; e < E; e += 32) k.mx = fmaxf(k.mx, k.logit(e));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) k.mx = fmaxf(k.mx, __shfl_xor_sync(0xffffffffu, k.mx, off));
    }
    values64(k, c);
    const bool groups = a.topk_group < a.n_group;
    const uint32_t keep = groups ? keep64(k, c) : 1u;
    __syncwarp();
    // what ranks the experts: c, or without a bias the logits; NaN where taken or outside the kept groups
    const double gone = __longlong_as_double(0x7ff8000000000000LL);
    for (int e = lane; e < E; e += 32) {
        if (!a.bias) c[e] = (double)k.logit(e);
        if (!(keep >> (groups ? e / gs : 0) & 1u)) c[e] = gone;
    }
    __syncwarp();
    int my_id = 0;
    for (int j = 0; j < a.topk; ++j) {
        double bv = 0.0;
        int bid = kNone;
#pragma unroll 8
        for (int e = lane; e < E; e += 32) {
            const double v = c[e];
            if (!isnan(v) && (bid == kNone || v > bv)) {
                bv = v;
                bid = e;
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const double ov = __shfl_xor_sync(0xffffffffu, bv, off);
            const int oid = __shfl_xor_sync(0xffffffffu, bid, off);
            if (oid != kNone && (bid == kNone || ov > bv || (ov == bv && oid < bid))) {
                bv = ov;
                bid = oid;
            }
        }
        // bid is valid: the kept groups hold at least topk experts
        if (lane == j) my_id = bid;
        if ((bid & 31) == lane) c[bid] = gone;
        __syncwarp();
    }
    double w = lane < a.topk ? k.part(k.logit(my_id)) / k.norm : 0.0;
    if (a.renormalize) {
        double tot = w;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, off);
        w = tot > 0.0 ? w / tot : 0.0;
    }
    if (lane < a.topk) {
        a.topk_ids[(size_t)t * a.topk + lane] = my_id;
        a.topk_w[(size_t)t * a.topk + lane] = (float)((double)a.routed_scaling_factor * w);
    }
}

// ----------------------------------------------------------------- fp32
// The order of floats as unsigned integers; 0 is below -inf.
MOE_DEV uint32_t order_key(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);  // -0 as +0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
MOE_DEV float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

// The largest key of an array, by a tree.
template <int N>
MOE_DEV uint32_t key_max(const uint32_t (&k)[N]) {
    uint32_t m[N];
#pragma unroll
    for (int i = 0; i < N; ++i) m[i] = k[i];
#pragma unroll
    for (int w = N / 2; w > 0; w >>= 1)
#pragma unroll
        for (int i = 0; i < w; ++i) m[i] = max(m[i], m[i + w]);
    return m[0];
}

// One token, in fp32 where that decides. False where it cannot (infinite logits, more than 32
// candidates within the error of each other); nothing is written then.
//
// Error of the scores. expf is within 2 units in the last place. Sigmoid: the sum 1 + e rounds once
// and __fdividef is within 2 units, so s <= 1 is within 4 * 2^-23 = 2^-21. Softmax: the argument l - max rounds,
// which moves e^(l - max) by at most 2^-25, and the sum of up to 1024 terms, a chain of 32 in a lane
// and 5 across, is within 37 * 2^-24: s is within 2^-18 of itself and 2^-22 of the largest. Adding the
// bias rounds once more, 2^-24 |c|. Two values compare as their exact ones do if they differ by more
// than twice the sum of both bounds (the factor of two is to spare): the slacks below. Logits compare exactly.
template <int EPL, bool BF16, bool GROUPS>
__device__ bool route_fast(const moe_route_args_t& a, const float (&l)[EPL], int t, const void* row, double* c64) {
    const int lane = lane_id(), E = a.E;
    const bool softmax = a.scoring == MOE_SCORE_SOFTMAX;
    float mx = 0.0f, inv = 1.0f, s[EPL];
    if (softmax) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) m = fmaxf(m, l[i]);
        mx = key_value(__reduce_max_sync(0xffffffffu, order_key(m)));
        if (!(mx < INFINITY && mx > -INFINITY)) return false;  // +inf logits, or no live expert
    }
    // scores of every expert, where the selection, the groups or the raw softmax weights need them
    const bool top2 = GROUPS && a.group_score == MOE_GROUP_TOP2;
    if (a.bias || (softmax && !a.renormalize) || top2) {
        if (softmax) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                s[i] = expf(l[i] - mx);  // 0 where masked
                sum += s[i];
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            inv = 1.0f / sum;
#pragma unroll
            for (int i = 0; i < EPL; ++i) s[i] *= inv;
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) s[i] = __fdividef(1.0f, 1.0f + expf(-l[i]));
        }
    }
    // what ranks the experts, as order keys: c, or the logits; below them masked experts (-inf),
    // then, with key 0, those absent or outside the kept groups
    uint32_t key[EPL];
    float bmax = 0.0f;
    const int live = min(max(E - lane * EPL, 0), EPL);  // this lane's experts
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        float v = l[i];
        if (a.bias && i < live) {
            const float b = __ldg(a.bias + lane * EPL + i);
            bmax = fmaxf(bmax, fabsf(b));
            if (l[i] > -INFINITY) v = s[i] + b;
        }
        key[i] = i < live ? order_key(v) : 0u;
    }
    if (a.bias) bmax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(bmax)));
    if (GROUPS) {
        const int gs = E / a.n_group;
        // each group's two largest values; lane g keeps group g's score
        float my = -INFINITY;
        auto merge = [](float& a1, float& a2, float b1, float b2) {
            a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
            a1 = fmaxf(a1, b1);
        };
        auto value = [&](int i) {  // c (s without a bias), or the logit where the best expert's ranks the group
            if (top2 && !a.bias) return l[i] > -INFINITY ? s[i] : -INFINITY;
            return key_value(key[i]);
        };
        auto score = [&](float a1, float a2) { return a1 + (top2 && a2 > -INFINITY ? a2 : 0.0f); };
        const int lanes = gs / EPL;
        const bool runs = gs % EPL == 0 && (lanes & (lanes - 1)) == 0;  // a group is an aligned run of lanes
        if (runs) {
            float a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (i < live) merge(a1, a2, value(i), -INFINITY);
            for (int off = 1; off < lanes; off <<= 1) {
                const float b1 = __shfl_xor_sync(0xffffffffu, a1, off), b2 = __shfl_xor_sync(0xffffffffu, a2, off);
                merge(a1, a2, b1, b2);
            }
            my = __shfl_sync(0xffffffffu, score(a1, a2), min(lane * lanes, 31));
        } else {
            for (int g = 0; g < a.n_group; ++g) {
                float a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const int e = lane * EPL + i - g * gs;
                    if (e >= 0 && e < gs) merge(a1, a2, value(i), -INFINITY);
                }
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) {
                    const float b1 = __shfl_xor_sync(0xffffffffu, a1, off), b2 = __shfl_xor_sync(0xffffffffu, a2, off);
                    merge(a1, a2, b1, b2);
                }
                if (lane == g) my = score(a1, a2);
            }
        }
        int rank = 0;  // how many groups come before this lane's
        for (int h = 0; h < a.n_group; ++h) {
            const float o = __shfl_sync(0xffffffffu, my, h);
            rank += o > my || (o == my && h < lane);
        }
        const bool is = lane < a.n_group, kept = is && rank < a.topk_group;
        uint32_t keep = __ballot_sync(0xffffffffu, kept);
        if (top2 || a.bias) {  // the lowest kept against the highest dropped score: up to four c
            const float lo = key_value(__reduce_min_sync(0xffffffffu, kept ? order_key(my) : 0xffffffffu));
            const float hi = key_value(__reduce_max_sync(0xffffffffu, is && !kept ? order_key(my) : 0u));
            const float slack = (softmax ? 0x1p-17f * 2.0f + 0x1p-19f : 0x1p-20f * 4.0f) + 0x1p-22f * 4.0f * (1.0f + bmax);
            if (!(lo - hi > slack)) keep = groups64<BF16>(a, t, mx, c64);
        }
        if (runs) {
            const int g = lane / lanes;
            if (g < a.n_group && !(keep >> g & 1u)) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) key[i] = 0u;
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (i < live && !(keep >> ((lane * EPL + i) / gs) & 1u)) key[i] = 0u;
        }
    }
    // top-k: each lane's best, the warp's best, the lowest lane that has it, its lowest expert. With a
    // bias the candidates go on to those within the error of the last chosen, and where two
    // neighbours are that close, fp64 orders the candidates: any other expert is below topk of them.
    float prev = 0.0f, last = 0.0f;
    int my_id = 0, count = 0;
    bool close = false;
    for (int j = 0;; ++j) {
        if (j >= a.topk && !a.bias) break;
        const uint32_t best = key_max<EPL>(key);
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        if (top == 0u) break;  // none left; the kept groups hold at least topk experts
        if (a.bias) {
            const float c = key_value(top);
            auto near = [&](float hi) {  // masked experts (-inf) are behind every live one, in order of id
                if (!(c > -INFINITY)) return false;
                const float ac = fabsf(hi) + fabsf(c);
                const float sb = fminf(2.0f, ac + 2.0f * bmax);  // s_i + s_j <= |c_i| + |c_j| + |b_i| + |b_j|
                return !(hi - c > (softmax ? 0x1p-17f * sb + 0x1p-20f * inv : 0x1p-19f) + 0x1p-22f * ac);
            };
            if (j >= a.topk && !near(last)) break;
            if (j && near(prev)) close = true;
            prev = c;
            if (j < a.topk) last = c;
        }
        if (j == 32) return false;
        const int from = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
        int bi = 0;
#pragma unroll
        for (int i = EPL - 1; i >= 0; --i)
            if (key[i] == top) bi = i;
        const int id = __shfl_sync(0xffffffffu, bi, from) + from * EPL;
        if (lane == j) my_id = id;
        count = j + 1;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (lane == from && i == bi) key[i] = 0u;
    }
    if (close) my_id = order64<BF16>(a, t, mx, my_id, count);
    const bool mine = lane < a.topk;
    float w = 0.0f, arg = 0.0f;
    if (mine) {
        // the chosen logit once more (from the cache): its score with an exact division
        const float x = load_logit<BF16>(row, my_id);
        const bool off = isnan(x) || x == -INFINITY;
        arg = off ? 0.0f : softmax ? x - mx : x;
        w = off ? 0.0f : softmax ? expf(arg) * (a.renormalize ? 1.0f : inv) : 1.0f / (1.0f + expf(-arg));
    }
    // far from the largest (or from 0) fp32's exponential leaves its normal range
    if (__any_sync(0xffffffffu, arg < -80.0f)) return false;
    if (a.renormalize) {
        float tot = w;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, off);
        if (!(tot > 0.0f)) return false;
        w /= tot;
    }
    if (mine) {
        a.topk_ids[(size_t)t * a.topk + lane] = my_id;
        a.topk_w[(size_t)t * a.topk + lane] = a.routed_scaling_factor * w;
    }
    return true;
}

// This lane's EPL consecutive logits, by wide loads where the rows allow them (whole 16-byte pieces
// inside the row), NaN as -inf.
template <int EPL, bool BF16>
MOE_DEV void load_logits(const moe_route_args_t& a, const void* row, bool wide, float (&l)[EPL]) {
    constexpr int V = BF16 ? 8 : 4;  // values in 16 bytes
    const int e0 = lane_id() * EPL;
    if (EPL % V == 0 && wide) {
#pragma unroll
        for (int q = 0; q < EPL / V; ++q) {
            uint4 u = make_uint4(0, 0, 0, 0);
            const bool in = e0 + q * V < a.E;
            if (in) u = __ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(row) + (size_t)(e0 + q * V) * (BF16 ? 2 : 4)));
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (BF16) {
                    l[q * V + 2 * i % V] = in ? __uint_as_float(w[i] << 16) : -INFINITY;
                    l[q * V + (2 * i + 1) % V] = in ? __uint_as_float(w[i] & 0xffff0000u) : -INFINITY;
                } else {
                    l[q * V + i] = in ? __uint_as_float(w[i]) : -INFINITY;
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) l[i] = e0 + i < a.E ? load_logit<BF16>(row, e0 + i) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (isnan(l[i])) l[i] = -INFINITY;
}

template <int EPL, bool BF16, bool GROUPS>
__global__ void __launch_bounds__(128) route_scored_kernel(const moe_route_args_t a, bool wide) {
    extern __shared__ double warps_c64[];  // [warps][E], for tokens taken up in fp64
    pdl_wait();
    const int t = blockIdx.x * (blockDim.x >> 5) + warp_id();
    if (t < a.T) {
        const void* row = static_cast<const char*>(a.logits) + (size_t)t * a.row_stride * (BF16 ? 2 : 4);
        float l[EPL];
        load_logits<EPL, BF16>(a, row, wide, l);
        double* c64 = warps_c64 + warp_id() * a.E;
        if (!route_fast<EPL, BF16, GROUPS>(a, l, t, row, c64)) route64<BF16>(a, t, c64);
    }
    pdl_launch();
}

template <int EPL, bool BF16>
cudaError_t run_route(const moe_route_args_t& r, cudaStream_t st, bool pdl) {
    const dim3 grid((r.T + 3) / 4), block(128);
    const int bytes = BF16 ? 2 : 4;
    const size_t smem = 4 * sizeof(double) * r.E;  // at most 32 KB
    const bool wide = (reinterpret_cast<uintptr_t>(r.logits) & 15) == 0 && r.row_stride * bytes % 16 == 0 && r.E * bytes % 16 == 0;
    if (r.topk_group < r.n_group) return launch_k(route_scored_kernel<EPL, BF16, true>, grid, block, smem, st, pdl, r, wide);
    return launch_k(route_scored_kernel<EPL, BF16, false>, grid, block, smem, st, pdl, r, wide);
}

template <int EPL>
cudaError_t run_route(const moe_route_args_t& r, cudaStream_t st, bool pdl) {
    return r.in_is_bf16 ? run_route<EPL, true>(r, st, pdl) : run_route<EPL, false>(r, st, pdl);
}

}  // namespace

cudaError_t launch_route_scored(const moe_route_args_t& r, cudaStream_t st, bool pdl) {
    const int epl = (r.E + 31) / 32;
    if (epl <= 1) return run_route<1>(r, st, pdl);
    if (epl <= 2) return run_route<2>(r, st, pdl);
    if (epl <= 4) return run_route<4>(r, st, pdl);
    if (epl <= 8) return run_route<8>(r, st, pdl);
    if (epl <= 16) return run_route<16>(r, st, pdl);
    return run_route<32>(r, st, pdl);
}

}  // namespace moe
