// S1 routing by scores: softmax or sigmoid scores s, a selection bias (c = s + bias), groups kept
// by their best or two best c, the top-k of c in the kept groups, weights from s, renormalised or
// raw. One warp per token; lane l holds the experts l EPL .. l EPL + EPL - 1, so that a lower lane
// has lower ids, a group of a multiple of EPL experts has lanes of its own, and a lane's logits
// are one wide load.
//
// A masked expert (logit -inf or NaN) has s = 0 and ranks below every live one of the kept
// groups, by id among its like, so that the ids a row gets are always valid and distinct. One
// whose bias is -inf or NaN ranks with them.
//
// The decisions are those of fp64. The scores are computed in fp32 first, with a bound on their
// error, and where every comparison that decides is wider than it (but for a token in some
// hundreds), that is the answer; else fp64 decides among the candidates that are too close. In fp64
// throughout 16384 tokens x 256 experts in 8 groups took 158 us. The weights of the chosen are formed in
// fp64 and rounded once.
#include <cfloat>

#include "internal.h"

namespace moe {

namespace {

constexpr int kNone = 0x7fffffff;

template <bool BF16>
MOE_DEV float load_logit(const void* row, int e) {
    if (BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(row)[e]);
    return static_cast<const float*>(row)[e];
}

MOE_DEV float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ----------------------------------------------------------------- fp64
// 1 / d for d > 0: fp32's reciprocal, within 2^-23, and one Newton step, r (2 - d r), which squares that:
// within 2^-45 (a division takes three times the instructions). Divided where fp32 does not hold d or 1 / d.
MOE_DEV double recip64(double d) {
    if (!(d > 0x1p-100 && d < 0x1p100)) return 1.0 / d;
    const double r = (double)rcp_approx((float)d);
    return fma(r, fma(-d, r, 1.0), r);
}

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
    MOE_DEV double expo(float l) const {
        return exp(a.scoring == MOE_SCORE_SIGMOID ? -(double)l : l == mx ? 0.0 : (double)l - (double)mx);
    }
    MOE_DEV double part(float l) const {
        const double z = expo(l);
        return l == -INFINITY ? 0.0 : a.scoring == MOE_SCORE_SIGMOID ? 1.0 / (1.0 + z) : z;
    }
    MOE_DEV double weight(float l) const {  // the score for the output, within 2^-44
        const double z = expo(l);
        return l == -INFINITY ? 0.0 : a.scoring == MOE_SCORE_SIGMOID ? recip64(1.0 + z) : z * recip64(norm);
    }
    MOE_DEV void set_norm(double sum) {  // sum: this lane's
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        norm = a.scoring == MOE_SCORE_SIGMOID || !(sum > 0.0) ? 1.0 : sum;
    }
    MOE_DEV double value(int e, float l, double p) const {  // c, -inf where masked; never NaN
        const float b = a.bias ? a.bias[e] : 0.0f;
        return l == -INFINITY || isnan(b) ? -(double)INFINITY : p / norm + (double)b;
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

// The sum of a softmax row's numerators.
template <bool BF16>
__device__ __noinline__ double norm64(const moe_route_args_t& a, int t, float mx) {
    Token64<BF16> k(a, t, mx);
    double sum = 0.0;
#pragma unroll 4
    for (int e = lane_id(); e < a.E; e += 32) sum += k.part(k.logit(e));
    k.set_norm(sum);
    return k.norm;
}

// Writes the choice, lane j's the j-th, with its weights.
template <bool BF16>
__device__ __forceinline__ void write64(const Token64<BF16>& k, int t, int my_id) {
    const moe_route_args_t& a = k.a;
    const int lane = lane_id();
    double w = lane < a.topk ? k.weight(k.logit(my_id)) : 0.0;
    if (a.renormalize) {
        double tot = w;
        for (int off = 1; off < a.topk; off <<= 1) tot += __shfl_xor_sync(0xffffffffu, tot, off);  // 0 from topk on
        w = tot > 0.0 ? w * recip64(tot) : 0.0;
    }
    if (lane < a.topk) {
        a.topk_ids[(size_t)t * a.topk + lane] = my_id;
        a.topk_w[(size_t)t * a.topk + lane] = (float)((double)a.routed_scaling_factor * w);
    }
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
    write64(k, t, my_id);
}

// ----------------------------------------------------------------- fp32
// The order of floats as unsigned integers; 0 is below -inf.
MOE_DEV uint32_t order_bits(float f) {
    const uint32_t u = __float_as_uint(f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
MOE_DEV uint32_t order_key(float f) { return order_bits(f + 0.0f); }  // -0 as +0
MOE_DEV float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

// Keys in descending order, by Batcher's odd-even merge sort (K. E. Batcher, Sorting networks and their
// applications, 1968); N a power of two.
template <int N>
MOE_DEV void sort_keys(uint32_t (&k)[N]) {
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const uint32_t hi = max(k[i + j], k[i + j + q]);
                        k[i + j + q] = min(k[i + j], k[i + j + q]);
                        k[i + j] = hi;
                    }
}

MOE_DEV float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// What the host works out once for the launch.
struct RoutePlan {
    bool wide;        // the rows' 16-byte pieces lie inside them and aligned
    bool wide_bias;   // and those of the bias, with E = 32 EPL
    int gs;           // experts to a group
    int lanes, shift; // GROUPS: a group is an aligned run of `lanes` = 2^shift lanes; lanes = 0: it is not
};

// One token, decided in fp32 where that decides. False where it cannot (infinite logits, more than 32
// candidates within the error of each other); nothing is written then. What bounds it is the number
// of instructions (with 256 experts in 8 groups 1090 a token, 28.8 us for 16384 tokens; 1046 and 27.0 with
// weights of fp32, 29.3 us with divisions in fp64; 1260 a token took 30 us, 1600 36).
//
// Error of the scores that rank. Sigmoid: the exponential's argument -l log2(e) rounds twice, 2^-23 |l|
// relative to the exponential e, whose approximation is within 2^-22; e / (1 + e)^2 <= 1/4 and |l| e / (1 + e)^2
// <= 0.23 bring that to 2^-23 in s; the sum rounds once and the reciprocal is within 2^-23: s is within 2^-21.
// Softmax: the argument (l - max) log2(e) rounds three times; |x| e^-|x| <= 0.37, so a term is within 2^-22 of
// the largest and, weighted by the terms, whose mean |x| is at most ln 1024 < 7, the sum within 13 * 2^-23,
// and 37 * 2^-24 for its additions, a chain of 32 in a lane and 5 across: s is within 2^-18 of itself and
// 2^-22 of the largest. Adding the bias rounds once more, 2^-24 |c|. Two values compare as their exact ones
// do if they differ by more than the sum of both bounds; the slacks below are twice that. They take the
// magnitudes of the values compared, not those of other experts: one that a bias of -1e9 switches off does
// not make the others close (with slacks from the largest |bias| it sent every token to fp64). Logits and
// infinite values compare exactly.
template <int EPL, bool BF16, bool GROUPS>
__device__ bool route_fast(const moe_route_args_t& a, const RoutePlan& plan, const float (&l)[EPL], int t,
                           double* c64) {
    constexpr float LOG2E = 1.44269504f;
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
    // raw softmax weights need the denominator in fp64 (renormalised, it cancels)
    Token64<BF16> k(a, t, mx);
    if (softmax && !a.renormalize) {
        if (EPL <= 8) {
            double sum = 0.0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) sum += k.part(l[i]);
            k.set_norm(sum);
        } else {
            k.norm = norm64<BF16>(a, t, mx);
        }
    }
    // scores of every expert, where the selection or the groups need them
    const bool top2 = GROUPS && a.group_score == MOE_GROUP_TOP2;
    auto approx = [&](float x) {  // softmax: without its denominator; 0 where masked
        return softmax ? exp2_approx((x - mx) * LOG2E) : rcp_approx(1.0f + exp2_approx(x * -LOG2E));
    };
    if (a.bias || top2) {
        if (softmax) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                s[i] = approx(l[i]);
                sum += s[i];
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            inv = 1.0f / sum;
#pragma unroll
            for (int i = 0; i < EPL; ++i) s[i] *= inv;
        } else if (a.bias) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) s[i] = approx(l[i]);
        }
    }
    // what ranks the experts, as order keys: c, or the logits; below them masked experts (-inf),
    // then, with key 0, those absent or outside the kept groups
    uint32_t key[EPL];
    float bmax = 0.0f;
    const int live = min(max(E - lane * EPL, 0), EPL);  // this lane's experts
    if (a.bias) {
        float b[EPL];
        if (EPL % 4 == 0 && plan.wide_bias) {
#pragma unroll
            for (int q = 0; q < EPL / 4; ++q) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(a.bias + lane * EPL) + q);
                b[4 * q] = f.x;
                b[4 * q + 1 % EPL] = f.y;
                b[4 * q + 2 % EPL] = f.z;
                b[4 * q + 3 % EPL] = f.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) b[i] = i < live ? __ldg(a.bias + lane * EPL + i) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if (softmax) bmax = fmaxf(bmax, fabsf(b[i]));
            const float c = s[i] + b[i];  // not -0: s is not
            key[i] = order_bits(l[i] > -INFINITY && c > -INFINITY ? c : -INFINITY);  // NaN as -inf
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = order_key(l[i]);
    }
    if (live < EPL) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (i >= live) key[i] = 0u;
    }
    if (a.bias && softmax) bmax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(bmax)));
    // A group's score from the two largest keys of c (of the logits without a bias, whose order is that of
    // s; where the best expert ranks the group, they are its score); mag: the sum of the magnitudes in it.
    constexpr uint32_t MASKED = 0x007fffffu;  // order_key(-INFINITY)
    auto score = [&](uint32_t a1, uint32_t a2, float& mag) {
        const float best = a1 ? key_value(a1) : -INFINITY;
        mag = fabsf(best);
        if (!top2 || a1 <= MASKED) return best;
        auto part = [&](float x) { return a.bias ? x : approx(x) * inv; };
        const float c1 = part(best), c2 = a2 <= MASKED ? 0.0f : part(key_value(a2));
        mag = fabsf(c1) + fabsf(c2);
        return c1 + c2;
    };
    auto merge = [](uint32_t& a1, uint32_t& a2, uint32_t b1, uint32_t b2) {
        a2 = max(min(a1, b1), max(a2, b2));
        a1 = max(a1, b1);
    };
    uint32_t* keys = reinterpret_cast<uint32_t*>(c64);  // [32][EPL]
    auto store_keys = [&] {
        __syncwarp();
        if (EPL % 4 == 0) {
#pragma unroll
            for (int i = 0; i + 3 < EPL; i += 4)
                reinterpret_cast<uint4*>(keys + lane * EPL)[i / 4] = make_uint4(key[i], key[i + 1], key[i + 2], key[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) keys[lane * EPL + i] = key[i];
        }
        __syncwarp();
    };
    if (GROUPS) {
        // each group's two largest keys from its lanes, or where a group has no lanes of its own out of
        // shared memory by `lanes` others, then lane g has group g's (16384 tokens x 160 experts in 8 groups:
        // 33 us; each group by the whole warp from the registers 53)
        const int gs = plan.gs;
        int lanes = plan.lanes;
        uint32_t a1 = 0u, a2 = 0u;
        if (lanes) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) merge(a1, a2, key[i], 0u);
        } else {
            lanes = 1 << (31 - __clz(32 / a.n_group));
            const int g = lane / lanes;
            store_keys();
            if (g < a.n_group)
                for (int e = g * gs + lane % lanes; e < (g + 1) * gs; e += lanes) merge(a1, a2, keys[e], 0u);
        }
        for (int off = 1; off < lanes; off <<= 1) {
            const uint32_t b1 = __shfl_xor_sync(0xffffffffu, a1, off), b2 = __shfl_xor_sync(0xffffffffu, a2, off);
            merge(a1, a2, b1, b2);
        }
        const int src = min(lane * lanes, 31);
        float mag;
        const float own = score(a1, a2, mag), my = __shfl_sync(0xffffffffu, own, src);
        int rank = 0;  // how many groups come before this lane's
        for (int h = 0; h < a.n_group; ++h) {
            const float o = __shfl_sync(0xffffffffu, my, h);
            rank += o > my || (o == my && h < lane);
        }
        const bool is = lane < a.n_group, kept = is && rank < a.topk_group;
        uint32_t keep = __ballot_sync(0xffffffffu, kept);
        if (top2 || a.bias) {  // the lowest kept score's lower end against the highest dropped one's upper end
            // a score's slack: of its s, up to two of them (softmax's sum to at most 1), and of the rounding of
            // its c and of their sum
            const float of_s = softmax ? 0x1p-17f + 0x1p-20f : 0x1p-19f;
            const float e = __shfl_sync(0xffffffffu, of_s + 0x1p-22f * fminf(mag, FLT_MAX), src);
            const float lo = key_value(__reduce_min_sync(0xffffffffu, kept ? order_key(my - e) : 0xffffffffu));
            const float hi = key_value(__reduce_max_sync(0xffffffffu, is && !kept ? order_key(my + e) : 0u));
            if (!(lo > hi)) keep = groups64<BF16>(a, t, mx, c64);
        }
        if (plan.lanes) {
            const int g = lane >> plan.shift;
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
    // Every lane sorts its keys. Which of its experts a key is, is looked up afterwards from the unsorted
    // keys in shared memory; of a lane's equal keys the n-th taken is the n-th in order of id.
    store_keys();
    sort_keys<EPL>(key);
    // Top-k: the warp takes the largest of the lanes' heads, the lowest lane's among equal ones, topk
    // times (the kept groups hold as many experts); lane j keeps the j-th. With a bias the candidates go
    // on to those within the error of the last chosen, and where two neighbours are that close, fp64
    // orders the candidates: any other expert is below topk of them.
    // The slack of two c. Softmax: s_i + s_j <= |c_i| + |c_j| + 2 bmax and at most twice the largest, inv;
    // sigmoid's s are at most 1. Masked experts (c = -inf) are behind every live one, in order of id.
    const bool by_c = softmax && bmax < inv;
    const float slack0 = softmax ? 0x1p-16f * fminf(bmax, inv) + 0x1p-20f * inv : 0x1p-19f;
    const float slack1 = by_c ? 0x1p-17f + 0x1p-22f : 0x1p-22f;
    auto near = [&](float hi, float c) {
        return fabsf(c) < INFINITY && !(hi - c > slack0 + slack1 * fminf(fabsf(hi) + fabsf(c), FLT_MAX));
    };
    uint32_t my_key = 0u, last = 0u;
    int my_from = 0, count = 0;
    for (;; ++count) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, key[0]);
        if (count < a.topk) last = top;
        else if (!a.bias || top == 0u || !near(key_value(last), key_value(top))) break;
        if (count == 32) return false;
        const int from = __ffs(__ballot_sync(0xffffffffu, key[0] == top)) - 1;
        if (lane == count) {
            my_key = top;
            my_from = from;
        }
        if (lane == from) {
#pragma unroll
            for (int i = 0; i + 1 < EPL; ++i) key[i] = key[i + 1];
            key[EPL - 1] = 0u;
        }
    }
    bool close = false;
    if (a.bias) {
        const float c = key_value(my_key), before = __shfl_up_sync(0xffffffffu, c, 1);
        close = __any_sync(0xffffffffu, lane > 0 && lane < count && near(before, c));
    }
    // a lane's equal keys are taken one after the other: lane j's is the n-th of its like
    const uint32_t key_before = __shfl_up_sync(0xffffffffu, my_key, 1);
    const int from_before = __shfl_up_sync(0xffffffffu, my_from, 1);
    const uint32_t firsts = __ballot_sync(0xffffffffu, lane == 0 || key_before != my_key || from_before != my_from);
    int n = __clz(firsts << (31 - lane));
    int my_id = 0;
    if (lane < count) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (keys[my_from * EPL + i] == my_key && n-- == 0) my_id = my_from * EPL + i;
    }
    if (close) my_id = order64<BF16>(a, t, mx, my_id, count);
    write64(k, t, my_id);
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
    for (int i = 0; i < EPL; ++i) l[i] = fmaxf(l[i], -INFINITY);
}

template <int EPL, bool BF16, bool GROUPS>
__global__ void __launch_bounds__(128, EPL <= 8 ? 8 : 4) route_scored_kernel(const moe_route_args_t a, const RoutePlan plan) {
    // [warps]: 32 EPL keys, or E values of a token taken up in fp64
    extern __shared__ __align__(16) double warps_c64[];
    pdl_wait();
    const int t = blockIdx.x * (blockDim.x >> 5) + warp_id();
    if (t < a.T) {
        const void* row = static_cast<const char*>(a.logits) + (size_t)t * a.row_stride * (BF16 ? 2 : 4);
        float l[EPL];
        load_logits<EPL, BF16>(a, row, plan.wide, l);
        double* c64 = warps_c64 + warp_id() * (32 * EPL);
        if (!route_fast<EPL, BF16, GROUPS>(a, plan, l, t, c64)) route64<BF16>(a, t, c64);
    }
    pdl_launch();
}

template <int EPL, bool BF16>
cudaError_t run_route(const moe_route_args_t& r, cudaStream_t st, bool pdl) {
    const dim3 grid((r.T - 1) / 4 + 1), block(128);
    const int bytes = BF16 ? 2 : 4;
    RoutePlan p{};
    p.wide = (reinterpret_cast<uintptr_t>(r.logits) & 15) == 0 && r.row_stride * bytes % 16 == 0 && r.E * bytes % 16 == 0;
    p.wide_bias = (reinterpret_cast<uintptr_t>(r.bias) & 15) == 0 && r.E == 32 * EPL;
    p.gs = r.E / r.n_group;
    if (p.gs % EPL == 0 && ((p.gs / EPL) & (p.gs / EPL - 1)) == 0) {
        p.lanes = p.gs / EPL;
        while ((1 << p.shift) < p.lanes) ++p.shift;
    }
    const size_t smem = 4 * sizeof(double) * 32 * EPL;  // at most 32 KB
    if (r.topk_group < r.n_group) return launch_k(route_scored_kernel<EPL, BF16, true>, grid, block, smem, st, pdl, r, p);
    return launch_k(route_scored_kernel<EPL, BF16, false>, grid, block, smem, st, pdl, r, p);
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
