// MXFP4 row quantisation, and the residual addition with root-mean-square norm whose rows come
// out in bf16 and/or quantised (MXFP8, MXFP4) for the experts.
//
// Both formats are OCP MX v1.0: per 32 values one e8m0 scale 2^e with e = floor(log2 amax) minus
// the exponent of the element type's largest value (8 for e4m3, 2 for e2m1), and every value
// rounded to nearest even after division by it. The division by a power of two is exact, so the
// codes do not depend on the arithmetic's precision. The largest magnitude is taken over the
// values' bits as integers: for fp32 that is the order of the magnitudes, its exponent field
// gives e without a logarithm, and infinities and NaN show as the largest values.
#include "internal.h"

namespace moe {

namespace {

// e8m0 byte of a block whose largest magnitude has these fp32 bits; 255 (NaN) for an infinity
// or NaN. A zero or subnormal maximum gives 0 (2^-127), the clamp's lower end.
template <int EMAX>
MOE_DEV uint32_t block_scale_byte(uint32_t maxbits) {
    if (maxbits >= 0x7f800000u) return 255u;
    return (uint32_t)max((int)(maxbits >> 23) - EMAX, 0);
}
// 2^(127 - s), the factor that divides by the scale; s <= 252 keeps it a normal number.
MOE_DEV float inv_scale(uint32_t s) { return __uint_as_float((254u - s) << 23); }
// 2^(s - 127); s = 0 is subnormal.
MOE_DEV float scale_value(uint32_t s) { return __uint_as_float(s ? s << 23 : 0x00400000u); }

MOE_DEV uint32_t cvt_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
MOE_DEV uint32_t cvt_e2m1_pair(float lo, float hi) {
    uint16_t r;
    asm("{ .reg .b8 t; cvt.rn.satfinite.e2m1x2.f32 t, %1, %2; cvt.u16.u8 %0, t; }" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
MOE_DEV float2 e4m3x2_values(uint32_t two) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<const __half2*>(&h2));
}
MOE_DEV float2 e2m1x2_values(uint32_t byte) {
    uint32_t h2;
    asm("{ .reg .b8 t; cvt.u8.u16 t, %1; cvt.rn.f16x2.e2m1x2 %0, t; }" : "=r"(h2) : "h"((uint16_t)byte));
    return __half22float2(*reinterpret_cast<const __half2*>(&h2));
}

MOE_DEV uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}
MOE_DEV uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
MOE_DEV void unpack8(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Eight consecutive values of a row from bf16 or fp32 memory.
template <bool F32>
MOE_DEV void load_chunk(const void* base, size_t off, float (&v)[8]) {
    if (F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
        const float4 a = p[0], b = p[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + off), v);
    }
}

// Quantises this lane's eight values; the four lanes 4i .. 4i+3 hold one 32-value block, and all
// lanes of the warp take part. c: index of the chunk of eight in the dense [rows, H] plane.
template <int Q>
MOE_DEV void quantize_chunk(const float (&v)[8], bool live, size_t c, uint8_t* codes, uint8_t* scales,
                            __nv_bfloat16* deq) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t s = block_scale_byte<Q == MOE_Q_MXFP8 ? 8 : 2>(m);
    const bool bad = s == 255u;
    const float inv = inv_scale(bad ? 127u : s);
    if (!live) return;
    if ((c & 3) == 0) scales[c >> 2] = (uint8_t)s;
    float d[8];
    if (Q == MOE_Q_MXFP8) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = bad ? 0x7f7fu : cvt_e4m3x2(v[2 * i] * inv, v[2 * i + 1] * inv);
            const float2 f = e4m3x2_values(w[i]);
            d[2 * i] = f.x;
            d[2 * i + 1] = f.y;
        }
        reinterpret_cast<uint2*>(codes)[c] = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = bad ? 0u : cvt_e2m1_pair(v[2 * i] * inv, v[2 * i + 1] * inv);
            const float2 f = e2m1x2_values(w[i]);
            d[2 * i] = f.x;
            d[2 * i + 1] = f.y;
        }
        reinterpret_cast<uint32_t*>(codes)[c] = w[0] | w[1] << 8 | w[2] << 16 | w[3] << 24;
    }
    if (deq) {
        const float sv = bad ? __uint_as_float(0x7fc00000u) : scale_value(s);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] *= sv;
        reinterpret_cast<uint4*>(deq)[c] = pack8(d);
    }
}

// Each thread takes kQuantUnroll chunks of eight values, a block's width apart, all loaded before the
// first is used. DENSE: the rows follow one another, and a chunk's place needs no division.
constexpr int kQuantUnroll = 4;
template <bool F32, bool DENSE>
__global__ void __launch_bounds__(256) quant_mxfp4_kernel(const void* in, long long stride, int R, int K, uint8_t* codes,
                                                          uint8_t* scales, __nv_bfloat16* deq) {
    pdl_wait();
    const int per_row = K / 8;
    const long long n = (long long)R * per_row;
    const long long c0 = (long long)blockIdx.x * (256 * kQuantUnroll) + threadIdx.x;
    float v[kQuantUnroll][8];
#pragma unroll
    for (int u = 0; u < kQuantUnroll; ++u) {
        const long long c = c0 + u * 256;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[u][j] = 0.0f;
        if (c < n) {
            size_t off = (size_t)c * 8;
            if (!DENSE) {
                const long long r = c / per_row;
                off = (size_t)r * stride + (size_t)(c - r * per_row) * 8;
            }
            load_chunk<F32>(in, off, v[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < kQuantUnroll; ++u) {
        const long long c = c0 + u * 256;
        quantize_chunk<MOE_Q_MXFP4>(v[u], c < n, (size_t)c, codes, scales, deq);
    }
    pdl_launch();
}

// 1 / sqrt(m), rounded once to fp32: fp32's value and one Newton step in fp64. The factor goes into
// every value of a row, and an error in it moves codes of the row across their rounding borders, all
// in one direction; with fp32 throughout 8192 rows of 7168 had twice the codes off that the two
// roundings of the products cost.
MOE_DEV float inv_sqrt(double m) {
    const float f = rsqrtf((float)m);
    const double r = (double)f;
    return f == 0.0f ? 0.0f : (float)(r * (1.5 - 0.5 * m * r * r));  // 0: an infinite m
}

// A block to a row (SHORT: a warp, blockDim.y of them to a block); thread t holds chunks t, t + blockDim.x of
// eight values in registers, so the row is read once. What bounds long inputs is the memory traffic in
// flight between the rows' barriers: the registers are held to 32 a thread, 2048 threads an SM (8192
// rows of 7168 with residual into bf16 and MXFP8: 90 us, 5.9 TB/s, on the same rows again and again, 95 on
// new ones; against the 90, with 34 registers, a block less, 97; with rows copied ahead into shared memory
// by blocks that walk over them 108).
template <int CPT, bool F32, int Q, bool SHORT>
__global__ void __launch_bounds__(1024, CPT <= 2 ? 2 : 1) add_rmsnorm_kernel(const moe_rmsnorm_args_t a) {
    __shared__ float part[32];
    pdl_wait();
    const size_t row = SHORT ? (size_t)blockIdx.x * blockDim.y + threadIdx.y : blockIdx.x;
    if (SHORT && row >= a.T) return;
    const int chunks = a.H / 8;
    const __nv_bfloat16* res = static_cast<const __nv_bfloat16*>(a.residual);
    __nv_bfloat16* res_out = static_cast<__nv_bfloat16*>(a.residual_out);
    float v[CPT][8];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
        if (c < chunks) {
            load_chunk<F32>(a.x, row * a.x_stride + (size_t)c * 8, v[i]);
            if (res) {
                float r[8];
                load_chunk<false>(res, row * a.residual_stride + (size_t)c * 8, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += r[j];
            }
            if (res_out) *reinterpret_cast<uint4*>(res_out + row * a.residual_out_stride + (size_t)c * 8) = pack8(v[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(v[i][j], v[i][j], sum);
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    double total = sum;
    if (!SHORT) {
        if (lane_id() == 0) part[warp_id()] = sum;
        __syncthreads();
        total = 0.0;
        for (int w = 0; w < (int)(blockDim.x >> 5); ++w) total += part[w];
    }
    const float rstd = inv_sqrt(total * (1.0 / a.H) + a.eps);
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        const bool live = c < chunks;
        float g[8] = {1, 1, 1, 1, 1, 1, 1, 1};
        if (live && a.weight) {
            if (a.weight_is_f32) load_chunk<true>(a.weight, (size_t)c * 8, g);
            else load_chunk<false>(a.weight, (size_t)c * 8, g);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * g[j];
        if (live && a.y)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.y) + row * a.y_stride + (size_t)c * 8) = pack8(v[i]);
        if (Q != MOE_Q_NONE)
            quantize_chunk<Q>(v[i], live, row * chunks + c, a.codes, a.scales, static_cast<__nv_bfloat16*>(a.deq));
    }
    pdl_launch();
}

template <int CPT, bool F32, bool SHORT = false>
cudaError_t run_rmsnorm(const moe_rmsnorm_args_t& a, dim3 grid, dim3 block, cudaStream_t st, bool pdl) {
    if (a.quant == MOE_Q_MXFP8) return launch_k(add_rmsnorm_kernel<CPT, F32, MOE_Q_MXFP8, SHORT>, grid, block, 0, st, pdl, a);
    if (a.quant == MOE_Q_MXFP4) return launch_k(add_rmsnorm_kernel<CPT, F32, MOE_Q_MXFP4, SHORT>, grid, block, 0, st, pdl, a);
    return launch_k(add_rmsnorm_kernel<CPT, F32, MOE_Q_NONE, SHORT>, grid, block, 0, st, pdl, a);
}

template <bool F32>
cudaError_t run_rmsnorm(const moe_rmsnorm_args_t& a, cudaStream_t st, bool pdl) {
    // Few rows: a row is spread as thin as it goes, for the shortest way through it. Many: two chunks
    // a thread; rows of up to 512 values go to a warp each, eight to a block (32768 rows of 256: 19 us,
    // a block to a row 39).
    const int chunks = a.H / 8;
    const bool many = a.T >= 2 * num_sms();
    if (many && chunks <= 64) return run_rmsnorm<2, F32, true>(a, dim3((a.T - 1) / 8 + 1), dim3(32, 8), st, pdl);
    const int cpt = chunks > 2048 ? 4 : many || chunks > 1024 ? 2 : 1;
    const dim3 grid(a.T), block(((chunks + cpt - 1) / cpt + 31) / 32 * 32);
    if (cpt == 1) return run_rmsnorm<1, F32>(a, grid, block, st, pdl);
    if (cpt == 2) return run_rmsnorm<2, F32>(a, grid, block, st, pdl);
    return run_rmsnorm<4, F32>(a, grid, block, st, pdl);
}

}  // namespace

cudaError_t launch_quant_mxfp4(const void* in, bool in_f32, long long stride, int R, int K, uint8_t* codes,
                               uint8_t* scales, void* deq, cudaStream_t st, bool pdl) {
    const long long n = (long long)R * (K / 8), per_block = 256 * kQuantUnroll;
    const long long blocks = (n + per_block - 1) / per_block;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    __nv_bfloat16* d = static_cast<__nv_bfloat16*>(deq);
    const dim3 grid((unsigned)blocks), block(256);
    const bool dense = stride == K || R == 1;
    if (in_f32) {
        if (dense) return launch_k(quant_mxfp4_kernel<true, true>, grid, block, 0, st, pdl, in, stride, R, K, codes, scales, d);
        return launch_k(quant_mxfp4_kernel<true, false>, grid, block, 0, st, pdl, in, stride, R, K, codes, scales, d);
    }
    if (dense) return launch_k(quant_mxfp4_kernel<false, true>, grid, block, 0, st, pdl, in, stride, R, K, codes, scales, d);
    return launch_k(quant_mxfp4_kernel<false, false>, grid, block, 0, st, pdl, in, stride, R, K, codes, scales, d);
}

cudaError_t launch_add_rmsnorm(const moe_rmsnorm_args_t& a, cudaStream_t st, bool pdl) {
    return a.x_is_f32 ? run_rmsnorm<true>(a, st, pdl) : run_rmsnorm<false>(a, st, pdl);
}

}  // namespace moe
