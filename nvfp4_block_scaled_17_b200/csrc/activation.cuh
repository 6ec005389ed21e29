// activation.cuh -- the activations of the GEMM epilogues, in fp32, two values at a time.
//
//   relu       max(v, 0)
//   gelu       v * Phi(v), Phi the normal distribution function
//   gelu_tanh  v / 2 * (1 + tanh(sqrt(2 / pi) * (v + 0.044715 v^3)))
//   silu       v / (1 + exp(-v))
// A gated epilogue takes column pairs: u[j] = act(v[2j]) * v[2j + 1].
//
// The last three are all v * s(L(v)), s the logistic function: L = v for silu, an odd cubic
// for gelu_tanh ((1 + tanh z) / 2 = s(2 z)), and for gelu the logit of Phi, an odd function
// that a polynomial of degree 13 meets to 7e-8 in v * Phi(v).  An exponential and a reciprocal
// per value, the rest packed fp32x2 arithmetic.  Errors against 64-bit values, before the one
// rounding to bf16: below 5e-7 max(|v|, 1).
//
// Each value has a reciprocal of its own, of 1 + 2^t with t unbounded: far to the left the sum
// is infinite and the factor, with it the result, exactly 0; a NaN stays where it is; -inf gives
// -inf * 0, a NaN, as the formula does.  One reciprocal for two values (1 / a and 1 / b from
// 1 / (a b)) takes less of the special-function pipe but needs t held below 60, which leaves
// results of 1e-11 v in the tail.  32768 x 4096 x 1024 FP4, us: gelu 106.9 with a reciprocal
// each, 108.4 with one for two (110.6 with the tail mended there); silu 95.5, 93.1 (95.1);
// gelu_tanh 99.9, 99.2 (101.8).
#pragma once

#include "common.cuh"

namespace nvfp4 {

__device__ __forceinline__ float ex2_approx(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float rcp_approx(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Two fp32 products in one instruction, each rounded by itself.  (The packed sum is not
// used after it: the two were contracted into one fused multiply-add, written-out rounding
// or not, and that rounds once where the plain products round twice.)
__device__ __forceinline__ float2 mul2_rn(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// -log2(e) L(v) of the two values.
template <int ACT>
__device__ __forceinline__ float2 minus_logit2(float2 v) {
    if constexpr (ACT == NVFP4_ACT_SILU) return __fmul2_rn(v, both(-kLog2e));
    const float2 u = __fmul2_rn(v, v);
    if constexpr (ACT == NVFP4_ACT_GELU_TANH) {
        constexpr float c = -2.0f * 0.79788456080286535588f * kLog2e;
        return __fmul2_rn(v, __ffma2_rn(u, both(c * 0.044715f), both(c)));
    }
    // gelu: logit Phi(v) = v Q(v^2); Q fitted on |v| <= 6 for the least largest error of
    // v Phi(v).  Above 6, where Phi is 1, it keeps growing (Q > 4 from there on).
    float2 q = __ffma2_rn(u, both(-kLog2e * 3.6392367769551445e-09f), both(-kLog2e * -2.680700010037935e-07f));
    q = __ffma2_rn(u, q, both(-kLog2e * 7.956275638921296e-06f));
    q = __ffma2_rn(u, q, both(-kLog2e * -0.00011060688607769335f));
    q = __ffma2_rn(u, q, both(-kLog2e * -6.584639140541981e-05f));
    q = __ffma2_rn(u, q, both(-kLog2e * 0.07266800159418906f));
    q = __ffma2_rn(u, q, both(-kLog2e * 1.5957686572495096f));
    return __fmul2_rn(v, q);
}

template <int ACT>
__device__ __forceinline__ float2 act_value2(float2 v) {
    if constexpr (ACT == NVFP4_ACT_NONE) return v;
    if constexpr (ACT == NVFP4_ACT_RELU) return make_float2(fmaxf(v.x, 0.0f), fmaxf(v.y, 0.0f));
    const float2 t = minus_logit2<ACT>(v);
    const float2 d = __fadd2_rn(make_float2(ex2_approx(t.x), ex2_approx(t.y)), both(1.0f));
    return __fmul2_rn(v, make_float2(rcp_approx(d.x), rcp_approx(d.y)));
}

// act over the values of v that it applies to: all of them, or (GATED) the even ones, whose
// odd neighbour is then multiplied in (the result stays at the even places).
template <int ACT, bool GATED, int N>
__device__ __forceinline__ void activate(float (&v)[N]) {
    constexpr int D = GATED ? 2 : 1;
#pragma unroll
    for (int j = 0; j < N; j += 2 * D) {
        const float2 u = act_value2<ACT>(make_float2(v[j], v[j + D]));
        v[j] = GATED ? u.x * v[j + 1] : u.x;
        v[j + D] = GATED ? u.y * v[j + 3] : u.y;
    }
}

// The same with the activation chosen at run time (the reduction phases, few values a thread).
template <int N>
__device__ __forceinline__ void apply_activation(float (&v)[N], int act) {
    switch (act) {
        case NVFP4_ACT_RELU: return activate<NVFP4_ACT_RELU, false>(v);
        case NVFP4_ACT_GELU: return activate<NVFP4_ACT_GELU, false>(v);
        case NVFP4_ACT_GELU_TANH: return activate<NVFP4_ACT_GELU_TANH, false>(v);
        case NVFP4_ACT_SILU: return activate<NVFP4_ACT_SILU, false>(v);
        case NVFP4_ACT_GATED: return activate<NVFP4_ACT_NONE, true>(v);
        case NVFP4_ACT_GATED + NVFP4_ACT_RELU: return activate<NVFP4_ACT_RELU, true>(v);
        case NVFP4_ACT_GATED + NVFP4_ACT_GELU: return activate<NVFP4_ACT_GELU, true>(v);
        case NVFP4_ACT_GATED + NVFP4_ACT_GELU_TANH: return activate<NVFP4_ACT_GELU_TANH, true>(v);
        case NVFP4_ACT_GATED + NVFP4_ACT_SILU: return activate<NVFP4_ACT_SILU, true>(v);
        default: return;
    }
}

// Four consecutive columns (n % 4 == 0) of an output row, summed over the partial tiles of a
// cluster (at shared offset `off` of each of its CTAs, in rank order; int8 sums are exact in
// any order), scaled and biased.
template <bool I8>
__device__ __forceinline__ void reduce_granule(float (&v)[4], uint32_t off, int splits, float alpha,
                                               float sx, const float* sw, const uint16_t* bias, int n,
                                               int N) {
    float4 t = ld_dsmem_f4(dsmem_addr(off, 0));
    if constexpr (I8) {
        int acc[4] = {__float_as_int(t.x), __float_as_int(t.y), __float_as_int(t.z), __float_as_int(t.w)};
        for (int r = 1; r < splits; ++r) {
            t = ld_dsmem_f4(dsmem_addr(off, (uint32_t)r));
            acc[0] += __float_as_int(t.x);
            acc[1] += __float_as_int(t.y);
            acc[2] += __float_as_int(t.z);
            acc[3] += __float_as_int(t.w);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = __fmul_rn(__fmul_rn(__int2float_rn(acc[j]), sx), sw[min(n + j, N - 1)]);
    } else {
        v[0] = t.x;
        v[1] = t.y;
        v[2] = t.z;
        v[3] = t.w;
        for (int r = 1; r < splits; ++r) {
            t = ld_dsmem_f4(dsmem_addr(off, (uint32_t)r));
            v[0] = __fadd_rn(v[0], t.x);
            v[1] = __fadd_rn(v[1], t.y);
            v[2] = __fadd_rn(v[2], t.z);
            v[3] = __fadd_rn(v[3], t.w);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __fmul_rn(alpha, v[j]);
    }
    if (bias) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = __fadd_rn(v[j], __uint_as_float((uint32_t)bias[min(n + j, N - 1)] << 16));
    }
}

// The rest of such a granule: activation, residual, one rounding, store.  n_out: columns of y.
__device__ __forceinline__ void finish_granule(float (&v)[4], int act, bool gated,
                                               const uint16_t* residual, uint16_t* y, int64_t row,
                                               int n, int n_out) {
    apply_activation(v, act);
    if (gated) {
        const int col = n >> 1;
        const int64_t at = row * n_out + col;
        float u[2] = {v[0], v[2]};
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (residual && col + j < n_out)
                u[j] = __fadd_rn(u[j], __uint_as_float((uint32_t)residual[at + j] << 16));
        const uint32_t w = bf16x2_rn(u[0], u[1]);
        if ((n_out & 1) == 0) {
            *reinterpret_cast<uint32_t*>(y + at) = w;
        } else {
            y[at] = (uint16_t)w;
            if (col + 1 < n_out) y[at + 1] = (uint16_t)(w >> 16);
        }
        return;
    }
    const int64_t at = row * n_out + n;
    if ((n_out & 3) == 0) {
        if (residual) {
            const uint2 r = *reinterpret_cast<const uint2*>(residual + at);
            v[0] = __fadd_rn(v[0], bf16lo(r.x));
            v[1] = __fadd_rn(v[1], bf16hi(r.x));
            v[2] = __fadd_rn(v[2], bf16lo(r.y));
            v[3] = __fadd_rn(v[3], bf16hi(r.y));
        }
        *reinterpret_cast<uint2*>(y + at) = make_uint2(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]));
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (n + j < n_out) {
            if (residual)
                v[j] = __fadd_rn(v[j], __uint_as_float((uint32_t)residual[at + j] << 16));
            y[at + j] = (uint16_t)bf16x2_rn(v[j], 0.0f);
        }
}

}  // namespace nvfp4
