// norm.cu -- residual addition, root-mean-square norm and quantization in one pass.
//
// What a transformer block does in front of a quantized linear:
//     h = bf16(x + residual)                       (h = x without a residual)
//     rstd = fp32(1 / sqrt(mean(h^2) + eps))       per row
//     n = bf16(fp32(fp32(h * rstd) * w))
// followed by the library's own encoding of n: per-row int8 codes (int8_quantize_rows) or
// NVFP4 codes under a static global scale (nvfp4_quantize without rotation).  The codes
// equal those of the separate passes on the bf16 n bit for bit, NaN and infinities included.
//
// The sum of squares is kept in 64 bits: the square of a bf16 value is exact there and the
// sum's relative error is below 2^-49 for any row, so rstd (one rounding to fp32) does not
// depend on the order of the additions, and with it neither do the codes.
//
// Layout: a unit is 16 consecutive values of a row (one NVFP4 block; 32 bytes of bf16, 16
// of int8 codes).  A thread owns C units of a row, lane-contiguous, so a row is read once
// into registers and every store is 16 bytes wide (8 for FP4 codes).
//
// Bound by HBM: with a residual 7 bytes a value (int8; 6.56 FP4), each moved once.  B200,
// graph replay: 32768 x 5120 int8 193 us, 6.08 TB/s (0.93 of the measured copy rate; 215
// before the arithmetic was packed in pairs and the codes were rounded by an addition, 199
// with a minimum per value that gives a NaN's code, where one branch per row takes 193);
// 32768 x 1024 FP4 37.8 us, 5.83 TB/s (0.89); a single row of 5120 2.7 us, of which a launch
// alone takes two.  Fetching the next row while the current one is worked on gained nothing:
// six blocks of 320 threads on an SM cover the latency already.
#include "common.cuh"
#include "kernels.h"

#include <atomic>
#include <type_traits>

namespace nvfp4 {

namespace {

constexpr int kNormWarpThreads = 256;      // warp-per-row blocks: eight rows at a time

struct NormParams {
    const uint16_t* x;
    const uint16_t* residual;   // or null
    const uint16_t* weight;     // or null: ones
    uint16_t* h_out;            // or null
    uint16_t* n_out;            // or null
    int64_t rows, rows_padded;  // rows_padded: rows of the scale layout (FP4), else rows
    int64_t K;
    int units;                  // K / 16
    int units_padded;           // scale columns (FP4: to a multiple of four), else units
    double inv_k, eps;
    // int8
    int8_t* q;
    float* scale;
    // NVFP4
    const float* gsf;
    const float* gsf_w;
    float* alpha_out;
    uint8_t* packed;
    uint8_t* sf;
    int64_t cgroups;            // four-block column groups of the scale layout
};

struct Unit {
    uint32_t w[8];              // 16 bf16 values
};

__device__ __forceinline__ Unit load_unit(const uint16_t* p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint4 b = *reinterpret_cast<const uint4*>(p + 8);
    return Unit{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

__device__ __forceinline__ void store_unit(uint16_t* p, const Unit& u) {
    *reinterpret_cast<uint4*>(p) = make_uint4(u.w[0], u.w[1], u.w[2], u.w[3]);
    *reinterpret_cast<uint4*>(p + 8) = make_uint4(u.w[4], u.w[5], u.w[6], u.w[7]);
}

// As absmax2_bf16, but a NaN in either operand stays.
__device__ __forceinline__ uint32_t absmax2_nan_bf16(uint32_t a, uint32_t b) {
    uint32_t m;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    return m;
}

template <uint32_t (*MAX)(uint32_t, uint32_t)>
__device__ __forceinline__ uint32_t unit_absmax(const Unit& u) {
    return MAX(MAX(MAX(u.w[0], u.w[1]), MAX(u.w[2], u.w[3])),
               MAX(MAX(u.w[4], u.w[5]), MAX(u.w[6], u.w[7])));
}

// The maximum over a row's units: of the lane's (h), the warp's, and with BLOCK the block's.
// red holds a value for each warp.
template <uint32_t (*MAX)(uint32_t, uint32_t), int C, bool BLOCK>
__device__ __forceinline__ uint32_t row_absmax(const Unit (&h)[C], uint32_t* red, int warps) {
    const int lane = threadIdx.x & 31;
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < C; ++i) m = MAX(m, unit_absmax<MAX>(h[i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = MAX(m, __shfl_xor_sync(0xffffffffu, m, o));
    if constexpr (BLOCK) {
        if (lane == 0) red[threadIdx.x >> 5] = m;
        __syncthreads();
        m = lane < warps ? red[lane] : 0u;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = MAX(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    return m;
}

__device__ __forceinline__ float2 pair_of(uint32_t w) { return make_float2(bf16lo(w), bf16hi(w)); }
__device__ __forceinline__ float2 twice(float v) { return make_float2(v, v); }

// 16 int8 codes of a unit under the row scale s; r = rn(1 / s).  fast: rn(n / s) by one
// remainder step (Markstein), as int8_quantize_rows computes it, and a whole number by adding
// 1.5 * 2^23, which rounds |t| <= 127 half to even and leaves the code in the low byte.
// Otherwise, for a subnormal s (its reciprocal would overflow; s = 0 gives zeros) and for rows
// with a NaN or an infinity, a division and a conversion, in which a NaN gives 0.
// 16 int8 codes of a unit under the row scale s; r = rn(1 / s).  FAST: rn(n / s) by one
// remainder step (Markstein), as int8_quantize_rows computes it, and a whole number by adding
// 1.5 * 2^23, which rounds |t| <= 127 half to even and leaves the code in the low byte.
// Otherwise, for a subnormal s (its reciprocal would overflow; s = 0 gives zeros) and for rows
// with a NaN or an infinity, a division and a conversion, in which a NaN gives 0.
template <bool FAST>
__device__ __forceinline__ uint4 int8_codes(const Unit& u, float s, float r) {
    uint32_t out[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 v = pair_of(u.w[2 * g + j]);
            if constexpr (FAST) {
                const float2 q0 = __fmul2_rn(v, twice(r));
                const float2 t = __ffma2_rn(__ffma2_rn(q0, twice(-s), v), twice(r), q0);
                c[2 * j] = __float_as_uint(__fadd_rn(t.x, 12582912.0f));
                c[2 * j + 1] = __float_as_uint(__fadd_rn(t.y, 12582912.0f));
            } else {
                c[2 * j] = s != 0.0f ? (uint32_t)__float2int_rn(__fdiv_rn(v.x, s)) : 0u;
                c[2 * j + 1] = s != 0.0f ? (uint32_t)__float2int_rn(__fdiv_rn(v.y, s)) : 0u;
            }
        }
        out[g] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

// One block of 16 values as nvfp4_quantize encodes it under a static global scale.
__device__ __forceinline__ uint32_t fp4_codes(const Unit& u, float gsf, uint2& codes) {
    const uint32_t s8 = e4m3_scale_of_scaled_max(__fmul_rn(gsf, absmax_of_pair(unit_absmax<absmax2_bf16>(u))));
    const float inv = (s8 == 0u || s8 == 127u) ? 0.0f : __fdiv_rn(gsf, f32_from_e4m3(s8));
    float v[2][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float2 t = __fmul2_rn(pair_of(u.w[j]), twice(inv));
        v[j >> 2][2 * (j & 3)] = t.x;
        v[j >> 2][2 * (j & 3) + 1] = t.y;
    }
    codes.x = s8 ? e2m1x8_from_f32(v[0]) : 0u;
    codes.y = s8 ? e2m1x8_from_f32(v[1]) : 0u;
    return s8;
}

// C units per thread; BLOCK: a row per block (blockDim.x threads), else a row per warp.
template <bool FP4, int C, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : kNormWarpThreads) norm_kernel(const NormParams p) {
    __shared__ double red_ss[32];
    __shared__ uint32_t red_mx[32];
    griddep_wait();
    griddep_launch_dependents();

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int span = BLOCK ? (int)blockDim.x : 32;         // threads of a row
    const int tid = BLOCK ? (int)threadIdx.x : lane;
    const int warps = (int)blockDim.x >> 5;
    const int64_t first = BLOCK ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * warps + warp;
    const int64_t step = BLOCK ? (int64_t)gridDim.x : (int64_t)gridDim.x * warps;
    const float gsf = FP4 ? *p.gsf : 0.0f;
    if (FP4 && p.alpha_out && blockIdx.x == 0 && threadIdx.x == 0)
        *p.alpha_out = __frcp_rn(__fmul_rn(gsf, *p.gsf_w));

    for (int64_t row = first; row < p.rows_padded; row += step) {
        if (FP4 && row >= p.rows) {                        // padding rows of the scale layout
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int u = i * span + tid;
                if (u < p.units_padded)
                    p.sf[((row >> 7) * p.cgroups + (u >> 2)) * 512 + ((row & 31) << 4) +
                         (((row >> 5) & 3) << 2) + (u & 3)] = 0;
            }
            continue;
        }
        Unit h[C];
        double ss0 = 0.0, ss1 = 0.0;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int u = i * span + tid;
            if (u < p.units) h[i] = load_unit(p.x + row * p.K + 16 * (int64_t)u);
            else h[i] = Unit{};
        }
        if (p.residual) {
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int u = i * span + tid;
                if (u >= p.units) continue;
                const int64_t at = row * p.K + 16 * (int64_t)u;
                const Unit r = load_unit(p.residual + at);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 t = __fadd2_rn(pair_of(h[i].w[j]), pair_of(r.w[j]));
                    h[i].w[j] = bf16x2_rn(t.x, t.y);
                }
                if (p.h_out) store_unit(p.h_out + at, h[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const double a = (double)bf16lo(h[i].w[j]), b = (double)bf16hi(h[i].w[j]);
                ss0 = fma(a, a, ss0);
                ss1 = fma(b, b, ss1);
            }
        double ss = ss0 + ss1;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if constexpr (BLOCK) {
            if (lane == 0) red_ss[warp] = ss;
            __syncthreads();
            ss = lane < warps ? red_ss[lane] : 0.0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        }
        const float rstd = (float)rsqrt(ss * p.inv_k + p.eps);

#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int u = i * span + tid;
            Unit w{{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u,
                    0x3f803f80u, 0x3f803f80u}};
            if (p.weight && u < p.units) w = load_unit(p.weight + 16 * (int64_t)u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 t = __fmul2_rn(__fmul2_rn(pair_of(h[i].w[j]), twice(rstd)), pair_of(w.w[j]));
                h[i].w[j] = bf16x2_rn(t.x, t.y);
            }
            if (p.n_out && u < p.units) store_unit(p.n_out + row * p.K + 16 * (int64_t)u, h[i]);
        }
        if constexpr (FP4) {
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int u = i * span + tid;
                uint2 codes = make_uint2(0u, 0u);
                uint32_t s8 = 0u;
                if (u < p.units) {
                    s8 = fp4_codes(h[i], gsf, codes);
                    *reinterpret_cast<uint2*>(p.packed + row * (p.K / 2) + 8 * (int64_t)u) = codes;
                }
                if (u < p.units_padded)
                    p.sf[((row >> 7) * p.cgroups + (u >> 2)) * 512 + ((row & 31) << 4) +
                         (((row >> 5) & 3) << 2) + (u & 3)] = (uint8_t)s8;
            }
        } else {
            // The scale comes from the values that are no NaN, as int8_quantize_rows takes it: a
            // second reduction in the rows that have one (the row's threads agree).
            uint32_t m = row_absmax<absmax2_nan_bf16, C, BLOCK>(h, red_mx, warps);
            const bool finite = (m & 0x7fffu) < 0x7f80u && (m & 0x7fff0000u) < 0x7f800000u;
            if (!finite) {
                if (BLOCK) __syncthreads();            // red_mx has been read
                m = row_absmax<absmax2_bf16, C, BLOCK>(h, red_mx, warps);
            }
            const float s = __fdiv_rn(absmax_of_pair(m), 127.0f);
            if (tid == 0) p.scale[row] = s;
            const bool fast = finite && s >= 1.17549435e-38f;
            auto store = [&](auto form, float r) {
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    const int u = i * span + tid;
                    if (u < p.units)
                        *reinterpret_cast<uint4*>(p.q + row * p.K + 16 * (int64_t)u) =
                            int8_codes<decltype(form)::value>(h[i], s, r);
                }
            };
            if (fast) store(std::true_type{}, __frcp_rn(s));
            else store(std::false_type{}, 0.0f);
        }
        if constexpr (FP4 && BLOCK) __syncthreads();   // red_ss is free for the next row
    }
}

template <bool FP4, int C, bool BLOCK>
nvfp4_status launch_norm(const NormParams& p, int threads, const DeviceInfo& dev,
                         cudaStream_t stream) {
    static std::atomic<int> per_sm[64][33];    // resident blocks, by warps of a block
    std::atomic<int>& cell = per_sm[dev.device & 63][threads / 32];
    int resident = cell.load(std::memory_order_relaxed);
    if (!resident) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, norm_kernel<FP4, C, BLOCK>,
                                                          threads, 0) != cudaSuccess ||
            resident <= 0)
            return NVFP4_ERR_CUDA;
        cell.store(resident, std::memory_order_relaxed);
    }
    const int per_block = BLOCK ? 1 : threads / 32;
    const int64_t need = (p.rows_padded + per_block - 1) / per_block;
    const int64_t cap = (int64_t)dev.sms * resident;
    const unsigned grid = (unsigned)(need < cap ? need : cap);
    return launch_pdl(norm_kernel<FP4, C, BLOCK>, grid, (unsigned)threads, 0, stream, p) ==
                   cudaSuccess
               ? NVFP4_OK
               : NVFP4_ERR_CUDA;
}

template <bool FP4>
nvfp4_status dispatch_norm(const NormParams& p, const DeviceInfo& dev, cudaStream_t stream) {
    // A warp per row as long as a lane has one unit (no block barrier; 32768 x 512 int8 20.4
    // us against 23.4 with a block per row), then a block per row with one unit per thread:
    // more units on fewer threads lengthen the chain of a row (1040 values: 777 rows int8 4.1 us
    // with a warp of three units a lane, 3.1 with a block of 96 threads; 32768 rows int8 50.4
    // and 57.0, FP4 55.1 and 51.1).  Above 1024 units a thread takes two or four.
    const int U = p.units_padded;
    if (U <= 32) return launch_norm<FP4, 1, false>(p, kNormWarpThreads, dev, stream);
    // Two units a lane as well from 2400 rows on, where blocks go into another round (16 rows a
    // SM is 2368).  Warps : blocks, us, 528 and 1024 values: int8 2048 rows 3.79 : 3.69 and
    // 4.01 : 4.00, 2400 rows 5.37 : 5.81 and 5.97 : 6.50, 32768 rows 30.5 : 37.7 and 39.1 :
    // 40.6; FP4 2368 rows 4.66 : 4.37 and 5.07 : 4.70, 2400 rows 5.41 : 5.45 and 5.97 : 6.25,
    // 32768 rows 28.2 : 33.7 and 37.4 : 37.8.
    if (U <= 64 && p.rows >= 2400) return launch_norm<FP4, 2, false>(p, kNormWarpThreads, dev, stream);
    if (U <= 1024) return launch_norm<FP4, 1, true>(p, (U + 31) / 32 * 32, dev, stream);
    if (U <= 2048) return launch_norm<FP4, 2, true>(p, ((U + 1) / 2 + 31) / 32 * 32, dev, stream);
    return launch_norm<FP4, 4, true>(p, ((U + 3) / 4 + 31) / 32 * 32, dev, stream);
}

NormParams norm_params(const NormInputs& in) {
    NormParams p{};
    p.x = static_cast<const uint16_t*>(in.x);
    p.residual = static_cast<const uint16_t*>(in.residual);
    p.weight = static_cast<const uint16_t*>(in.weight);
    p.h_out = static_cast<uint16_t*>(in.residual_out);
    p.n_out = static_cast<uint16_t*>(in.norm_out);
    p.rows = p.rows_padded = in.rows;
    p.K = in.K;
    p.units = p.units_padded = (int)(in.K / 16);
    p.inv_k = 1.0 / (double)in.K;
    p.eps = in.eps;
    return p;
}

}  // namespace

nvfp4_status launch_int8_norm(const NormInputs& in, int8_t* q, float* scale, cudaStream_t stream) {
    DeviceInfo dev;
    nvfp4_status st = device_info(&dev);
    if (st != NVFP4_OK) return st;
    NormParams p = norm_params(in);
    p.q = q;
    p.scale = scale;
    return dispatch_norm<false>(p, dev, stream);
}

nvfp4_status launch_nvfp4_norm(const NormInputs& in, const float* gsf, uint8_t* packed,
                               uint8_t* sf, const float* gsf_w, float* alpha_out,
                               cudaStream_t stream) {
    DeviceInfo dev;
    nvfp4_status st = device_info(&dev);
    if (st != NVFP4_OK) return st;
    NormParams p = norm_params(in);
    p.gsf = gsf;
    p.gsf_w = gsf_w;
    p.alpha_out = alpha_out;
    p.packed = packed;
    p.sf = sf;
    p.rows_padded = (in.rows + 127) / 128 * 128;
    p.units_padded = (p.units + 3) / 4 * 4;
    p.cgroups = p.units_padded / 4;
    return dispatch_norm<true>(p, dev, stream);
}

}  // namespace nvfp4
