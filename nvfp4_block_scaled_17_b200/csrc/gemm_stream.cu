// gemm_stream.cu -- the products with an activation and a residual in their epilogue, for few
// activation rows and a weight that is long enough to occupy every SM.
//
// With M <= 64 rows the call is the weight's one trip from HBM (N x K bytes, or 9/16 of them
// for FP4), so the design keeps that stream going: one persistent CTA per SM walks tiles of
// 128 weight rows, and its copies run ahead across tile boundaries, as many stages as shared
// memory holds (ten of 22 KiB at M = 16).  The operands are swapped as in gemm_small.cu: the
// weight rows fill the MMA's M = 128, the activation rows (to a multiple of 16) its N.
// 51200 x 5120 FP4 for one token: 147 MB, 22.6 us at the measured copy rate; the cluster
// kernel, one tile of 256 rows per CTA and no split left, ran it as 1.35 waves in 38.7 us;
// this one takes 28.2 us, 0.80 of that rate (int8 42.6 us), of which 3 us are start and end.
//
//   warp 0      TMA producer: per stage (128 bytes of K) the 128-row weight box and its scale
//               chunks, the activation box and its chunks.
//   warp 1      MMA issue (converged, one election per K step) into one of two accumulators.
//   warps 2-5   epilogue: warp q holds weight rows 32 q + lane of the tile, so the 32 lanes
//               of a warp write 32 neighbouring columns of a row of y; a gated pair of
//               columns is a pair of lanes.
// Every wait is bounded; on expiry the kernel records NVFP4_ERR_TIMEOUT, lets its copies and
// MMAs finish, frees tensor memory and returns.  No load uses cluster multicast.
#include "activation.cuh"
#include "common.cuh"
#include "kernels.h"

#include <atomic>

namespace nvfp4 {

namespace {

constexpr int TROWS = 128;                    // weight rows of a tile
constexpr int TKB = 128;                      // bytes of K per stage
constexpr int TMAX_STAGES = 10;
constexpr int TTHREADS = 192;
constexpr int TS_W = TROWS * TKB;             // 16 KiB
constexpr int TS_SF = 4 * 512;                // one operand's scale chunks of a stage
constexpr int TSMEM = 232448;                 // all that a CTA can have
constexpr int TS_BARRIERS = 512;
constexpr uint32_t TTMEM_ACC1 = 64;           // second accumulator (kStreamMaxRows columns each)
constexpr uint32_t TTMEM_SF = 128;            // per K step of a stage 4 columns each for W and x
constexpr int TTMEM_COLS = 256;

struct StreamParams {
    const float* alpha;
    const float* sx;           // int8: fp32 row scales of the activation and of the weight
    const float* sw;
    const uint16_t* bias;      // bf16 [N] or null
    const uint16_t* residual;  // bf16 [M, n_out] or null
    uint16_t* y;               // bf16 [M, n_out]
    int M, N, n_out;
    int mpad;                  // the MMA's N: M rounded up to 16
    uint32_t idesc;
    int act, gated;
    int prepared;              // weight scales: 1 = prepared blocks, 0 = 128x4 chunks
    int tiles, k_tiles, kchunks;
    int stages, stage_bytes;
    int w_early;               // the weight was complete before the previous kernel started
    int* status;
    uint64_t budget_ns;
};

template <bool I8>
__device__ __forceinline__ void stream_step_w(uint32_t acc, uint64_t wd, uint64_t xd, uint32_t idesc,
                                              uint32_t sf_t, uint64_t sfw_d, uint64_t sfx_d,
                                              uint32_t accumulate) {
    if constexpr (I8) {
        mma_i8_w(acc, wd, xd, idesc, accumulate);
    } else {
        asm volatile(
            "{\n\t"
            ".reg .pred p, e;\n\t"
            ".reg .b32 t;\n\t"
            "elect.sync _|e, 0xffffffff;\n\t"
            "setp.ne.b32 p, %7, 0;\n\t"
            "add.u32 t, %4, 4;\n\t"
            "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%4], %5;\n\t"
            "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [t], %6;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.block16 [%0], %1, %2, %3, "
            "[%4], [t], p;\n\t"
            "}" ::"r"(acc),
            "l"(wd), "l"(xd), "r"(idesc), "r"(sf_t), "l"(sfw_d), "l"(sfx_d), "r"(accumulate)
            : "memory");
    }
}

template <bool I8>
__global__ void __launch_bounds__(TTHREADS, 1)
gemm_stream_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const __grid_constant__ CUtensorMap tmSFW, const __grid_constant__ CUtensorMap tmSFX,
                   const StreamParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.stages * p.stage_bytes);
    uint64_t* empty = full + TMAX_STAGES;
    uint64_t* acc_full = empty + TMAX_STAGES;    // [2]
    uint64_t* acc_free = acc_full + 2;           // [2]
    uint64_t* drain = acc_free + 2;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_free[b], 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc(tmem_holder, TTMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    // A stage: W box | scales of W | scales of x | x box.
    auto load_w = [&](int stage, int kt, int tile) {
        uint8_t* s = smem + stage * p.stage_bytes;
        tma_load_2d_w(s, &tmW, &full[stage], kt * TKB, tile * TROWS);
        if constexpr (!I8)
            tma_load_3d_w(s + TS_W, &tmSFW, &full[stage], 0,
                          p.prepared ? ((tile >> 1) * p.k_tiles + kt) * 8 + (tile & 1) * 4 : 4 * kt,
                          p.prepared ? 0 : tile);
    };
    auto load_x = [&](int stage, int kt) {
        uint8_t* s = smem + stage * p.stage_bytes;
        tma_load_2d_w(s + TS_W + (I8 ? 0 : 2 * TS_SF), &tmX, &full[stage], kt * TKB, 0);
        if constexpr (!I8) tma_load_3d_w(s + TS_W + TS_SF, &tmSFX, &full[stage], 0, 4 * kt, 0);
    };
    const uint32_t bytes = TS_W + (uint32_t)p.mpad * TKB + (I8 ? 0u : 2u * TS_SF);
    int n_early = 0;
    if (warp == 0) {
        if (lane == 0) {
            prefetch_tensormap(&tmW);
            prefetch_tensormap(&tmX);
        }
        if (p.w_early && (int)blockIdx.x < p.tiles) {
            n_early = min(p.stages, p.k_tiles);
            for (int i = 0; i < n_early; ++i) {
                mbar_arrive_expect_tx_w(&full[i], bytes);
                load_w(i, i, (int)blockIdx.x);
            }
        }
    }
    griddep_wait();
    griddep_launch_dependents();

    if (warp == 0) {
        int stage = 0, fills = 0;
        uint32_t phase = 0, issued = 0, issued_phase = 0;
        bool ok = true;
        for (int tile = blockIdx.x; ok && tile < p.tiles; tile += gridDim.x) {
            for (int kt = 0; kt < p.k_tiles; ++kt, ++fills) {
                if (fills >= n_early) {
                    if (!mbar_wait_bounded_warp(&empty[stage], phase ^ 1, abort_flag, p.status,
                                                p.budget_ns)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx_w(&full[stage], bytes);
                    load_w(stage, kt, tile);
                }
                load_x(stage, kt);
                issued |= 1u << stage;
                issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        // every fill this warp started must land before the block can exit
        for (int s = 0; s < p.stages; ++s)
            if (issued & (1u << s)) {
                volatile int no_abort = 0;
                mbar_wait_bounded(&full[s], (issued_phase >> s) & 1, &no_abort, p.status, p.budget_ns);
            }
    } else if (warp == 1) {
        int stage = 0, it = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int tile = blockIdx.x; ok && tile < p.tiles; tile += gridDim.x, ++it) {
            const int b = it & 1;
            if (!mbar_wait_bounded_warp(&acc_free[b], (uint32_t)((it >> 1) & 1) ^ 1, abort_flag,
                                        p.status, p.budget_ns)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + (b ? TTMEM_ACC1 : 0u);
            for (int kt = 0; kt < p.k_tiles; ++kt) {
                if (!mbar_wait_bounded_warp(&full[stage], phase, abort_flag, p.status, p.budget_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t s = smem_u32(smem + stage * p.stage_bytes);
                const uint64_t wd = sdesc_kmajor_sw128(s);
                const uint64_t xd = sdesc_kmajor_sw128(s + TS_W + (I8 ? 0 : 2 * TS_SF));
                const uint64_t sfw_d = sdesc_sf(s + TS_W), sfx_d = sdesc_sf(s + TS_W + TS_SF);
                // Four steps to every stage, without a branch between them: past the end of K
                // both operands are zero (as in gemm_pair.cu).
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    stream_step_w<I8>(acc, wd + 2 * kk, xd + 2 * kk, p.idesc,
                                      tmem + TTMEM_SF + 8u * (uint32_t)kk, sfw_d + 32 * kk,
                                      sfx_d + 32 * kk, kk > 0 || kt > 0 ? 1u : 0u);
                tc_commit_w(&empty[stage]);
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (!ok) break;
            tc_commit_w(&acc_full[b]);
        }
        tc_commit_w(drain);
        volatile int no_abort = 0;
        mbar_wait_bounded(drain, 0, &no_abort, p.status, p.budget_ns);
        __syncwarp();
    } else {
        const int quad = warp & 3;
        const float alpha = I8 ? 0.0f : *p.alpha;
        int it = 0;
        for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x, ++it) {
            const int b = it & 1;
            const int n = tile * TROWS + quad * 32 + lane;
            const bool live = n < p.N;
            const float bias = p.bias && live ? __uint_as_float((uint32_t)p.bias[n] << 16) : 0.0f;
            const float sw = I8 && live ? p.sw[n] : 0.0f;
            if (!mbar_wait_bounded_warp(&acc_full[b], (uint32_t)((it >> 1) & 1), abort_flag, p.status,
                                        p.budget_ns))
                break;
            tc_fence_after();
            const uint32_t at = tmem + ((uint32_t)(quad * 32) << 16) + (b ? TTMEM_ACC1 : 0u);
            for (int m0 = 0; m0 < p.M; m0 += 16) {
                uint32_t r[16];
                tmem_ld16(at + (uint32_t)m0, r);
                tmem_ld_wait();
                if (m0 + 16 >= p.M) {            // the accumulator has been read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&acc_free[b]);
                }
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    if constexpr (I8)
                        v[j] = __fmul_rn(__fmul_rn(__int2float_rn((int)r[j]),
                                                   m0 + j < p.M ? p.sx[m0 + j] : 0.0f), sw);
                    else
                        v[j] = __fmul_rn(alpha, __uint_as_float(r[j]));
                    if (p.bias) v[j] = __fadd_rn(v[j], bias);
                }
                // A gated pair is two lanes: the even one holds the gate, the odd one up.
                float up[16];
                if (p.gated) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) up[j] = __shfl_down_sync(0xffffffffu, v[j], 1);
                }
                apply_activation(v, p.act & ~NVFP4_ACT_GATED);
                const int col = p.gated ? n >> 1 : n;
                const bool writes = live && (!p.gated || (lane & 1) == 0);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    if (m0 + j >= p.M || !writes) continue;
                    const size_t o = (size_t)(m0 + j) * p.n_out + col;
                    float u = p.gated ? v[j] * up[j] : v[j];
                    if (p.residual) u = __fadd_rn(u, __uint_as_float((uint32_t)p.residual[o] << 16));
                    p.y[o] = (uint16_t)bf16x2_rn(u, 0.0f);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TTMEM_COLS);
    }
}

template <bool I8>
nvfp4_status launch_stream_impl(const GemmActArgs& g, cudaStream_t stream) {
    DeviceInfo dev;
    nvfp4_status st = device_info(&dev);
    if (st != NVFP4_OK) return st;
    int* status = nullptr;
    if ((st = status_word(&status)) != NVFP4_OK) return st;
    static std::atomic<int> attr_set[64];
    if (!attr_set[dev.device & 63].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(gemm_stream_kernel<I8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 TSMEM) != cudaSuccess)
            return NVFP4_ERR_CUDA;
        attr_set[dev.device & 63].store(1, std::memory_order_release);
    }
    const int64_t kbytes = I8 ? g.K : g.K / 2;
    StreamParams p{};
    p.alpha = g.alpha;
    p.sx = g.sx;
    p.sw = g.sw;
    p.bias = static_cast<const uint16_t*>(g.bias);
    p.residual = static_cast<const uint16_t*>(g.epi.residual);
    p.y = static_cast<uint16_t*>(g.y);
    p.M = (int)g.M;
    p.N = (int)g.N;
    p.act = g.epi.activation;
    p.gated = (g.epi.activation & NVFP4_ACT_GATED) ? 1 : 0;
    p.n_out = (int)(p.gated ? g.N / 2 : g.N);
    p.mpad = (int)((g.M + 15) / 16 * 16);
    p.idesc = (I8 ? 2u << 4 : 0u) | (1u << 7) | (1u << 10) | ((uint32_t)(p.mpad >> 3) << 17) |
              ((uint32_t)(TROWS >> 4) << 24);
    p.prepared = g.sfb_prepared ? 1 : 0;
    p.tiles = (int)((g.N + TROWS - 1) / TROWS);
    p.k_tiles = (int)((kbytes + TKB - 1) / TKB);
    p.kchunks = (int)(kbytes / 32);
    // the x box starts on a 1 KiB boundary, and so does the next stage
    p.stage_bytes = (TS_W + (I8 ? 0 : 2 * TS_SF) + p.mpad * TKB + 1023) / 1024 * 1024;
    p.stages = (TSMEM - 1024 - TS_BARRIERS) / p.stage_bytes;
    if (p.stages > TMAX_STAGES) p.stages = TMAX_STAGES;
    p.w_early = g.weights_ready ? 1 : 0;
    p.status = status;
    p.budget_ns = 4000000000ull;   // 4 s
    CUtensorMap mapW, mapX, mapSFW, mapSFX;
    if (!make_operand_map(&mapW, g.b, g.N, kbytes, TROWS) ||
        !make_operand_map(&mapX, g.a, g.M, kbytes, p.mpad))
        return NVFP4_ERR_CUDA;
    mapSFW = mapSFX = mapX;                    // unused by int8
    if (!I8) {
        if (!(p.prepared ? make_scale_map(&mapSFW, g.sfb, (g.N + 255) / 256 * p.k_tiles * 8, 1)
                         : make_scale_map(&mapSFW, g.sfb, p.kchunks, p.tiles)) ||
            !make_scale_map(&mapSFX, g.sfa, p.kchunks, 1))
            return NVFP4_ERR_CUDA;
    }
    const unsigned grid = (unsigned)(p.tiles < dev.sms ? p.tiles : dev.sms);
    return launch_pdl(gemm_stream_kernel<I8>, grid, TTHREADS, TSMEM, stream, mapW, mapX, mapSFW, mapSFX,
                      p) == cudaSuccess
               ? NVFP4_OK
               : NVFP4_ERR_CUDA;
}

}  // namespace

nvfp4_status launch_gemm_stream(const GemmActArgs& g, cudaStream_t stream) {
    if (g.M < 1 || g.M > kStreamMaxRows) return NVFP4_ERR_INVALID_ARG;
    return g.int8 ? launch_stream_impl<true>(g, stream) : launch_stream_impl<false>(g, stream);
}

}  // namespace nvfp4
