// gemm_pair.cu -- the products with an activation and a residual in their epilogue, for
// grids that fill the GPU: two SMs on one 256 x 256 output tile.
//
//     v = fp32(scale * acc) + bias;  u = act(v), or act(v[2j]) v[2j + 1];  y = bf16(u + r)
//
// Why pairs.  An SM's shared memory moves 128 bytes a cycle.  A 128 x 256 tile on one SM
// reads 12 KiB per 128-cycle MMA (4 KiB of A, 8 KiB of B) and takes the same 12 KiB in from
// TMA: 192 bytes a cycle, so such a kernel runs the tensor cores at two thirds.  With
// cta_group::2 each SM holds 128 rows of A and 128 of B, and the pair shares B: 8 KiB read
// and 8 KiB written per MMA, 128 bytes a cycle; the traffic from L2 falls by a third too.
//
// Design (a cluster of two CTAs, persistent over tiles; 576 threads each):
//   warp 0      TMA producer of its CTA: per stage (128 bytes of K) a 128-row A box, a
//               128-row B box (128-byte swizzle) and, for FP4, the scale chunks of its own
//               A rows and of all 256 B rows, which each SM needs in its tensor memory.
//               Every load signals the leader's full barrier (cta_group::2 loads may).
//   warp 1      in the leader: MMA issue for both SMs (M = 256, N = 256), the whole warp
//               converged, one election per K step; commits arrive at both CTAs' barriers.
//   warps 2-17  epilogue of the CTA's 128 rows, two groups of eight warps that take the
//               tiles in turn, so the latencies of one (tensor-memory loads, stores, barriers)
//               are covered by the arithmetic of the other.  A warp has a tensor-memory
//               quadrant and 128 columns, in two parts of 64 that it reads into registers at
//               once; the second part's read releases the accumulator.  Output chunks of
//               32 x 32 go through a swizzled staging tile and a TMA store; with a residual,
//               its chunk is loaded into the same staging tile beforehand.
// The tiles of a last, at most half full wave are cut into two of 128 columns each, which
// then all run at once: 4096 x 5120 x 25600 is 320 tiles on 74 pairs, 4.5 waves instead of 5.
// int8 accumulators are two full 256-column buffers; FP4 ones share 64 columns ([0, 256) and
// [192, 448)) to leave room for the scales of a stage's four K steps at [448, 496).
//
// Every wait is bounded; on expiry the kernel records NVFP4_ERR_TIMEOUT, lets its copies
// land, frees tensor memory and returns.  No load uses cluster multicast.
#include "activation.cuh"
#include "common.cuh"
#include "kernels.h"

#include <atomic>
#include <type_traits>

namespace nvfp4 {

namespace {

constexpr int PROWS = 128;                    // A rows, and B rows, of one CTA
constexpr int PN = 256;                       // columns of a tile
constexpr int PKB = 128;                      // bytes of K per stage
constexpr int PSTAGES = 4;
constexpr int PEPI = 16;                      // epilogue warps
constexpr int PTHREADS = 64 + 32 * PEPI;
constexpr int PS_OP = PROWS * PKB;            // 16 KiB: A, and B
constexpr int PS_SFA = 4 * 512;
constexpr int PS_SFB = 8 * 512;
constexpr int P_STG = 32 * 64;                // one 32 x 32 bf16 staging tile; two per warp
constexpr int P_GROUP = 8;                    // row blocks of a supertile
template <bool I8>
struct PairSmem {
    static constexpr int STAGE = 2 * PS_OP + (I8 ? 0 : PS_SFA + PS_SFB);
    static constexpr int COLS = (I8 ? 2 : 1) * 128 * 4;   // a warp's bias and column scales (int8)
    static constexpr int BYTES = 1024 + PSTAGES * STAGE + PEPI * (2 * P_STG + COLS) + 512;
};
static_assert(PairSmem<false>::BYTES <= 232448 && PairSmem<true>::BYTES <= 232448,
              "dynamic shared memory above the 227 KiB a CTA can have");
constexpr uint32_t PTMEM_SF = 448;
// E2M1 x E2M1 (format 1), or signed int8 (format 1) with an int32 accumulator; K-major,
// N = 256, M = 256 over the pair
constexpr uint32_t PIDESC = (1u << 7) | (1u << 10) | ((uint32_t)(PN >> 3) << 17) | (16u << 24);
constexpr uint32_t PIDESC_I8 = PIDESC | (2u << 4);
constexpr uint32_t PIDESC_HALF = (uint32_t)(PN >> 4) << 17;   // N = 128: subtracted

struct PairParams {
    const float* alpha;
    const float* sx;           // int8: fp32 row scales of A and of B
    const float* sw;
    const uint16_t* bias;      // bf16 [N] or null
    const uint16_t* residual;  // bf16 [M, n_out] or null
    uint16_t* y;               // bf16 [M, n_out]
    int M, N, n_out;
    int m_blocks, n_blocks;
    int items, whole;          // work items: whole tiles, then halves of the tiles after them
    FastDiv div_super, div_last;   // by the tiles of a supertile, by the last one's rows
    int k_tiles;               // stages of K
    int kchunks;               // 32-byte K steps
    int prepared;              // B scales: 1 = prepared blocks, 0 = 128x4 chunks
    int w_early;               // B was complete before the previous kernel started
    int* status;
    uint64_t budget_ns;
};

// ---- cta_group::2 forms -------------------------------------------------------------------

__device__ __forceinline__ void tma_load_2d_pair_w(uint32_t dst, const CUtensorMap* map,
                                                   uint32_t leader_bar, int32_t x, int32_t y) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(leader_bar), "r"(x), "r"(y)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair_w(uint32_t dst, const CUtensorMap* map,
                                                   uint32_t leader_bar, int32_t x, int32_t y,
                                                   int32_t z) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(leader_bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Completion of all earlier MMAs and scale copies, to the barrier at this offset in both CTAs.
__device__ __forceinline__ void commit_both_w(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
        ".b64 [%0], m;\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void commit_own_w(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            smem_u32(bar))
        : "memory");
}

template <bool HALF>
__device__ __forceinline__ void pair_step_i8_w(uint32_t d, uint64_t ad, uint64_t bd,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(HALF ? PIDESC_I8 - PIDESC_HALF : PIDESC_I8), "r"(accumulate)
        : "memory");
}

// One FP4 K step: each SM's scale chunks (its A rows; the one or two 128-row halves of B) from
// its own shared memory into its own tensor memory, then the MMA over both.
template <bool HALF>
__device__ __forceinline__ void pair_step_fp4_w(uint32_t d, uint64_t ad, uint64_t bd, uint32_t sf_t,
                                                uint64_t sfa_d, uint64_t sfb_d,
                                                uint32_t accumulate) {
    if constexpr (HALF) {
        asm volatile(
            "{\n\t.reg .pred p, e;\n\t.reg .b32 t;\n\t"
            "elect.sync _|e, 0xffffffff;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "add.u32 t, %5, 4;\n\t"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%5], %6;\n\t"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [t], %7;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.block16 [%0], %1, %2, %3, "
            "[%5], [t], p;\n\t}" ::"r"(d),
            "l"(ad), "l"(bd), "r"(PIDESC - PIDESC_HALF), "r"(accumulate), "r"(sf_t), "l"(sfa_d),
            "l"(sfb_d)
            : "memory");
        return;
    }
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b32 t, u;\n\t.reg .b64 s;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "add.u32 t, %5, 4;\n\t"
        "add.u32 u, %5, 8;\n\t"
        "add.u64 s, %7, 128;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%5], %6;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [t], %7;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [u], s;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.block16 [%0], %1, %2, %3, [%5], "
        "[t], p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(PIDESC), "r"(accumulate), "r"(sf_t), "l"(sfa_d), "l"(sfb_d)
        : "memory");
}

// Arrival at a barrier of either CTA.  It hands over tensor memory (ordered by the tcgen05
// fences around it), no generic writes, so the default scope is enough: a release at cluster
// scope costs a memory barrier on the path from one tile's accumulator to the next MMA.
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// Bounded wait of a whole warp, converged; lane 0's outcome decides.  Arrivals may come from
// the other CTA.  The clock and the abort flag are read once in 32 polls: read in every one,
// the waiting warps kept the pipe that the epilogue's conversions need 92 % busy.
__device__ __forceinline__ bool pair_wait_w(uint64_t* bar, uint32_t parity, volatile int* abort,
                                            int* status, uint64_t budget_ns) {
    const uint32_t addr = smem_u32(bar);
    bool ok = false;
    uint64_t t0 = 0;
    for (uint32_t poll = 1; !ok; ++poll) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(addr), "r"(parity)
            : "memory");
        ok = __shfl_sync(0xffffffffu, done, 0) != 0;
        if (!ok && (poll & 31u) == 0u) {
            if (t0 == 0) t0 = globaltimer_ns();
            int give_up = *abort;
            if (!give_up && globaltimer_ns() - t0 > budget_ns) {
                record_status(status, NVFP4_ERR_TIMEOUT);
                *abort = 1;
                give_up = 1;
            }
            if (__shfl_sync(0xffffffffu, give_up, 0)) break;
        }
    }
    return ok;
}

// Tile order: supertiles of eight row blocks, walked column block by column block, so the
// 74 tiles in flight share about as many panels of A as of B (8192^3 int8: 685 MB of DRAM
// reads when they walked whole rows of tiles, the operands being 134 MB).
struct Item {
    int m_blk, n0;             // row block; first column
    bool half;                 // 128 columns instead of 256
};
__device__ __forceinline__ Item pair_item(const PairParams& p, int item) {
    const bool half = item >= p.whole;
    const int tile = half ? p.whole + ((item - p.whole) >> 1) : item;
    const int super = (int)fast_div((uint32_t)tile, p.div_super);
    const int rest = tile - super * P_GROUP * p.n_blocks;
    const int rows = p.m_blocks - super * P_GROUP;
    const int n_blk = rows >= P_GROUP ? rest / P_GROUP : (int)fast_div((uint32_t)rest, p.div_last);
    const int m_blk = super * P_GROUP + rest - n_blk * min(rows, P_GROUP);
    return {m_blk, n_blk * PN + (half ? ((item - p.whole) & 1) * (PN / 2) : 0), half};
}

// How a tile leaves: by TMA without a residual, by TMA with one (both n_out % 8 == 0), or, with
// rows that are not 16-byte multiples, by the lanes (RAGGED).  Each a build of its own: a
// residual tested per value was a quarter of the instructions of a call without one, and the
// lanes' code beside the TMA form cost that its registers (FFN-in with GELU 111 -> 116 us).
enum { OUT_PLAIN, OUT_RES, OUT_RAGGED };

template <bool I8, int ACT, bool GATED, int OUT>
__global__ void __launch_bounds__(PTHREADS, 1)
gemm_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmBh, const __grid_constant__ CUtensorMap tmSFA,
                 const __grid_constant__ CUtensorMap tmSFB, const __grid_constant__ CUtensorMap tmY,
                 const __grid_constant__ CUtensorMap tmR, const PairParams p) {
    using SM = PairSmem<I8>;
    constexpr bool RES = OUT == OUT_RES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    uint8_t* sStg = smem + PSTAGES * SM::STAGE;
    uint8_t* sCols = sStg + PEPI * 2 * P_STG;
    uint64_t* full = reinterpret_cast<uint64_t*>(sCols + PEPI * SM::COLS);   // used in the leader
    uint64_t* empty = full + PSTAGES;
    uint64_t* acc_full = empty + PSTAGES;    // [2]
    uint64_t* acc_free = acc_full + 2;       // [2], used in the leader
    uint64_t* ovl_free = acc_free + 2;       // used in the leader
    uint64_t* drain = ovl_free + 1;
    uint64_t* res_full = drain + 1;          // [PEPI][2]
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(res_full + 2 * PEPI);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int pair = (int)blockIdx.x >> 1, pairs = (int)gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < PSTAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_free[b], PEPI);          // a group of both CTAs
        }
        mbar_init(ovl_free, 2 * PEPI / 4);
        mbar_init(drain, 1);
        for (int s = 0; s < 2 * PEPI; ++s) mbar_init(&res_full[s], 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
            smem_u32(tmem_holder)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();          // both CTAs' barriers and tensor memory exist
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    // Producer: one stage's B side (box and scales) and A side.
    const uint32_t full0 = dsmem_addr(smem_u32(full), 0);    // the leader's full barriers
    auto load_b = [&](int stage, int kt, const Item& w) {
        const uint32_t s = smem_u32(smem + stage * SM::STAGE), bar = full0 + 8u * (uint32_t)stage;
        const uint32_t sf = s + 2 * PS_OP + PS_SFA;
        if (w.half) tma_load_2d_pair_w(s + PS_OP, &tmBh, bar, kt * PKB, w.n0 + rank * (PROWS / 2));
        else tma_load_2d_pair_w(s + PS_OP, &tmB, bar, kt * PKB, w.n0 + rank * PROWS);
        if constexpr (!I8) {
            // 512-byte scale chunks of the tile's 128-row halves, four K steps each
            const int h = w.n0 >> 7, n_blk = w.n0 >> 8;
            const int at = p.prepared ? (n_blk * p.k_tiles + kt) * 8 + (h & 1) * 4 : 4 * kt;
            const int tile = p.prepared ? 0 : h;
            tma_load_3d_pair_w(sf, &tmSFB, bar, 0, at, tile);
            if (!w.half)
                tma_load_3d_pair_w(sf + 2048, &tmSFB, bar, 0, at + (p.prepared ? 4 : 0),
                                   tile + (p.prepared ? 0 : 1));
        }
    };
    auto load_a = [&](int stage, int kt, const Item& w) {
        const uint32_t s = smem_u32(smem + stage * SM::STAGE), bar = full0 + 8u * (uint32_t)stage;
        tma_load_2d_pair_w(s, &tmA, bar, kt * PKB, w.m_blk * 2 * PROWS + rank * PROWS);
        if constexpr (!I8)
            tma_load_3d_pair_w(s + 2 * PS_OP, &tmSFA, bar, 0, 4 * kt, 2 * w.m_blk + rank);
    };
    // both CTAs' bytes of a stage
    auto stage_bytes = [&](const Item& w) -> uint32_t {
        return 2u * (SM::STAGE - (w.half ? PS_OP / 2 + (I8 ? 0 : PS_SFB / 2) : 0));
    };
    int n_early = 0;
    if (warp == 0) {
        if (lane == 0) {
            prefetch_tensormap(&tmA);
            prefetch_tensormap(&tmB);
        }
        if (p.w_early && pair < p.items) {
            const Item w = pair_item(p, pair);
            n_early = min(PSTAGES, p.k_tiles);
            for (int i = 0; i < n_early; ++i) {
                if (rank == 0) mbar_arrive_expect_tx_w(&full[i], stage_bytes(w));
                load_b(i, i, w);
            }
        }
    }
    griddep_wait();
    griddep_launch_dependents();

    if (warp == 0) {
        int stage = 0, fills = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int item = pair; ok && item < p.items; item += pairs) {
            const Item w = pair_item(p, item);
            for (int kt = 0; kt < p.k_tiles; ++kt, ++fills) {
                if (fills >= n_early) {
                    if (!pair_wait_w(&empty[stage], phase ^ 1, abort_flag, p.status,
                                                p.budget_ns)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx_w(&full[stage], stage_bytes(w));
                    load_b(stage, kt, w);
                }
                load_a(stage, kt, w);
                if (++stage == PSTAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        // Every fill is consumed by an MMA before the epilogue ends; only after a wait that
        // ran out can copies still be on their way, and they land within microseconds.
        if (!ok) {
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 2000000) {}
        }
    } else if (warp == 1) {
        if (rank == 0) {
            int stage = 0, it = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int item = pair; ok && item < p.items; item += pairs, ++it) {
                const int b = it & 1;
                const uint32_t use = (uint32_t)(it >> 1);
                if (!pair_wait_w(&acc_free[b], (use & 1) ^ 1, abort_flag, p.status, p.budget_ns) ||
                    (!I8 && !pair_wait_w(ovl_free, (uint32_t)(it & 1) ^ 1, abort_flag, p.status,
                                            p.budget_ns))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t acc = tmem + (b ? (I8 ? 256u : 192u) : 0u);
                // One loop for each width, and in it four K steps to every stage, without a branch
                // or a running index: whatever comes between two steps is time the tensor pipe
                // waits.  In a loop of nothing else a 128-cycle step took 204 with a test against
                // the end of K before each step and the scale slot taken from a ring, 169 with a
                // second path for the last stage, and 134 like this.  Past the end of K both
                // operands are zero (TMA's fill); their scales there are the next row tile's or
                // zero, so the steps add nothing.
                auto mainloop = [&](auto width) {
                    constexpr bool HALF = decltype(width)::value;
                    for (int kt = 0; kt < p.k_tiles; ++kt) {
                        if (!pair_wait_w(&full[stage], phase, abort_flag, p.status, p.budget_ns)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t s = smem_u32(smem + stage * SM::STAGE);
                        const uint64_t ad = sdesc_kmajor_sw128(s), bd = sdesc_kmajor_sw128(s + PS_OP);
                        const uint64_t sad = sdesc_sf(s + 2 * PS_OP);
                        const uint64_t sbd = sdesc_sf(s + 2 * PS_OP + PS_SFA);
                        auto step = [&](int kk, uint32_t accumulate) {
                            if constexpr (I8)
                                pair_step_i8_w<HALF>(acc, ad + 2 * kk, bd + 2 * kk, accumulate);
                            else
                                pair_step_fp4_w<HALF>(acc, ad + 2 * kk, bd + 2 * kk,
                                                      tmem + PTMEM_SF + 12u * (uint32_t)kk, sad + 32 * kk,
                                                      sbd + 32 * kk, accumulate);
                        };
                        step(0, kt > 0 ? 1u : 0u);
                        step(1, 1u);
                        step(2, 1u);
                        step(3, 1u);
                        commit_both_w(&empty[stage]);
                        if (++stage == PSTAGES) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                };
                if (item >= p.whole) mainloop(std::true_type{});
                else mainloop(std::false_type{});
                if (!ok) break;
                commit_both_w(&acc_full[b]);
            }
            // every tensor-core operation of the pair has finished
            commit_own_w(drain);
            volatile int no_abort = 0;
            pair_wait_w(drain, 0, &no_abort, p.status, p.budget_ns);
        }
        __syncwarp();
    } else {
        const int e = warp - 2;
        const int group = e >> 3;                // tiles group, group + 2, ... of the pair
        const int quad = warp & 3;               // tensor-memory lanes 32 quad .. + 31
        const int half = (e >> 2) & 1;           // columns 128 half .. + 127
        uint8_t* stg = sStg + e * 2 * P_STG;
        float* sbias = reinterpret_cast<float*>(sCols + e * SM::COLS);   // 128 bias values
        float* ssw = sbias + 128;                                        // 128 column scales (int8)
        uint64_t* rfull = res_full + 2 * e;
        const int b = group;                     // this group's accumulator buffer
        const uint32_t free_b = dsmem_addr(smem_u32(&acc_free[b]), 0);
        const uint32_t ovl0 = dsmem_addr(smem_u32(ovl_free), 0);
        // The columns that the FP4 buffers share are buffer 0's last 64 and buffer 1's first:
        // their owners read that part first.
        const int part0 = (!I8 && b == 0 && half == 1) ? 1 : 0;
        const bool owns_shared = !I8 && half == 1 - b;
        const float alpha = I8 ? 0.0f : *p.alpha;
        uint32_t res_phase = 0, res_ahead = 0;   // per staging tile: parity; loaded, not used
        // Loads the residual chunks of the warp's part of a tile (rows from row, columns from
        // n0) into the staging tiles that its output will take: chunk c in staging tile c (one
        // chunk when gated).
        auto load_residual = [&](int row, int n0) {
#pragma unroll
            for (int c = 0; c < (GATED ? 1 : 2); ++c) {
                const int col = GATED ? n0 >> 1 : n0 + 32 * c;
                if (col >= p.n_out) continue;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&rfull[c], P_STG);
                    tma_load_2d(stg + c * P_STG, &tmR, &rfull[c], col, row);
                }
                res_ahead |= 1u << c;
            }
        };
        // This lane's four columns of a tile (bias, scale) and its row's scale, fetched a tile
        // ahead.  Columns past N repeat the last one; they are not stored.
        float4 sw4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f), bias4 = sw4;
        float row_scale = alpha;
        auto fetch_columns = [&](int row, int n0) {
            const int n = n0 + 4 * lane;
            const bool whole = n + 4 <= p.N;
            if (p.bias) {
                uint2 w;
                if (whole) {
                    w = *reinterpret_cast<const uint2*>(p.bias + n);
                } else {
                    w.x = (uint32_t)p.bias[min(n, p.N - 1)] | ((uint32_t)p.bias[min(n + 1, p.N - 1)] << 16);
                    w.y = (uint32_t)p.bias[min(n + 2, p.N - 1)] | ((uint32_t)p.bias[min(n + 3, p.N - 1)] << 16);
                }
                bias4 = make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
            }
            if constexpr (I8) {
                if (whole) sw4 = *reinterpret_cast<const float4*>(p.sw + n);
                else sw4 = make_float4(p.sw[min(n, p.N - 1)], p.sw[min(n + 1, p.N - 1)],
                                       p.sw[min(n + 2, p.N - 1)], p.sw[min(n + 3, p.N - 1)]);
                row_scale = row + lane < p.M ? p.sx[row + lane] : 0.0f;
            }
        };
        int next_row = 0, next_n0 = 0;           // the warp's part of its next tile
        auto next_part = [&](int item) {
            const Item w = pair_item(p, item);
            next_row = w.m_blk * 2 * PROWS + rank * PROWS + quad * 32;
            // half an item has no columns for the second half's warps
            next_n0 = half == 0 ? w.n0 : w.half ? p.N : w.n0 + 128;
        };
        const int first = pair + group * pairs, stride = 2 * pairs;
        if (first < p.items) {
            next_part(first);
            if (RES) load_residual(next_row, next_n0 + 64 * part0);
            fetch_columns(next_row, next_n0);
        }
        uint32_t use = 0;
        bool ok = true;
        for (int item = first; ok && item < p.items; item += stride, ++use) {
            const int row0 = next_row, tile_n0 = next_n0;
            const bool more = item + stride < p.items;
            __syncwarp();                        // the last tile's values have been read
            if (I8) reinterpret_cast<float4*>(ssw)[lane] = sw4;
            reinterpret_cast<float4*>(sbias)[lane] = bias4;
            const float scale = row_scale;
            __syncwarp();
            if (!pair_wait_w(&acc_full[b], use & 1, abort_flag, p.status, p.budget_ns)) {
                ok = false;
                break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                const int part = part0 ^ i;
                const int n0 = tile_n0 + 64 * part;
                uint32_t r[2][32];
                const uint32_t at = tmem + ((uint32_t)(quad * 32) << 16) + (b ? (I8 ? 256u : 192u) : 0u) +
                                    (uint32_t)(half * 128 + part * 64);
                tmem_ld32(at, r[0]);
                tmem_ld32(at + 32, r[1]);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (i == 0 && owns_shared) arrive_cluster(ovl0);
                    if (i == 1) arrive_cluster(free_b);
                }
                if (i == 0 && more) {
                    next_part(item + stride);
                    fetch_columns(next_row, next_n0);
                }

                // Eight columns 8 g .. 8 g + 7 of chunk c: scale, bias, activation.
                auto columns8 = [&](int c, int g, float (&v)[8]) {
                    const float4* b4 = reinterpret_cast<const float4*>(sbias) + 16 * part + 8 * c + 2 * g;
                    const float4* s4 = reinterpret_cast<const float4*>(ssw) + 16 * part + 8 * c + 2 * g;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float4 bb = b4[q];
                        float2 lo, hi;
                        if constexpr (I8) {
                            const float4 ss = s4[q];
                            lo = make_float2(__int2float_rn((int)r[c][8 * g + 4 * q]),
                                             __int2float_rn((int)r[c][8 * g + 4 * q + 1]));
                            hi = make_float2(__int2float_rn((int)r[c][8 * g + 4 * q + 2]),
                                             __int2float_rn((int)r[c][8 * g + 4 * q + 3]));
                            lo = mul2_rn(mul2_rn(lo, make_float2(scale, scale)), make_float2(ss.x, ss.y));
                            hi = mul2_rn(mul2_rn(hi, make_float2(scale, scale)), make_float2(ss.z, ss.w));
                        } else {
                            lo = make_float2(__uint_as_float(r[c][8 * g + 4 * q]),
                                             __uint_as_float(r[c][8 * g + 4 * q + 1]));
                            hi = make_float2(__uint_as_float(r[c][8 * g + 4 * q + 2]),
                                             __uint_as_float(r[c][8 * g + 4 * q + 3]));
                            lo = mul2_rn(lo, make_float2(scale, scale));
                            hi = mul2_rn(hi, make_float2(scale, scale));
                        }
                        v[4 * q] = __fadd_rn(lo.x, bb.x);
                        v[4 * q + 1] = __fadd_rn(lo.y, bb.y);
                        v[4 * q + 2] = __fadd_rn(hi.x, bb.z);
                        v[4 * q + 3] = __fadd_rn(hi.y, bb.w);
                    }
                    activate<ACT, GATED>(v);
                };
                // Output values 8 o .. 8 o + 7 of chunk c: one 8-column group, or, gated, the even
                // places of two.
                auto outputs8 = [&](int c, int o, float (&u)[8]) {
                    if constexpr (GATED) {
                        float v[8];
                        columns8(o >> 1, 2 * (o & 1), v);
#pragma unroll
                        for (int j = 0; j < 4; ++j) u[j] = v[2 * j];
                        columns8(o >> 1, 2 * (o & 1) + 1, v);
#pragma unroll
                        for (int j = 0; j < 4; ++j) u[4 + j] = v[2 * j];
                    } else {
                        columns8(c, o, u);
                    }
                };
                if constexpr (OUT != OUT_RAGGED) {
                    bool stored = false;
#pragma unroll
                    for (int c = 0; c < (GATED ? 1 : 2); ++c) {
                        const int col = GATED ? n0 >> 1 : n0 + 32 * c;
                        if (!ok || col >= p.n_out) continue;     // warp-uniform
                        uint8_t* sb = stg + c * P_STG;
                        if (RES) {
                            ok = pair_wait_w(&rfull[c], (res_phase >> c) & 1, abort_flag, p.status, p.budget_ns);
                            if (!ok) continue;
                            res_phase ^= 1u << c;
                            res_ahead &= ~(1u << c);
                        }
                        // 64-byte swizzle: 16-byte piece o of row r sits at o ^ ((r >> 1) & 3)
#pragma unroll
                        for (int o = 0; o < 4; ++o) {
                            float u[8];
                            outputs8(c, o, u);
                            uint4* to = reinterpret_cast<uint4*>(sb + lane * 64 + ((o ^ ((lane >> 1) & 3)) << 4));
                            uint32_t w[4];
                            if (RES) {
                                const uint4 t = *to;
                                const uint32_t rw[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    u[2 * j] = __fadd_rn(u[2 * j], bf16lo(rw[j]));
                                    u[2 * j + 1] = __fadd_rn(u[2 * j + 1], bf16hi(rw[j]));
                                }
                            } else if (c == 0 && o == 0) {
                                // the last part's stores have read the staging tiles
                                if (lane == 0) bulk_wait_read<0>();
                                __syncwarp();
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j) w[j] = bf16x2_rn(u[2 * j], u[2 * j + 1]);
                            *to = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        stored = true;
                    }
                    if (stored) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            tma_store_2d(&tmY, stg, GATED ? n0 >> 1 : n0, row0);
                            if (!GATED && n0 + 32 < p.n_out) tma_store_2d(&tmY, stg + P_STG, n0 + 32, row0);
                            bulk_commit();
                        }
                    }
                    if (ok && RES && (i == 0 || more)) {
                        if (lane == 0) bulk_wait_read<0>();
                        __syncwarp();
                        if (i == 0) load_residual(row0, tile_n0 + 64 * (part0 ^ 1));
                        else load_residual(next_row, next_n0 + 64 * part0);
                    }
                } else {
                    // Rows of y are not 16-byte multiples, so TMA cannot store them.  The values of
                    // a chunk go through the staging tiles in fp32 (4 KiB), where 16-byte piece o
                    // of row r sits at o ^ (r & 7), and leave in rows of neighbouring columns:
                    // straight from the accumulator each lane would write its own row, 32 sectors
                    // an instruction, with the residual's loads held up by the stores before
                    // them (the residual may be y).  8538 x 6230 x 3584 FP4 537 -> 107 us (6232
                    // columns: 93), with a residual 839 -> 126; 531 x 8982 x 416 int8 104 -> 18.5
                    // (8984: 13.6), 8981 columns 105 -> 35.
                    const int rows = min(32, p.M - row0);
#pragma unroll
                    for (int c = 0; c < (GATED ? 1 : 2); ++c) {
                        const int col = GATED ? n0 >> 1 : n0 + 32 * c;
                        if (col >= p.n_out || rows <= 0) continue;    // warp-uniform
                        __syncwarp();                                 // the last chunk has been read
#pragma unroll
                        for (int o = 0; o < 4; ++o) {
                            float u[8];
                            outputs8(c, o, u);
#pragma unroll
                            for (int q = 0; q < 2; ++q)
                                *reinterpret_cast<float4*>(stg + lane * 128 + (((2 * o + q) ^ (lane & 7)) << 4)) =
                                    make_float4(u[4 * q], u[4 * q + 1], u[4 * q + 2], u[4 * q + 3]);
                        }
                        __syncwarp();
                        const size_t to0 = (size_t)row0 * p.n_out + col;
                        const uint16_t* res = p.residual;
                        if (p.n_out & 1) {
                            // one value a lane, a row at a time; eight rows' loads in flight (with
                            // sixteen 8538 x 6229 x 3584 takes 175 us, with eight 113)
                            const bool mine = col + lane < p.n_out;
#pragma unroll 1
                            for (int r8 = 0; r8 < rows; r8 += 8) {
                                uint32_t t[8];
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    t[k] = res && mine && r8 + k < rows
                                               ? res[to0 + (size_t)(r8 + k) * p.n_out + lane] : 0u;
#pragma unroll
                                for (int k = 0; k < 8; ++k) {
                                    float u = *reinterpret_cast<const float*>(
                                        stg + (r8 + k) * 128 + (((lane >> 2) ^ k) << 4) + (lane & 3) * 4);
                                    if (res) u = __fadd_rn(u, bf16lo(t[k]));
                                    if (mine && r8 + k < rows)
                                        p.y[to0 + (size_t)(r8 + k) * p.n_out + lane] = (uint16_t)bf16x2_rn(u, 0.0f);
                                }
                            }
                        } else {
                            // two values a lane, two rows at a time, all loads in flight (of four
                            // steps' at a time: 531 x 8982 x 416 23.6 us)
                            const int cl = 2 * (lane & 15), rl = lane >> 4;
                            const bool mine = col + cl < p.n_out;
                            uint32_t t[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                t[k] = res && mine && 2 * k + rl < rows
                                           ? *reinterpret_cast<const uint32_t*>(
                                                 res + to0 + (size_t)(2 * k + rl) * p.n_out + cl)
                                           : 0u;
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const int r = 2 * k + rl;
                                float2 u = *reinterpret_cast<const float2*>(
                                    stg + r * 128 + (((cl >> 2) ^ (r & 7)) << 4) + (cl & 3) * 4);
                                if (res) {
                                    u.x = __fadd_rn(u.x, bf16lo(t[k]));
                                    u.y = __fadd_rn(u.y, bf16hi(t[k]));
                                }
                                if (mine && r < rows)
                                    *reinterpret_cast<uint32_t*>(p.y + to0 + (size_t)r * p.n_out + cl) =
                                        bf16x2_rn(u.x, u.y);
                            }
                        }
                    }
                }
            }
        }
        // residual chunks still on their way must land before the block can exit
#pragma unroll
        for (int s = 0; s < 2; ++s)
            if (res_ahead & (1u << s)) {
                volatile int no_abort = 0;
                pair_wait_w(&rfull[s], (res_phase >> s) & 1, &no_abort, p.status, p.budget_ns);
            }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }

    // Every thread gets here after bounded work.  The barrier keeps both CTAs' shared and
    // tensor memory alive until neither is used by the other.
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

}  // namespace

bool make_scale_map(CUtensorMap* map, const void* base, int64_t chunks, int64_t tiles) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {128, (cuuint64_t)chunks, (cuuint64_t)tiles};
    cuuint64_t strides[2] = {512, (cuuint64_t)chunks * 512};
    cuuint32_t box[3] = {128, 4, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_INT32, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

using PairKernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap,
                            CUtensorMap, CUtensorMap, PairParams);

template <bool I8, bool GATED, int OUT>
PairKernel pair_kernel_of(int base) {
    static const PairKernel table[5] = {gemm_pair_kernel<I8, NVFP4_ACT_NONE, GATED, OUT>,
                                        gemm_pair_kernel<I8, NVFP4_ACT_RELU, GATED, OUT>,
                                        gemm_pair_kernel<I8, NVFP4_ACT_GELU, GATED, OUT>,
                                        gemm_pair_kernel<I8, NVFP4_ACT_GELU_TANH, GATED, OUT>,
                                        gemm_pair_kernel<I8, NVFP4_ACT_SILU, GATED, OUT>};
    return table[base];
}

template <bool I8, bool GATED>
PairKernel pair_kernel_of(int base, int out) {
    if (out == OUT_RES) return pair_kernel_of<I8, GATED, OUT_RES>(base);
    if (out == OUT_RAGGED) return pair_kernel_of<I8, GATED, OUT_RAGGED>(base);
    return pair_kernel_of<I8, GATED, OUT_PLAIN>(base);
}

template <bool I8>
PairKernel pair_kernel(int activation, int out) {
    const int base = activation & ~NVFP4_ACT_GATED;
    return activation & NVFP4_ACT_GATED ? pair_kernel_of<I8, true>(base, out)
                                        : pair_kernel_of<I8, false>(base, out);
}

template <bool I8>
nvfp4_status launch_pair_impl(const GemmActArgs& g, cudaStream_t stream) {
    DeviceInfo dev;
    nvfp4_status st = device_info(&dev);
    if (st != NVFP4_OK) return st;
    int* status = nullptr;
    if ((st = status_word(&status)) != NVFP4_OK) return st;
    PairParams p{};
    const int64_t kbytes = I8 ? g.K : g.K / 2;
    p.alpha = g.alpha;
    p.sx = g.sx;
    p.sw = g.sw;
    p.bias = static_cast<const uint16_t*>(g.bias);
    p.residual = static_cast<const uint16_t*>(g.epi.residual);
    p.y = static_cast<uint16_t*>(g.y);
    p.M = (int)g.M;
    p.N = (int)g.N;
    p.n_out = (int)((g.epi.activation & NVFP4_ACT_GATED) ? g.N / 2 : g.N);
    p.m_blocks = (int)((g.M + 2 * PROWS - 1) / (2 * PROWS));
    p.n_blocks = (int)((g.N + PN - 1) / PN);
    const int tiles = p.m_blocks * p.n_blocks, max_pairs = dev.sms / 2;
    const int last = tiles % max_pairs;        // tiles of the last wave
    p.whole = 2 * last <= max_pairs ? tiles - last : tiles;
    p.items = p.whole + 2 * (tiles - p.whole);
    p.div_super = make_fastdiv((uint32_t)(P_GROUP * p.n_blocks));
    p.div_last = make_fastdiv((uint32_t)(p.m_blocks % P_GROUP ? p.m_blocks % P_GROUP : P_GROUP));
    p.k_tiles = (int)((kbytes + PKB - 1) / PKB);
    p.kchunks = (int)(kbytes / 32);
    p.prepared = g.sfb_prepared ? 1 : 0;
    p.w_early = g.weights_ready ? 1 : 0;
    p.status = status;
    p.budget_ns = 4000000000ull;   // 4 s
    const int out = p.n_out % 8 ? OUT_RAGGED : p.residual ? OUT_RES : OUT_PLAIN;
    const PairKernel kernel = pair_kernel<I8>(g.epi.activation, out);
    static std::atomic<int> attr_set[64][3][32];
    std::atomic<int>& set = attr_set[dev.device & 63][out][g.epi.activation & 31];
    if (!set.load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 PairSmem<I8>::BYTES) != cudaSuccess)
            return NVFP4_ERR_CUDA;
        set.store(1, std::memory_order_release);
    }
    CUtensorMap mapA, mapB, mapBh, mapSFA, mapSFB, mapY, mapR;
    if (!make_operand_map(&mapA, g.a, g.M, kbytes, PROWS) ||
        !make_operand_map(&mapB, g.b, g.N, kbytes, PROWS) ||
        !make_operand_map(&mapBh, g.b, g.N, kbytes, PROWS / 2))
        return NVFP4_ERR_CUDA;
    mapSFA = mapSFB = mapY = mapA;             // where unused
    if (!I8) {
        if (!make_scale_map(&mapSFA, g.sfa, p.kchunks, (g.M + 127) / 128) ||
            !(p.prepared ? make_scale_map(&mapSFB, g.sfb, (int64_t)p.n_blocks * p.k_tiles * 8, 1)
                         : make_scale_map(&mapSFB, g.sfb, p.kchunks, (g.N + 127) / 128)))
            return NVFP4_ERR_CUDA;
    }
    if (out != OUT_RAGGED && !make_output_map(&mapY, g.y, g.M, p.n_out)) return NVFP4_ERR_CUDA;
    mapR = mapY;
    if (out == OUT_RES && !make_output_map(&mapR, const_cast<void*>(g.epi.residual), g.M, p.n_out))
        return NVFP4_ERR_CUDA;

    const int pairs = p.items < max_pairs ? p.items : max_pairs;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs), 1, 1);
    cfg.blockDim = dim3(PTHREADS, 1, 1);
    cfg.dynamicSmemBytes = PairSmem<I8>::BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, mapA, mapB, mapBh, mapSFA, mapSFB, mapY, mapR, p) ==
                   cudaSuccess
               ? NVFP4_OK
               : NVFP4_ERR_CUDA;
}

}  // namespace

nvfp4_status launch_gemm_act(const GemmActArgs& g, cudaStream_t stream) {
    DeviceInfo dev;
    nvfp4_status st = device_info(&dev);
    if (st != NVFP4_OK) return st;
    // A weight whose 256-row tiles leave no SMs to split K over streams through all SMs for up
    // to 32 rows, and for up to 64 when K is long enough (20 stages) to cover the stream
    // kernel's narrow stores.  Against SM pairs, us: 51200 x 5120 FP4 at 1 row 28.2 : 45.8, 64
    // rows 31.9 : 35.4; 20480 x 2560 FP4 (10 stages) 32 rows 11.4 : 13.7, 48 rows 13.0 : 14.1,
    // 64 rows 15.1 : 13.9; 19456 x 512 int8 32 rows 7.6 : 9.3, 48 rows 10.0 : 9.4.
    const bool long_weight = (g.N + 255) / 256 * 2 > dev.sms;
    const int64_t stages = ((g.int8 ? g.K : g.K / 2) + 127) / 128;
    if (long_weight && (g.M <= kSmallMaxRows || (g.M <= kStreamMaxRows && stages >= 20)))
        return launch_gemm_stream(g, stream);
    if (g.M <= kSmallMaxRows) return launch_gemm_small_act(g, stream);
    bool taken = false;
    st = launch_gemm_act_split_k(g, &taken, stream);
    if (st != NVFP4_OK || taken) return st;
    return g.int8 ? launch_pair_impl<true>(g, stream) : launch_pair_impl<false>(g, stream);
}

}  // namespace nvfp4
