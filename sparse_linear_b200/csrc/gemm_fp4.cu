// Product of two microscaled 4-bit operands on the block-scaled tensor cores:
// tcgen05.mma kind::mxf4nvf4, K = 64 per instruction, E2M1 codes packed two
// per byte in shared memory (128-byte swizzle, 256 channels per 128-byte row),
// scales in tensor memory (scale_vec::4X: four E4M3 scales of 16 channels,
// scale_vec::2X: two E8M0 scales of 32).
//
// Scales.  A 512-byte tile of the scale buffer (128 rows x 4 blocks) is what
// tcgen05.cp.32x128b.warpx4 moves into four tensor-memory columns: row r of
// the tile at lane r % 32 (repeated in each quarter of the lanes), column
// r / 32, its four blocks in the column's bytes.  One tile covers one
// instruction (NV) or two (MX: bytes 0-1, then 2-3, by the scale id of the
// instruction descriptor).  256 rows of B take eight consecutive columns.
//
// k_gemm_fp4_pair   long prompts: 256 x 256 tiles on CTA pairs, as
//                   k_gemm_dense_pair; each CTA holds its own 128 rows of A
//                   with their scales, half of B, and all of B's scales.
//                   Its scales go to tensor memory through the registers of
//                   four warps (tcgen05.st), not by tcgen05.cp: a stage needs
//                   12 copies of about 45 clocks beside 512 clocks of MMAs,
//                   and the two overlap only in part (717 clocks together);
//                   the stores leave the MMAs at 513.  An SM takes in about
//                   53 bytes per clock, 38 KB per stage: 4096 x 14336 x 4096
//                   NV runs in 100 us (4.8 PFLOP/s), 777 x 11008 x 4096 MX in
//                   21.5 us (MMAs 11 us, operands 15 us), calls one after
//                   another with cold operands.
// k_gemm_fp4_few    few tokens: the weights are the M = 128 operand and the
//                   tokens the N operand, so that every SM streams weights; K
//                   is split over the CTAs of a cluster, whose sums are added
//                   through distributed shared memory in rank order.  Bound
//                   by latency (launch, first loads, exchange): 16 x 4096 x
//                   4096 6.3 us, 512 x 1024 x 4096 7.5 us; by the weights
//                   when they are many: 16 x 14336 x 14336 24 us (4.8 TB/s).
// No load uses cluster multicast.  Every mbarrier wait is bounded.
#include "common.cuh"
#include "fp4.cuh"
#include "kernels.cuh"

namespace as {

// The issuing warp runs its loop as a whole and every tcgen05 instruction is
// predicated on one elected lane (`lead`): addresses and descriptors then stay
// in uniform registers.  Issued from a branch of one lane each instruction cost
// some 90 clocks of moves.
__device__ __forceinline__ uint32_t elect_lane()
{
    uint32_t lead;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(lead));
    return lead;
}

// Index of this warp, known to be the same in all its lanes.
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0); }

// D[tmem] (+)= (A * scales) (B * scales)^T; PAIR: over a CTA pair.
#define AS_MMA_FP4(GROUP, VEC)                                                                                    \
    asm volatile(                                                                                                 \
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"                            \
        "@q tcgen05.mma.cta_group::" GROUP ".kind::mxf4nvf4.block_scale.scale_vec::" VEC                            \
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa),     \
        "r"(sfb), "r"(accumulate), "r"(lead)                                                                       \
        : "memory")
template <int FMT, bool PAIR>
__device__ __forceinline__ void mma_fp4(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t accumulate)
{
    if constexpr (PAIR && FMT == AS_FP4_NV) AS_MMA_FP4("2", "4X");
    else if constexpr (PAIR) AS_MMA_FP4("2", "2X");
    else if constexpr (FMT == AS_FP4_NV) AS_MMA_FP4("1", "4X");
    else AS_MMA_FP4("1", "2X");
}
#undef AS_MMA_FP4

// 512 bytes (32 rows x 16 bytes) of shared memory -> 4 TMEM columns, repeated
// in the four lane quarters.
__device__ __forceinline__ void tmem_cp_sf(uint32_t lead, uint32_t taddr, uint64_t s_desc)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
                 "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(s_desc), "r"(lead)
                 : "memory");
}

// Arrive on `bar` (PAIR: in both CTAs) once this lane's tcgen05 operations so
// far have completed.
template <bool PAIR>
__device__ __forceinline__ void tc_commit_lead(uint32_t lead, uint64_t *bar)
{
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], "
            "%1;\n\t}" ::"r"(smem_u32(bar)), "h"((uint16_t)3), "r"(lead)
            : "memory");
    else
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
                     "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
                         smem_u32(bar)),
                     "r"(lead)
                     : "memory");
}

// Instruction descriptor of kind::mxf4nvf4: A and B format code 1 (E2M1) in
// [7,10) and [10,13), N >> 3 in [17,23), scale format in bit 23 (0 E4M3, 1
// E8M0), M >> 7 in [27,29); the scale ids of B in [4,6) and of A in [29,31)
// are added per instruction.
template <int FMT>
__host__ __device__ constexpr uint32_t idesc_fp4(int M, int N)
{
    return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (FMT == AS_FP4_MX ? 1u << 23 : 0u) |
           ((uint32_t)(M >> 7) << 27);
}

template <int FMT>
struct Fp4Cfg {
    static constexpr int KB = 256;                         // channels per stage
    static constexpr int SFT = FMT == AS_FP4_NV ? 4 : 2;   // scale tiles per stage and 128 rows
    static constexpr int SFB = SFT * 512;                  // their bytes
    // tile and scale id of instruction j (64 channels) of a stage
    __device__ static constexpr int tile(int j) { return FMT == AS_FP4_NV ? j : j >> 1; }
    __device__ static constexpr uint32_t ids(int j)
    {
        return FMT == AS_FP4_NV ? 0u : (((uint32_t)(j & 1) * 2u) << 4) | (((uint32_t)(j & 1) * 2u) << 29);
    }
};

struct Fp4Params {
    const float *x_scale, *w_scale;
    void *y;
    int T, K, n_out, out_bf16;
    int m_tiles, n_tiles, k_blocks, kt;
};

// ------------------------------------------------------------- CTA pairs
//   warp 0       TMA producer of A and B (both CTAs' bytes count on the
//                leader's barrier).
//   warp 1       tensor-memory allocation; lane 0 of the leader issues MMAs.
//   warps 2-9    epilogue: (lane quarter, column half) per warp.
//   warps 10-13  scales: shared memory -> registers -> tensor memory, then an
//                arrival on the leader's full barrier (both CTAs' warps).
//   warp 14      TMA producer of the scales.
// The scales have a shared-memory ring of their own (FP_SF slots), so that
// they are at hand when a stage (and its slot in tensor memory) is freed.
constexpr int FP_STAGES = 5;
constexpr int FP_SF = 8;
constexpr int FP_THREADS = 480;
template <int FMT>
struct FpPair {
    static constexpr int A = 128 * 128, B = 128 * 128;
    static constexpr int SA = Fp4Cfg<FMT>::SFB, SB = 2 * Fp4Cfg<FMT>::SFB;
    static constexpr int SCOLS = 12 * Fp4Cfg<FMT>::SFT;  // TMEM columns of scales per K block
    static constexpr size_t smem = 1024 + (size_t)FP_STAGES * (A + B) + (size_t)FP_SF * (SA + SB) + 256;
    static_assert(PAIR_BN + FP_STAGES * SCOLS <= 512, "tensor memory");
};

// 32 lanes x N columns from N registers.
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t *r)
{
    if constexpr (N == 8)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                     "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    else {
        static_assert(N == 16, "8 or 16 columns");
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::
                "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
            : "memory");
    }
}

template <int FMT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(FP_THREADS, 1)
    k_gemm_fp4_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB, Fp4Params p)
{
    using C = Fp4Cfg<FMT>;
    using P = FpPair<FMT>;
    constexpr int S = FP_STAGES;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                            ~uintptr_t(1023));
    unsigned char *sA = smem, *sB = sA + S * P::A, *sSA = sB + S * P::B, *sSB = sSA + FP_SF * P::SA;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sSB + FP_SF * P::SB);
    uint64_t *full = bars, *empty = full + S;                // A and B
    uint64_t *sf_land = empty + S, *sf_read = sf_land + FP_SF;    // scales in shared memory
    uint64_t *acc_full = sf_read + FP_SF, *acc_empty = acc_full + 1, *drain = acc_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);
    __shared__ __align__(16) float s_ws[8][128];  // every epilogue warp's weight row scales

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int num_tiles = p.m_tiles * p.n_tiles;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 9);     // the leader's expect_tx arrival (+ both CTAs' bytes), 8 scale warps
            mbar_init(&empty[s], 1);    // one commit from the leader's MMA thread
        }
        for (int s = 0; s < FP_SF; ++s) {
            mbar_init(&sf_land[s], 1);  // own expect_tx arrival (+ own scale bytes)
            mbar_init(&sf_read[s], 4);  // own scale warps
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 16);  // 8 epilogue warps in each CTA (the leader's copy is used)
        mbar_init(drain, 1);  // the leader's last commit
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
        prefetch_tensormap(&tmSA);
        prefetch_tensormap(&tmSB);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync_all();  // barriers of both CTAs initialised before either uses the other's
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            for (int tile = pair; tile < num_tiles && !*(volatile int *)abort_flag; tile += npairs) {
                int mt, nt;
                tile_coords(tile, p.m_tiles, p.n_tiles, mt, nt);
                const int arow = mt * PAIR_BM + 128 * (int)rank;
                const int brow = nt * PAIR_BN + 128 * (int)rank;
                for (int kb = 0; kb < p.k_blocks; ++kb) {
                    if (!mbar_wait(&empty[stage], phase ^ 1)) { *(volatile int *)abort_flag = 1; break; }
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * (P::A + P::B));
                    const uint32_t bar = mapa_u32(smem_u32(&full[stage]), 0);
                    tma_load_2d_pair(sA + stage * P::A, &tmA, bar, kb * 128, arow);
                    tma_load_2d_pair(sB + stage * P::B, &tmB, bar, kb * 128, brow);
                    if (++stage == S) { stage = 0; phase ^= 1; }
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (leader only)
        if (rank == 0) {
            const uint32_t lead = elect_lane();
            constexpr uint32_t idesc = idesc_fp4<FMT>(PAIR_BM, PAIR_BN);
            int stage = 0;
            uint32_t phase = 0;
            int it = 0;
            // A barrier's answer takes some 240 clocks here even when it is
            // ready: the next stage is asked for before this one's MMAs issue.
            // (test_wait, which never suspends and then has to ask again:
            // 777 x 11008 x 4096 22.3 us against 21.5.)
            bool ready = false;
            for (int tile = pair; tile < num_tiles && !*(volatile int *)abort_flag; tile += npairs, ++it) {
                if (!mbar_wait(acc_empty, (it & 1) ^ 1)) { *(volatile int *)abort_flag = 1; break; }
                bool ok = true;
                for (int kb = 0; kb < p.k_blocks; ++kb) {
                    if (!ready && !mbar_wait(&full[stage], phase)) { ok = false; break; }
                    tc_fence_after();
                    const int next = stage + 1 == S ? 0 : stage + 1;
                    const uint32_t nphase = stage + 1 == S ? phase ^ 1 : phase;
                    // not after the pair's last K block: nothing would fill it
                    ready = (kb + 1 < p.k_blocks || tile + npairs < num_tiles) && mbar_try_wait(&full[next], nphase);
                    const int steps = min(4, (p.K - kb * C::KB + 63) >> 6);
                    const uint32_t sfa = tmem + PAIR_BN + stage * P::SCOLS, sfb = sfa + 4 * C::SFT;
                    const uint64_t a_desc = sdesc_kmajor_sw128(smem_u32(sA + stage * P::A));
                    const uint64_t b_desc = sdesc_kmajor_sw128(smem_u32(sB + stage * P::B));
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < steps)
                            mma_fp4<FMT, true>(lead, tmem, a_desc + (uint64_t)((32 * j) >> 4),
                                               b_desc + (uint64_t)((32 * j) >> 4), idesc | C::ids(j),
                                               sfa + 4 * C::tile(j), sfb + 8 * C::tile(j), (kb | j) != 0);
                    tc_commit_lead<true>(lead, &empty[stage]);  // frees the stage and its scales in both CTAs
                    stage = next;
                    phase = nphase;
                }
                if (!ok) { *(volatile int *)abort_flag = 1; break; }
                tc_commit_lead<true>(lead, acc_full);
            }
            tc_commit_lead<true>(lead, drain);
        }
        // Both CTAs: the commits of the leader arrive at both, so neither
        // leaves before the last one has arrived.
        mbar_wait(drain, 0);
    } else if (warp == 14) {
        // ------------------------------------------------ TMA producer of scales
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            for (int tile = pair; tile < num_tiles && !*(volatile int *)abort_flag; tile += npairs) {
                int mt, nt;
                tile_coords(tile, p.m_tiles, p.n_tiles, mt, nt);
                const int sa = (2 * mt + (int)rank) * p.kt, sb = 2 * nt * p.kt;  // scale tiles
                for (int kb = 0; kb < p.k_blocks; ++kb) {
                    if (!mbar_wait(&sf_read[stage], phase ^ 1)) { *(volatile int *)abort_flag = 1; break; }
                    // the scales of the whole K block; tiles past K hold other
                    // rows' scales and are not used
                    mbar_arrive_expect_tx(&sf_land[stage], P::SA + P::SB);
                    tma_load_2d(sSA + stage * P::SA, &tmSA, &sf_land[stage], 0, 2 * (sa + kb * C::SFT));
                    tma_load_2d(sSB + stage * P::SB, &tmSB, &sf_land[stage], 0, 2 * (sb + kb * C::SFT));
                    tma_load_2d(sSB + stage * P::SB + C::SFB, &tmSB, &sf_land[stage], 0,
                                2 * (sb + p.kt + kb * C::SFT));
                    if (++stage == FP_SF) { stage = 0; phase ^= 1; }
                }
            }
        }
    } else if (warp >= 10) {
        // ------------------------------------------------ scales (warps 10..13)
        const int q = warp & 3;
        int stage = 0, slot = 0;
        uint32_t phase = 0, sphase = 0;
        const uint32_t full0 = mapa_u32(smem_u32(full), 0);
        for (int tile = pair; tile < num_tiles && !*(volatile int *)abort_flag; tile += npairs) {
            for (int kb = 0; kb < p.k_blocks; ++kb) {
                if (!mbar_wait(&sf_land[stage], phase)) { *(volatile int *)abort_flag = 1; break; }
                // a tile's 16 bytes of lane l are its columns 0..3; B's two
                // row tiles of one K tile lie side by side in tensor memory
                const unsigned char *a = sSA + stage * P::SA + 16 * lane, *b = sSB + stage * P::SB + 16 * lane;
                uint32_t ra[4 * C::SFT], rb[8 * C::SFT];
#pragma unroll
                for (int t = 0; t < C::SFT; ++t) {
                    *reinterpret_cast<uint4 *>(ra + 4 * t) = *reinterpret_cast<const uint4 *>(a + 512 * t);
                    *reinterpret_cast<uint4 *>(rb + 8 * t) = *reinterpret_cast<const uint4 *>(b + 512 * t);
                    *reinterpret_cast<uint4 *>(rb + 8 * t + 4) =
                        *reinterpret_cast<const uint4 *>(b + C::SFB + 512 * t);
                }
                if (!mbar_wait(&empty[slot], sphase ^ 1)) { *(volatile int *)abort_flag = 1; break; }
                tc_fence_after();
                const uint32_t col = tmem + ((uint32_t)(32 * q) << 16) + PAIR_BN + slot * P::SCOLS;
                tmem_st<4 * C::SFT>(col, ra);
                tmem_st<4 * C::SFT>(col + 4 * C::SFT, rb);
                tmem_st<4 * C::SFT>(col + 8 * C::SFT, rb + 4 * C::SFT);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();  // all lanes have read the slot and written theirs
                if (lane == 0) {
                    mbar_arrive(&sf_read[stage]);
                    mbar_arrive_cluster(full0 + 8u * (uint32_t)slot);
                }
                if (++stage == FP_SF) { stage = 0; phase ^= 1; }
                if (++slot == S) { slot = 0; sphase ^= 1; }
            }
        }
    } else {
        // ------------------------------------------------ epilogue (warps 2..9)
        const int q = warp & 3;           // TMEM lanes 32q..32q+31
        const int h = (warp - 2) >> 2;    // accumulator columns [128h, 128h+128)
        const uint32_t acc_empty_leader = mapa_u32(smem_u32(acc_empty), 0);
        int it = 0;
        for (int tile = pair; tile < num_tiles && !*(volatile int *)abort_flag; tile += npairs, ++it) {
            int mt, nt;
            tile_coords(tile, p.m_tiles, p.n_tiles, mt, nt);
            // the tile's weight row scales, while its MMAs run
            const int col0 = nt * PAIR_BN + 128 * h;
            float *ws = s_ws[warp - 2];
            __syncwarp();  // the last tile's reads
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ws[32 * i + lane] = p.w_scale && col0 + 32 * i + lane < p.n_out ? p.w_scale[col0 + 32 * i + lane] : 1.0f;
            __syncwarp();
            const int row = mt * PAIR_BM + 128 * (int)rank + 32 * q + lane;
            const bool row_ok = row < p.T;
            const float xs = p.x_scale && row_ok ? p.x_scale[row] : 1.0f;
            if (!mbar_wait(acc_full, it & 1)) { *(volatile int *)abort_flag = 1; break; }
            tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16) + 128 * h;
            if (p.out_bf16) {  // rounded in registers, so that the accumulator is free before the stores
                uint32_t out[4][16];
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(taddr + 32 * ch, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 w = *reinterpret_cast<const float2 *>(ws + 32 * ch + 2 * i);
                        const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(r[2 * i]) * xs * w.x,
                                                                       __uint_as_float(r[2 * i + 1]) * xs * w.y);
                        out[ch][i] = *reinterpret_cast<const uint32_t *>(&v);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(acc_empty_leader);
                if (row_ok) {
                    __nv_bfloat16 *yr = static_cast<__nv_bfloat16 *>(p.y) + (size_t)row * p.n_out;
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        if (col0 + 8 * c < p.n_out &&
                            as_in((long long)row * p.n_out + col0 + 8 * c + 7, (long long)p.T * p.n_out))
                            *reinterpret_cast<uint4 *>(yr + col0 + 8 * c) = *reinterpret_cast<uint4 *>(&out[c >> 2][4 * (c & 3)]);
                }
            } else {
#pragma unroll 1
                for (int ch = 0; ch < 4; ++ch) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(taddr + 32 * ch, r);
                    tmem_ld_wait();
                    if (row_ok) {
                        float *yr = static_cast<float *>(p.y) + (size_t)row * p.n_out;
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const int col = col0 + 32 * ch + 4 * c;
                            if (col < p.n_out && as_in((long long)row * p.n_out + col + 3, (long long)p.T * p.n_out)) {
                                const float4 w = *reinterpret_cast<const float4 *>(ws + 32 * ch + 4 * c);
                                *reinterpret_cast<float4 *>(yr + col) =
                                    make_float4(__uint_as_float(r[4 * c]) * xs * w.x,
                                                __uint_as_float(r[4 * c + 1]) * xs * w.y,
                                                __uint_as_float(r[4 * c + 2]) * xs * w.z,
                                                __uint_as_float(r[4 * c + 3]) * xs * w.w);
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(acc_empty_leader);
            }
        }
    }

    // Both CTAs' tensor memory stays allocated until the leader's last MMA
    // has completed and both epilogues have read their accumulators.
    tc_fence_before();
    __syncwarp();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ------------------------------------------------------------ few tokens
// Tile: 128 outputs (M) x N tokens.  Each CTA of a cluster takes a contiguous
// part of the K blocks; one pass, so one accumulator and no accumulator ring.
constexpr int FF_THREADS = 192;
template <int FMT, int N>
struct FpFew {
    static constexpr int A = 128 * 128, B = N * 128;
    static constexpr int NSB = (N + 127) / 128;  // scale row tiles of B
    static constexpr int SA = Fp4Cfg<FMT>::SFB, SB = NSB * Fp4Cfg<FMT>::SFB;
    static constexpr int STAGE = A + B + SA + SB;
    static constexpr int SCOLS = 4 * (1 + NSB) * Fp4Cfg<FMT>::SFT;
    static constexpr int STAGES = N <= 32 ? 8 : (N <= 64 ? 6 : 4);
    static constexpr int RSTR = 128 + 4;                        // reduction row of a token, floats
    static constexpr size_t ring = (size_t)STAGES * STAGE;
    static constexpr size_t red = (size_t)N * RSTR * 4;
    static constexpr size_t smem = 1024 + (ring > red ? ring : red) + 256;
    static constexpr uint32_t TCOLS = N + STAGES * SCOLS <= 256 ? 256 : 512;
    static_assert(N + STAGES * SCOLS <= 512, "tensor memory");
};

// The sum of R CTAs' partial tiles, in rank order.  A warp takes a token's 128
// outputs, 4 per lane, so that its loads cover a peer's row without gaps, and
// two tokens at a time, with the loads from all peers in flight.  R is a
// constant: branches on it between the loads cost more than the loads (one
// CTA, 128 tokens: 6400 clocks).
template <int N, int RSTR, int R>
__device__ __forceinline__ void few_sum(const Fp4Params &p, const float *red, const float *s_xs, const float *s_ws,
                                        int rank, int ot, int tt, int warp, int lane)
{
    const int tn = min(N, p.T - tt * N), col = ot * 128 + 4 * lane;
    constexpr int step = R * (FF_THREADS / 32);
    const float4 ws = *reinterpret_cast<const float4 *>(s_ws + 4 * lane);
    for (int t0 = rank * (FF_THREADS / 32) + warp; t0 < tn; t0 += 2 * step) {
        float4 f[2][R];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float *own = red + min(t0 + k * step, tn - 1) * RSTR + 4 * lane;
            if constexpr (R == 1) {
                f[k][0] = *reinterpret_cast<const float4 *>(own);
            } else if (k == 0 || t0 + k * step < tn) {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(f[k][r].x), "=f"(f[k][r].y), "=f"(f[k][r].z), "=f"(f[k][r].w)
                                 : "r"(mapa_u32(smem_u32(own), (uint32_t)r)));
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int t = t0 + k * step, row = tt * N + t;
            if (t >= tn || col >= p.n_out || !as_in((long long)row * p.n_out + col + 3, (long long)p.T * p.n_out))
                continue;
            float4 v = f[k][0];
#pragma unroll
            for (int r = 1; r < R; ++r) {
                v.x += f[k][r].x; v.y += f[k][r].y; v.z += f[k][r].z; v.w += f[k][r].w;
            }
            const float xs = s_xs[t];
            v.x = v.x * xs * ws.x; v.y = v.y * xs * ws.y; v.z = v.z * xs * ws.z; v.w = v.w * xs * ws.w;
            if (p.out_bf16) {
                const __nv_bfloat162 h0 = __floats2bfloat162_rn(v.x, v.y), h1 = __floats2bfloat162_rn(v.z, v.w);
                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.y) + (size_t)row * p.n_out + col) = make_uint2(
                    *reinterpret_cast<const uint32_t *>(&h0), *reinterpret_cast<const uint32_t *>(&h1));
            } else {
                *reinterpret_cast<float4 *>(static_cast<float *>(p.y) + (size_t)row * p.n_out + col) = v;
            }
        }
    }
}

template <int FMT, int N>
__global__ void __launch_bounds__(FF_THREADS, 1)
    k_gemm_fp4_few(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB, Fp4Params p)
{
    using C = Fp4Cfg<FMT>;
    using P = FpFew<FMT, N>;
    constexpr int S = P::STAGES;
    extern __shared__ unsigned char smem_raw[];
    // the reduction reads the peers' buffers at this CTA's offset: the
    // dynamic window starts at the same address in every CTA of a kernel
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                            ~uintptr_t(1023));
    unsigned char *sA = smem, *sB = sA + S * P::A, *sSA = sB + S * P::B, *sSB = sSA + S * P::SA;
    float *red = reinterpret_cast<float *>(smem);  // after the main loop
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + (P::ring > P::red ? P::ring : P::red));
    uint64_t *full = bars, *empty = bars + S, *done = bars + 2 * S;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * S + 1);
    int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);
    __shared__ float s_xs[N];
    __shared__ __align__(16) float s_ws[128];  // row scales of the tile

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank(), nranks = gridDim.x;
    const int ot = blockIdx.y, tt = blockIdx.z;  // output tile, token tile
    const int per = (p.k_blocks + nranks - 1) / nranks;
    const int kb0 = min(p.k_blocks, rank * per), kb1 = min(p.k_blocks, kb0 + per);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
        prefetch_tensormap(&tmSA);
        prefetch_tensormap(&tmSB);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, P::TCOLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            const int sa = ot * p.kt, sb = tt * P::NSB * p.kt;  // tiles of fewer than 128 tokens: tt is 0
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait(&empty[stage], phase ^ 1)) { *(volatile int *)abort_flag = 1; break; }
                mbar_arrive_expect_tx(&full[stage], P::STAGE);
                tma_load_2d(sA + stage * P::A, &tmA, &full[stage], kb * 128, ot * 128);
                tma_load_2d(sB + stage * P::B, &tmB, &full[stage], kb * 128, tt * N);
                tma_load_2d(sSA + stage * P::SA, &tmSA, &full[stage], 0, 2 * (sa + kb * C::SFT));
#pragma unroll
                for (int c = 0; c < P::NSB; ++c)
                    tma_load_2d(sSB + stage * P::SB + c * C::SFB, &tmSB, &full[stage], 0,
                                2 * (sb + c * p.kt + kb * C::SFT));
                if (++stage == S) { stage = 0; phase ^= 1; }
            }
        }
    } else if (warp == 1) {
        const uint32_t lead = elect_lane();
        constexpr uint32_t idesc = idesc_fp4<FMT>(128, N);
        int stage = 0;
        uint32_t phase = 0;
        bool ready = false;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!ready && !mbar_wait(&full[stage], phase)) { *(volatile int *)abort_flag = 1; break; }
            tc_fence_after();
            const int next = stage + 1 == S ? 0 : stage + 1;
            const uint32_t nphase = stage + 1 == S ? phase ^ 1 : phase;
            // test_wait: this stage's MMAs are ready and do not wait for the next's
            ready = kb + 1 < kb1 && mbar_test(&full[next], nphase);
            const int steps = min(4, (p.K - kb * C::KB + 63) >> 6);
            const uint32_t sfa = tmem + N + stage * P::SCOLS, sfb = sfa + 4 * C::SFT;
#pragma unroll
            for (int t = 0; t < C::SFT; ++t) {
                tmem_cp_sf(lead, sfa + 4 * t, sdesc_rows16(smem_u32(sSA + stage * P::SA + 512 * t)));
#pragma unroll
                for (int c = 0; c < P::NSB; ++c)
                    tmem_cp_sf(lead, sfb + 4 * P::NSB * t + 4 * c,
                               sdesc_rows16(smem_u32(sSB + stage * P::SB + c * C::SFB + 512 * t)));
            }
            const uint64_t a_desc = sdesc_kmajor_sw128(smem_u32(sA + stage * P::A));
            const uint64_t b_desc = sdesc_kmajor_sw128(smem_u32(sB + stage * P::B));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < steps)
                    mma_fp4<FMT, false>(lead, tmem, a_desc + (uint64_t)((32 * j) >> 4), b_desc + (uint64_t)((32 * j) >> 4),
                                        idesc | C::ids(j), sfa + 4 * C::tile(j), sfb + 4 * P::NSB * C::tile(j),
                                        (kb > kb0 || j > 0));
            tc_commit_lead<false>(lead, &empty[stage]);
            stage = next;
            phase = nphase;
        }
        tc_commit_lead<false>(lead, done);  // every MMA above has completed
    }
    // ---- all MMAs done: the accumulator (row = output, column = token) goes
    // to shared memory transposed, over the drained ring
    const bool some = kb1 > kb0;
    bool ok = true;
    if (warp >= 2) {
        for (int i = (int)threadIdx.x - 64; i < 128; i += FF_THREADS - 64)
            s_ws[i] = p.w_scale && ot * 128 + i < p.n_out ? p.w_scale[ot * 128 + i] : 1.0f;
        for (int i = (int)threadIdx.x - 64; i < N; i += FF_THREADS - 64)
            s_xs[i] = p.x_scale && tt * N + i < p.T ? p.x_scale[tt * N + i] : 1.0f;
        ok = mbar_wait(done, 0);
        tc_fence_after();
        const int q = warp & 3;
        if (ok) {
#pragma unroll
            for (int c = 0; c < N / 16; ++c) {
                uint32_t r[16];
                if (some) {
                    asm volatile(
                        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
                          "=r"(r[14]), "=r"(r[15])
                        : "r"(tmem + ((uint32_t)(32 * q) << 16) + 16 * c));
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) r[i] = 0u;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) red[(16 * c + i) * P::RSTR + 32 * q + lane] = __uint_as_float(r[i]);
            }
        }
        tc_fence_before();
    }
    __syncwarp();
    cluster_sync_all();
    tc_fence_after();
    // ---- sum over the cluster and write
    switch (nranks) {
    case 1: few_sum<N, P::RSTR, 1>(p, red, s_xs, s_ws, rank, ot, tt, warp, lane); break;
    case 2: few_sum<N, P::RSTR, 2>(p, red, s_xs, s_ws, rank, ot, tt, warp, lane); break;
    case 3: few_sum<N, P::RSTR, 3>(p, red, s_xs, s_ws, rank, ot, tt, warp, lane); break;
    case 4: few_sum<N, P::RSTR, 4>(p, red, s_xs, s_ws, rank, ot, tt, warp, lane); break;
    case 5: few_sum<N, P::RSTR, 5>(p, red, s_xs, s_ws, rank, ot, tt, warp, lane); break;
    case 6: few_sum<N, P::RSTR, 6>(p, red, s_xs, s_ws, rank, ot, tt, warp, lane); break;
    case 7: few_sum<N, P::RSTR, 7>(p, red, s_xs, s_ws, rank, ot, tt, warp, lane); break;
    default: few_sum<N, P::RSTR, 8>(p, red, s_xs, s_ws, rank, ot, tt, warp, lane); break;
    }
    cluster_sync_all();  // no CTA leaves while another reads its sums
    if (warp == 1) tmem_dealloc(tmem, P::TCOLS);
}

// ---------------------------------------------------------------- host side
// Scale tiles as a 2-D uint32 tensor of 256-byte rows, box {64, 2 * tiles}.
static bool make_map_sf(CUtensorMap *m, const void *base, uint64_t tiles, uint32_t box_tiles)
{
    PFN_encodeTiled_t enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[2] = {64, tiles * 2};
    cuuint64_t strides[1] = {256};
    cuuint32_t box[2] = {64, box_tiles * 2};
    cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static Fp4Params fp4_params(const Fp4GemmArgs &a)
{
    Fp4Params p{};
    p.x_scale = a.x_scale;
    p.w_scale = a.w_scale;
    p.y = a.y;
    p.T = a.T;
    p.K = a.K;
    p.n_out = a.n_out;
    p.out_bf16 = a.out_bf16;
    p.k_blocks = (a.K + 255) / 256;
    p.kt = fp4_sf_ktiles(a.K, a.fmt);
    return p;
}

template <int FMT>
static cudaError_t launch_fp4_pair(const Fp4GemmArgs &a, cudaStream_t st)
{
    CUtensorMap mA, mB, mSA, mSB;
    Fp4Params p = fp4_params(a);
    p.m_tiles = (a.T + PAIR_BM - 1) / PAIR_BM;
    p.n_tiles = (a.n_out + PAIR_BN - 1) / PAIR_BN;
    if (!make_map_u8(&mA, a.xq, (uint64_t)a.T, (uint64_t)a.K / 2, 128) ||
        !make_map_u8(&mB, a.Wq, (uint64_t)a.n_out, (uint64_t)a.K / 2, 128) ||
        !make_map_sf(&mSA, a.x_sf, (uint64_t)((a.T + 127) / 128) * p.kt, Fp4Cfg<FMT>::SFT) ||
        !make_map_sf(&mSB, a.w_sf, (uint64_t)((a.n_out + 127) / 128) * p.kt, Fp4Cfg<FMT>::SFT))
        return cudaErrorInvalidValue;
    static DeviceAnswer cached;
    const int clusters = pair_clusters_of(k_gemm_fp4_pair<FMT>, FpPair<FMT>::smem, cached, FP_THREADS);
    if (clusters <= 0) return cudaErrorNotSupported;
    static RaisedLimit done;
    cudaError_t e = smem_limit_once(k_gemm_fp4_pair<FMT>, FpPair<FMT>::smem, done);
    if (e != cudaSuccess) return e;
    const int grid = 2 * std::min(p.m_tiles * p.n_tiles, clusters);
    k_gemm_fp4_pair<FMT><<<grid, FP_THREADS, FpPair<FMT>::smem, st>>>(mA, mB, mSA, mSB, p);
    return cudaGetLastError();
}

// CTAs of a cluster: the most (at most 8, the portable size, and one per K
// block) with which the clusters of all tiles are resident at once.  CTAs that
// the SMs hold / tiles is not that: a cluster stays within one GPC, so that 16
// clusters of 8 need two waves on 148 SMs (256 x 1024 x 4096: 18.8 us so, 10.7
// with the most that fit).  fit[r] keeps each device's answer for r.
// With two CTAs per SM the SMs' count decides: the answer counts one per SM,
// and a cluster that is left over shares SMs (decode, one token, 11008 x 14336:
// 19.6 us so, 26.9 by the answer).
template <typename Kernel>
static int cluster_that_fits(Kernel kernel, cudaLaunchConfig_t cfg, int tiles, int per_sm, int k_blocks, DeviceAnswer (&fit)[9])
{
    int r = std::max(1, std::min(8, k_blocks)), dev = 0;
    cudaGetDevice(&dev);
    for (; r > 1; --r) {
        if (tiles > per_sm * sm_count() / r) continue;
        if (per_sm > 1) break;
        const int clusters = fit[r].get(dev, [&] {
            cudaLaunchAttribute at{};
            at.id = cudaLaunchAttributeClusterDimension;
            at.val.clusterDim.x = r;
            at.val.clusterDim.y = at.val.clusterDim.z = 1;
            cfg.gridDim = dim3(r, 1, 1);
            cfg.attrs = &at;
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
                cudaGetLastError();
                n = 0;
            }
            return n;
        });
        if (tiles <= clusters) break;
    }
    return r;
}

template <int FMT, int N>
static cudaError_t launch_fp4_few(const Fp4GemmArgs &a, cudaStream_t st)
{
    using P = FpFew<FMT, N>;
    CUtensorMap mA, mB, mSA, mSB;
    Fp4Params p = fp4_params(a);
    p.m_tiles = (a.n_out + 127) / 128;
    p.n_tiles = (a.T + N - 1) / N;
    if (!make_map_u8(&mA, a.Wq, (uint64_t)a.n_out, (uint64_t)a.K / 2, 128) ||
        !make_map_u8(&mB, a.xq, (uint64_t)a.T, (uint64_t)a.K / 2, N) ||
        !make_map_sf(&mSA, a.w_sf, (uint64_t)p.m_tiles * p.kt, Fp4Cfg<FMT>::SFT) ||
        !make_map_sf(&mSB, a.x_sf, (uint64_t)((a.T + 127) / 128) * p.kt, Fp4Cfg<FMT>::SFT))
        return cudaErrorInvalidValue;
    static RaisedLimit done;
    cudaError_t e = smem_limit_once(k_gemm_fp4_few<FMT, N>, P::smem, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(FF_THREADS);
    cfg.dynamicSmemBytes = P::smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    static DeviceAnswer fit[9];
    const int ranks = cluster_that_fits(k_gemm_fp4_few<FMT, N>, cfg, p.m_tiles * p.n_tiles, 1, p.k_blocks, fit);
    cfg.gridDim = dim3(ranks, p.m_tiles, p.n_tiles);
    attr[0].val.clusterDim.x = ranks;
    return cudaLaunchKernelEx(&cfg, k_gemm_fp4_few<FMT, N>, mA, mB, mSA, mSB, p);
}

template <int FMT>
static cudaError_t launch_fp4_t(const Fp4GemmArgs &a, cudaStream_t st)
{
    if (a.T <= 16) return launch_fp4_few<FMT, 16>(a, st);
    if (a.T <= 32) return launch_fp4_few<FMT, 32>(a, st);
    if (a.T <= 64) return launch_fp4_few<FMT, 64>(a, st);
    // One wave of 128 x 128 tiles at most: with K split over the SMs left and a
    // short epilogue it beats 256 x 256 tiles at every length (tokens x outputs x
    // K: 512 x 1024 x 4096 8.1 against 13.5 us, 512 x 4096 x 14336 24.3 against
    // 25.9, 128 x 14336 x 14336 30.0 against 32.7); with a second wave it loses
    // (256 x 14336 x 4096 22.3 against 16.1, 768 x 4096 x 4096 21.1 against 14.1).
    // At most 16, 32 or 64 tokens take narrower tiles: fewer bytes and MMAs
    // (64 x 4096 x 4096 7.4 us as 64 columns, 8.7 as 128; 16 tokens 6.3).
    if ((long long)((a.T + 127) / 128) * ((a.n_out + 127) / 128) <= sm_count()) return launch_fp4_few<FMT, 128>(a, st);
    return launch_fp4_pair<FMT>(a, st);
}

cudaError_t launch_gemm_fp4(const Fp4GemmArgs &a, cudaStream_t st)
{
    return a.fmt == AS_FP4_NV ? launch_fp4_t<AS_FP4_NV>(a, st) : launch_fp4_t<AS_FP4_MX>(a, st);
}

}  // namespace as
