// gated_ffn.cu -- the gated projections of a feed-forward block,
//   out = act(x Wg^T) * (x Wu^T),   w = [2F, K]: Wg's rows, then Wu's,
// in one kernel, and the elementwise part of their gradient.
//
// Both projections share x, so one tile computes c = 128 columns of each (64 to
// 112 where that fills the pairs better, plan_gated_cols): the B operand of the
// 256 x 2c MMA is c rows of Wg and c rows of Wu (one half staged by each CTA of the
// pair), the accumulator's columns 0..c-1 are the gate and c..2c-1 the up
// projection of the same output columns, and the epilogue
// has both in the same TMEM lane: activation and product happen in registers
// and neither projection is written unless the caller keeps it for the
// backward pass.  Compute bound from a few hundred rows on (4 M F K FLOP):
// 4096 x 5120 x 13824 takes 583 us in a burst (2.0 PFLOP/s; 599 with the
// pre-activations kept), 665 us sustained under the power limit, and in e4m3 304 us
// (3.8 PFLOP/s) and 347.  Stages of two K blocks: 603 us with one.
//
// The roles, barriers and bounded waits are those of gemm_nt_pair.cu (whole
// tiles only: nothing here waits for another pair).
#include <atomic>

#include "gated_common.cuh"

namespace lf {
namespace {

constexpr int ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2;
constexpr float GELU_C2 = 1.5957691216057308f;  // 2 sqrt(2 / pi): gelu_tanh(v) = v sigmoid(GELU_C2 (v + a v^3))
constexpr float GELU_A = 0.044715f;

// 1 / (1 + exp(-v)) in fp32: off by about 2^-21, and for negative v by |v| 2^-24 more,
// what the rounding of its exponent makes of exp(-v).  Below -87, where 1 + exp(-v)
// passes 2^126, it is 0.
__device__ __forceinline__ float sigmoid_f(float v) { return __fdividef(1.f, 1.f + ex2_approx(-v * LOG2E)); }

// Activations, act(v) = v phi(v), two values at a time: the polynomials of gelu and
// gelu_tanh run in packed operations (2048 x 1024 x 4096 gelu 28.1 -> 25.4 us, 4096 x
// 2048 x 5632 113.3 -> 105.8, e4m3 64.5 -> 60.3); silu's sigmoid, an exponential and a
// reciprocal, is faster one value at a time (2621 x 224 x 12368 40.8 against 41.4).
//
// The standard normal distribution function, with a = |v| and t = 1 / (1 + 0.3 a):
//   Phi(-a) = exp(-a^2 / 2) t Q(t),  Phi(a) = 1 - Phi(-a).
// exp(a^2 / 2) Phi(-a) falls from 1/2 like 1 / a, so divided by t it is smooth over all of
// 0 < t <= 1, and Q of degree 7 comes within 1.8e-7 of it (relative; least squares on
// Chebyshev nodes for a up to 14, reweighted until the errors were level, coefficients
// rounded to fp32; 0.3 was the best of 0.15 to 0.75).  As evaluated here Phi(-a) is off
// by up to 2^-20 + a^2 2^-24: the rest is the rounding of a^2 in the exponent.  One
// polynomial, one exponential and one reciprocal: with normcdff the epilogue of a tile
// took 10 us.
__device__ __forceinline__ float2 normal_cdf(float2 v)
{
    const float2 t = make_float2(__fdividef(1.f, fmaf(0.3f, fabsf(v.x), 1.f)),
                                 __fdividef(1.f, fmaf(0.3f, fabsf(v.y), 1.f)));
    float2 q = fma2(t, both(0.03567476f), both(-0.15720302f));
    q = fma2(t, q, both(0.2063534f));
    q = fma2(t, q, both(-0.05368354f));
    q = fma2(t, q, both(0.12856157f));
    q = fma2(t, q, both(0.09991351f));
    q = fma2(t, q, both(0.12075395f));
    q = fma2(t, q, both(0.1196293f));
    const float2 x = mul2(mul2(v, v), both(-0.5f * LOG2E));
    const float2 e = mul2(mul2(t, q), make_float2(ex2_approx(x.x), ex2_approx(x.y)));
    const float2 r = fma2(e, both(-1.f), both(1.f));
    return make_float2(v.x < 0.f ? e.x : r.x, v.y < 0.f ? e.y : r.y);
}

// phi(v)
template <int ACT>
__device__ __forceinline__ float2 act_phi(float2 v)
{
    if (ACT == ACT_GELU)
        return normal_cdf(v);
    if (ACT == ACT_GELU_TANH)
        v = mul2(both(GELU_C2), fma2(mul2(mul2(both(GELU_A), v), v), v, v));
    return make_float2(sigmoid_f(v.x), sigmoid_f(v.y));
}

// d phi / d v, given p = phi(v)
template <int ACT>
__device__ __forceinline__ float act_dphi(float v, float p)
{
    if (ACT == ACT_SILU)
        return p * (1.f - p);
    if (ACT == ACT_GELU)
        return 0.3989422804014327f * ex2_approx(-0.5f * LOG2E * v * v);
    return p * (1.f - p) * GELU_C2 * fmaf(3.f * GELU_A * v, v, 1.f);
}

// Tile order: bands of band_m M blocks (M block fastest), as gemm_nt_pair.cu.
__device__ __forceinline__ void g_tile_coords(const GemmParams &p, int tile, int &mb, int &nb)
{
    const int MB = p.num_m_blocks;
    const int bm = p.band_m > 0 && p.band_m < MB ? p.band_m : MB;
    const int per_band = bm * p.num_n_blocks;
    const int band = tile / per_band;
    const int local = tile - band * per_band;
    const int rows = min(bm, MB - band * bm);
    mb = band * bm + local % rows;
    nb = local / rows;
}

// 32 columns of one projection as they stand for: f times the token's scale, then
// the output channels' (e4m3 operands), or f itself.  (f sx is what the token stands
// for; sx w alone may be a subnormal number that has lost its bits.)
template <bool E4M3>
__device__ __forceinline__ void g_scale(float (&f)[32], float sx, const float *w_scale, int valid)
{
    if (E4M3) {
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            if (i < valid) {  // N % 8 == 0
                const float4 w = *reinterpret_cast<const float4 *>(w_scale + i);
                const float2 a = mul2(mul2(make_float2(f[i], f[i + 1]), both(sx)), make_float2(w.x, w.y));
                const float2 b = mul2(mul2(make_float2(f[i + 2], f[i + 3]), both(sx)), make_float2(w.z, w.w));
                f[i] = a.x;
                f[i + 1] = a.y;
                f[i + 2] = b.x;
                f[i + 3] = b.y;
            }
        }
    }
}

// The warp's 32 rows x 64 columns (from c0) of a finished tile.  The gate of
// output column c is accumulator column c, its up projection accumulator column
// gp.cols + c.  Returns once the accumulator has been read.
template <bool E4M3, int ACT>
__device__ __forceinline__ void g_epilogue(const GatedParams &gp, const CUtensorMap *tmO, const CUtensorMap *tmG,
                                           const CUtensorMap *tmU, uint32_t taddr, int row0, int nb, int c0,
                                           float sx, uint8_t *stg, uint32_t stg_s)
{
    const GemmParams &p = gp.g;
    const int col = nb * gp.cols + c0;
    if (col >= p.N)
        return;  // warp-uniform
    // (the accumulator is read before the wait for the staging buffer: the two overlap)
    if (!E4M3 && gp.save) {
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {
            const uint32_t t = taddr + static_cast<uint32_t>(side * gp.cols + c0);
            float f[32], h[32];
            load_acc2(t, t + 32, f, h);
            stage_begin();
            stage_half(stg, 0, f);
            stage_half(stg, 1, h);
            stage_end(side ? tmU : tmG, stg_s, col, row0, p.M);
        }
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const uint32_t t = taddr + static_cast<uint32_t>(c0 + 32 * half);
        float g[32], u[32];
        load_acc2(t, t + static_cast<uint32_t>(gp.cols), g, u);
        g_scale<E4M3>(g, sx, gp.w_scale + col + 32 * half, p.N - col - 32 * half);
        g_scale<E4M3>(u, sx, gp.w_scale + p.N + col + 32 * half, p.N - col - 32 * half);
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            const float2 v = make_float2(g[i], g[i + 1]);
            const float2 r = mul2(mul2(v, act_phi<ACT>(v)), make_float2(u[i], u[i + 1]));
            g[i] = r.x;
            g[i + 1] = r.y;
        }
        if (half == 0)
            stage_begin();
        stage_half(stg, half, g);
    }
    stage_end(tmO, stg_s, col, row0, p.M);
}

template <bool E4M3, int ACT>
__global__ void __launch_bounds__(G_THREADS, 1)
    k_gated_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                 const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmG,
                 const __grid_constant__ CUtensorMap tmU, const __grid_constant__ GatedParams gp)
{
    const GemmParams &p = gp.g;
    constexpr int KELEMS = E4M3 ? 128 : 64;  // elements of K per block
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const uint32_t sA = base;
    const uint32_t sB = base + G_SLOTS * G_A_BYTES;
    const uint32_t bar0 = base + G_SLOTS * G_SLOT_BYTES;
    const uint32_t drain_bar = bar0 + 8u * (2 * G_STAGES + 2 * G_ACC_BUFS);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + G_SLOTS * G_SLOT_BYTES + G_NUM_BARS * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
#define FULL_BAR(s) (bar0 + 8u * (s))
#define EMPTY_BAR(s) (bar0 + 8u * (G_STAGES + (s)))
#define TFULL_BAR(b) (bar0 + 8u * (2 * G_STAGES + (b)))
#define TEMPTY_BAR(b) (bar0 + 8u * (2 * G_STAGES + G_ACC_BUFS + (b)))

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1;
    const int num_pairs = gridDim.x >> 1;
    const int cols = gp.cols;

    if (threadIdx.x == 0) {
        for (int s = 0; s < G_STAGES; ++s) {
            mbar_init(FULL_BAR(s), 1);   // leader: its arrive.expect_tx + both CTAs' bytes
            mbar_init(EMPTY_BAR(s), 1);  // the leader's multicast commit
        }
        for (int b = 0; b < G_ACC_BUFS; ++b) {
            mbar_init(TFULL_BAR(b), 1);                 // the leader's multicast commit
            mbar_init(TEMPTY_BAR(b), 2 * G_EPI_WARPS);  // leader: one arrive per epilogue warp of each CTA
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmO);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), G_TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any cross-CTA signal
    tc_fence_after();
    wait_previous_kernel();
    let_next_kernel_start();
    const uint32_t tmem_base = *tmem_slot;
    const uint32_t peer_abort = mapa_shared(smem_u32(const_cast<int *>(abort_flag)), rank ^ 1u);

    if (warp == 0) {
        // ------------------------------------------------ TMA producer (both CTAs)
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            const uint32_t slot_bytes = 2u * static_cast<uint32_t>(G_A_BYTES + cols * G_ROW);
            uint32_t armed[G_STAGES];
#pragma unroll
            for (int s = 0; s < G_STAGES; ++s)
                armed[s] = 0;
            bool ok = true, first = true;
            for (int tile = pair; ok && tile < p.num_tiles; tile += num_pairs) {
                int mb, nb;
                g_tile_coords(p, tile, mb, nb);
                const int arow = mb * G_M + static_cast<int>(rank) * BM;
                // gate rows in the leader, up rows in its peer
                const int brow = static_cast<int>(rank) * p.N + nb * cols;
                for (int kb = 0; kb < p.num_k_blocks; kb += G_KSUB) {
                    const int nsub = min(G_KSUB, p.num_k_blocks - kb);
                    if (!wait_bar(EMPTY_BAR(stage), phase ^ 1u, abort_flag, p, ERR_PRODUCER, peer_abort)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full_leader = mapa_shared(FULL_BAR(stage), 0u);
                    const bool skip = first && p.inject == 1 && blockIdx.x == 0;  // test hook
                    first = false;
                    if (!skip) {
                        if (leader) {
                            mbar_arrive_expect_tx(FULL_BAR(stage), slot_bytes * static_cast<uint32_t>(nsub));
                            ++armed[stage];
                        }
#pragma unroll
                        for (int j = 0; j < G_KSUB; ++j) {
                            if (j >= nsub)
                                break;
                            const uint32_t slot = static_cast<uint32_t>(stage * G_KSUB + j);
                            tma_load_2d_pair(sA + slot * G_A_BYTES, &tmA, (kb + j) * KELEMS, arow, full_leader);
                            tma_load_2d_pair(sB + slot * G_B_BYTES, &tmW, (kb + j) * KELEMS, brow, full_leader);
                        }
                    }
                    if (++stage == G_STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (leader)
                for (int s = 0; s < G_STAGES; ++s)
                    if (armed[s])
                        wait_bar_drain(FULL_BAR(s), (armed[s] - 1u) & 1u, abort_flag, p, peer_abort);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (leader only)
        // (the whole warp, converged, with one thread issuing: see lf_ptx_ffn.cuh; after a
        // wait that gave up the loops run on without doing anything)
        if (leader) {
            const uint32_t one = elect_one();
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool alive = true;
            const uint32_t idesc = E4M3 ? idesc_e4m3_f32(G_M, 2 * cols) : idesc_bf16_f32(G_M, 2 * cols);
            for (int tile = pair; tile < p.num_tiles; tile += num_pairs) {
                if (alive)
                    alive = __all_sync(0xffffffffu, wait_bar(TEMPTY_BAR(acc), acc_phase ^ 1u, abort_flag, p, ERR_MMA_ACC,
                                                             peer_abort));
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
                for (int kb = 0; kb < p.num_k_blocks; kb += G_KSUB) {
                    const int nsub = min(G_KSUB, p.num_k_blocks - kb);
                    if (alive)
                        alive = __all_sync(0xffffffffu, wait_bar(FULL_BAR(stage), phase, abort_flag, p, ERR_MMA_FULL,
                                                                 peer_abort));
                    if (alive) {
                        tc_fence_after();
#pragma unroll
                        for (int j = 0; j < G_KSUB; ++j) {
                            if (j >= nsub)
                                break;
                            const uint32_t a0 = sA + (stage * G_KSUB + j) * G_A_BYTES;
                            const uint32_t b0 = sB + (stage * G_KSUB + j) * G_B_BYTES;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {  // 32 bytes of K per MMA
                                const uint64_t da = smem_desc_k128(a0 + k * 32), db = smem_desc_k128(b0 + k * 32);
                                const uint32_t accumulate = (kb | j | k) != 0 ? 1u : 0u;
                                if (E4M3)
                                    umma_f8_pair_one(one, d_tmem, da, db, idesc, accumulate);
                                else
                                    umma_f16_pair_one(one, d_tmem, da, db, idesc, accumulate);
                            }
                        }
                        umma_commit_pair_mc_one(one, EMPTY_BAR(stage), 0x3);
                    }
                    if (++stage == G_STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (alive)
                    umma_commit_pair_mc_one(one, TFULL_BAR(acc), 0x3);
                if (++acc == G_ACC_BUFS) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
            umma_commit_pair_mc_one(one, drain_bar, 0x1);
            if (lane == 0)
                wait_bar_drain(drain_bar, 0u, abort_flag, p, peer_abort);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ epilogue (both CTAs)
        // warp w reads TMEM lanes 32 (w % 4) ..; warps 2..5 take the tile's first 64
        // output columns, warps 6..9 its last 64 (columns that both cover are
        // written twice, with the same values; a tile of 64 columns needs one of them)
        const int q = warp & 3;
        const bool second = warp >= 2 + G_EPI_WARPS / 2;
        const int c0 = second ? cols - G_MIN_F : 0;
        int acc = 0;
        uint32_t acc_phase = 0;
        uint8_t *stg = gbase + G_STG_OFF + (warp - 2) * G_STG_WARP;
        const uint32_t stg_s = base + static_cast<uint32_t>(G_STG_OFF + (warp - 2) * G_STG_WARP);
        for (int tile = pair; tile < p.num_tiles; tile += num_pairs) {
            int mb, nb;
            g_tile_coords(p, tile, mb, nb);
            const int row0 = mb * G_M + static_cast<int>(rank) * BM + q * 32;
            float sx = 1.f;  // the token's scale, loaded during the wait
            if (E4M3)
                sx = row0 + lane < p.M ? gp.x_scale[row0 + lane] : 0.f;
            const bool ok = wait_bar(TFULL_BAR(acc), acc_phase, abort_flag, p, ERR_EPI, peer_abort);
            if (!__all_sync(0xffffffffu, ok))
                break;
            tc_fence_after();
            if (!second || cols > G_MIN_F)
                g_epilogue<E4M3, ACT>(gp, &tmO, &tmG, &tmU,
                                  tmem_base + static_cast<uint32_t>(acc * BN) + (static_cast<uint32_t>(q * 32) << 16),
                                  row0, nb, c0, sx, stg, stg_s);
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(mapa_shared(TEMPTY_BAR(acc), 0u));
            if (++acc == G_ACC_BUFS) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
        if (lane == 0)
            bulk_wait_group_all();
    }
#undef FULL_BAR
#undef EMPTY_BAR
#undef TFULL_BAR
#undef TEMPTY_BAR

    if (*abort_flag) {
        // Copies this CTA issued complete on the leader's barrier, so nothing
        // here can wait for them: give them a fixed, generous time to land.
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < G_ABORT_SETTLE_NS) {
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the peer no longer touches this CTA's barriers, smem or TMEM
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, G_TMEM_COLS);
    }
}

template <bool E4M3, int ACT>
cudaError_t launch_gated_pair_t(const CUtensorMap &ta, const CUtensorMap &tw, const CUtensorMap &to,
                                const CUtensorMap &tg, const CUtensorMap &tu, const GatedParams &p, int grid,
                                cudaStream_t s)
{
    static std::atomic<unsigned long long> done{0};  // the shared-memory opt-in, once per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load() & bit)) {
        e = cudaFuncSetAttribute(k_gated_pair<E4M3, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize, G_SMEM);
        if (e != cudaSuccess)
            return e;
        done.fetch_or(bit);
    }
    return launch_overlapped(k_gated_pair<E4M3, ACT>, dim3(static_cast<unsigned>(grid)), dim3(G_THREADS), G_SMEM, 2, s,
                             ta, tw, to, tg, tu, p);
}

// ---------------------------------------------------------------- few tokens
// Up to 128 tokens (and groups of 128 where tiles are few and K long, see
// plan_gated_skinny): the weights' bytes bound the call, so the operands are
// swapped -- 128 gate rows and 128 up rows of w are the A operands of two
// 128 x n MMAs whose B operand is the tokens (n: M rounded up to 16) -- and a CTA
// only streams its share of w through a ring of 32 KiB stages (plus the tokens'
// slice).  With few tiles of 128 output columns the K blocks of a tile are split
// over a cluster of 2, 4 or 8 CTAs: each leaves its fp32 sums in its own shared
// memory, and after a cluster barrier every CTA adds, in rank order, its part of
// the tokens from all of them.  5120 x 13824: one token 45-47 us bf16 (90 % of the
// copy rate), 48 tokens e4m3 27.0 us; 8192 x 28672 97-99 %: what is left is the
// launch's 4-5 us.
constexpr int S_THREADS = 192;     // producer, MMA, 4 epilogue warps
constexpr int S_WARPS = S_THREADS / 32;
constexpr int S_MAX_STAGES = 8;
constexpr int S_W_BYTES = 2 * BM * G_ROW;
constexpr int S_MISC = 1024 + (2 * S_MAX_STAGES + 1) * 8 + 32;  // alignment, barriers, TMEM address, abort flag
constexpr int S_SMEM_ONE = 220 * 1024, S_SMEM_TWO = 113 * 1024;  // dynamic shared memory with one / two CTAs per SM

// Output columns f .. f + 3 of token m from its sums g and u (e4m3 operands: sx the
// token's scale, wg and wu the columns').
template <bool E4M3, int ACT>
__device__ __forceinline__ void s_finish(const GatedParams &gp, __nv_bfloat16 *gu, float4 g, float4 u, int m, int f,
                                         float sx, float4 wg, float4 wu)
{
    const size_t F = static_cast<size_t>(gp.g.N);
    if (E4M3) {
        g = make_float4(g.x * sx * wg.x, g.y * sx * wg.y, g.z * sx * wg.z, g.w * sx * wg.w);
        u = make_float4(u.x * sx * wu.x, u.y * sx * wu.y, u.z * sx * wu.z, u.w * sx * wu.w);
    }
    const float2 p = act_phi<ACT>(make_float2(g.x, g.y)), q = act_phi<ACT>(make_float2(g.z, g.w));
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(gp.g.out) + m * F + f) =
        make_uint2(pack_bf16(g.x * p.x * u.x, g.y * p.y * u.y), pack_bf16(g.z * q.x * u.z, g.w * q.y * u.w));
    if (!E4M3 && gu) {
        *reinterpret_cast<uint2 *>(gu + m * 2 * F + f) = make_uint2(pack_bf16(g.x, g.y), pack_bf16(g.z, g.w));
        *reinterpret_cast<uint2 *>(gu + m * 2 * F + F + f) = make_uint2(pack_bf16(u.x, u.y), pack_bf16(u.z, u.w));
    }
}

template <bool E4M3, int ACT>
__global__ void __launch_bounds__(S_THREADS, 2)
    k_gated_skinny(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                   const __grid_constant__ GatedParams gp, const GatedSkinny plan, __nv_bfloat16 *gu)
{
    const GemmParams &p = gp.g;
    constexpr int KELEMS = E4M3 ? 128 : 64;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const uint32_t x_bytes = static_cast<uint32_t>(plan.n) * G_ROW;
    const uint32_t stage_bytes = S_W_BYTES + x_bytes;
    const uint32_t bar0 = base + static_cast<uint32_t>(plan.stages) * stage_bytes;
    const uint32_t done_bar = bar0 + 8u * (2 * S_MAX_STAGES);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + (done_bar + 8u - base));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
#define FULL_BAR(s) (bar0 + 8u * (s))
#define EMPTY_BAR(s) (bar0 + 8u * (S_MAX_STAGES + (s)))

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int split = plan.split;
    const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int f0 = static_cast<int>(blockIdx.x) / split * G_F;
    const int m0 = static_cast<int>(blockIdx.y) * plan.tokens;  // this CTA's tokens: m0 .. m0 + M - 1
    const int M = min(plan.tokens, p.M - m0);
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.num_k_blocks) * rank / split);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.num_k_blocks) * (rank + 1) / split);
    uint32_t cols = 32;
    while (cols < 2u * static_cast<uint32_t>(plan.n))
        cols *= 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < plan.stages; ++s) {
            mbar_init(FULL_BAR(s), 1);
            mbar_init(EMPTY_BAR(s), 1);
        }
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    wait_previous_kernel();
    let_next_kernel_start();
    const uint32_t tmem_base = *tmem_slot;
    // The scales this thread finishes with, loaded while the weights stream: of its
    // four output columns, and of the warp's tokens m_first + 6 i (in lane i).
    const int f = f0 + 4 * lane;
    const int m_first = M * rank / split + warp, m_end = M * (rank + 1) / split;
    float4 wg4 = make_float4(1.f, 1.f, 1.f, 1.f), wu4 = wg4;
    float sx_lane = 1.f;
    if (E4M3) {
        if (f < p.N) {  // N % 8 == 0
            wg4 = *reinterpret_cast<const float4 *>(gp.w_scale + f);
            wu4 = *reinterpret_cast<const float4 *>(gp.w_scale + p.N + f);
        }
        if (m_first + S_WARPS * lane < m_end)
            sx_lane = gp.x_scale[m0 + m_first + S_WARPS * lane];
    }

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!wait_bar(EMPTY_BAR(stage), phase ^ 1u, abort_flag, p, ERR_PRODUCER))
                    break;
                if (!(kb == kb0 && p.inject == 1 && blockIdx.x == 0 && blockIdx.y == 0)) {  // (test hook)
                    const uint32_t dst = base + stage * stage_bytes;
                    mbar_arrive_expect_tx(FULL_BAR(stage), stage_bytes);
                    tma_load_2d(dst, &tmW, kb * KELEMS, f0, FULL_BAR(stage));
                    tma_load_2d(dst + BM * G_ROW, &tmW, kb * KELEMS, p.N + f0, FULL_BAR(stage));
                    tma_load_2d(dst + S_W_BYTES, &tmA, kb * KELEMS, m0, FULL_BAR(stage));
                }
                if (++stage == plan.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (*abort_flag) {  // let the copies in flight land
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < G_ABORT_SETTLE_NS) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            const uint32_t n = static_cast<uint32_t>(plan.n);
            const uint32_t idesc = E4M3 ? idesc_e4m3_f32(BM, n) : idesc_bf16_f32(BM, n);
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!wait_bar(FULL_BAR(stage), phase, abort_flag, p, ERR_MMA_FULL))
                    break;
                tc_fence_after();
                const uint32_t wg = base + stage * stage_bytes, wu = wg + BM * G_ROW, xs = wg + S_W_BYTES;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint64_t db = smem_desc_k128(xs + k * 32);
                    const uint32_t accumulate = (kb != kb0 || k != 0) ? 1u : 0u;
                    if (E4M3) {
                        umma_f8(tmem_base, smem_desc_k128(wg + k * 32), db, idesc, accumulate);
                        umma_f8(tmem_base + n, smem_desc_k128(wu + k * 32), db, idesc, accumulate);
                    } else {
                        umma_f16(tmem_base, smem_desc_k128(wg + k * 32), db, idesc, accumulate);
                        umma_f16(tmem_base + n, smem_desc_k128(wu + k * 32), db, idesc, accumulate);
                    }
                }
                umma_commit(EMPTY_BAR(stage));
                if (++stage == plan.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            umma_commit(done_bar);  // also after an abort: what was issued drains
            wait_bar_drain(done_bar, 0u, abort_flag, p);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ sums to shared memory, one output column per thread
        const int q = warp & 3;
        const bool ok = __all_sync(0xffffffffu, wait_bar(done_bar, 0u, abort_flag, p, ERR_EPI));
        tc_fence_after();
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
        float *part = reinterpret_cast<float *>(gbase) + q * 32 + lane;  // the ring is idle: [2 M][128] sums
        for (int c = 0; ok && c < M; c += 16) {
            uint32_t g[16], u[16];
            tmem_ld_32x32b_x16(taddr + static_cast<uint32_t>(c), g);
            tmem_ld_32x32b_x16(taddr + static_cast<uint32_t>(plan.n + c), u);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (c + i < M) {
                    part[(2 * (c + i)) * BM] = __uint_as_float(g[i]);
                    part[(2 * (c + i) + 1) * BM] = __uint_as_float(u[i]);
                }
            }
        }
        tc_fence_before();
        __syncwarp();
    }
    // Every CTA's sums are in place: this one finishes its share of the tokens,
    // one token per warp at a time, four output columns per lane.
    if (split > 1)
        cluster_sync();
    else
        __syncthreads();
#pragma unroll(E4M3 ? 4 : 2)
    for (int i = 0; m_first + S_WARPS * i < m_end; ++i) {
        const int m = m_first + S_WARPS * i;
        const uint32_t a = base + static_cast<uint32_t>((2 * m * BM + 4 * lane) * 4);
        float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g;
        for (int r = 0; r < split; ++r) {
            const uint32_t ar = split > 1 ? mapa_shared(a, static_cast<uint32_t>(r)) : a;
            const float4 dg = ld_cluster_f32x4(ar), du = ld_cluster_f32x4(ar + BM * 4);
            g = make_float4(g.x + dg.x, g.y + dg.y, g.z + dg.z, g.w + dg.w);
            u = make_float4(u.x + du.x, u.y + du.y, u.z + du.z, u.w + du.w);
        }
        const float sx = E4M3 ? __shfl_sync(0xffffffffu, sx_lane, i) : 1.f;
        if (f < p.N)
            s_finish<E4M3, ACT>(gp, gu, g, u, m0 + m, f, sx, wg4, wu4);
    }
    __syncwarp();
    if (split > 1)
        cluster_sync();  // no CTA leaves while a peer reads its sums
#undef FULL_BAR
#undef EMPTY_BAR
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, cols);
    }
}

template <bool E4M3, int ACT>
cudaError_t launch_gated_skinny_t(const CUtensorMap &ta, const CUtensorMap &tw, const GatedParams &p,
                                  const GatedSkinny &plan, void *gu, cudaStream_t s)
{
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load() & bit)) {
        e = cudaFuncSetAttribute(k_gated_skinny<E4M3, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S_SMEM_ONE);
        if (e != cudaSuccess)
            return e;
        done.fetch_or(bit);
    }
    return launch_overlapped(k_gated_skinny<E4M3, ACT>, dim3(static_cast<unsigned>(p.g.num_n_blocks * plan.split),
                                  static_cast<unsigned>((p.g.M + plan.tokens - 1) / plan.tokens)),
                             dim3(S_THREADS), static_cast<size_t>(plan.smem), plan.split, s, ta, tw, p, plan,
                             static_cast<__nv_bfloat16 *>(gu));
}

// ---------------------------------------------------------------- gradient
// dgu = [dout u act'(g), dout act(g)] from the kept pre-activations gu = [g, u]:
// 8 columns per thread and step, 6 bytes read and 4 written per column: bound by
// HBM (4096 x 13824: 79 us silu, 7.1 TB/s; gelu 83, 98 without room for six blocks
// per SM).
template <int ACT>
__global__ void __launch_bounds__(256, 6)
    k_gated_bwd(const __nv_bfloat16 *dout, const __nv_bfloat16 *gu, __nv_bfloat16 *dgu, int64_t M, int64_t F)
{
    wait_previous_kernel();
    let_next_kernel_start();
    const int64_t packs = F / 8;
    for (int64_t row = blockIdx.y; row < M; row += gridDim.y) {
        for (int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; c < packs;
             c += static_cast<int64_t>(gridDim.x) * blockDim.x) {
            const uint4 dv = *reinterpret_cast<const uint4 *>(dout + row * F + c * 8);
            const uint4 gv = *reinterpret_cast<const uint4 *>(gu + row * 2 * F + c * 8);
            const uint4 uv = *reinterpret_cast<const uint4 *>(gu + row * 2 * F + F + c * 8);
            const __nv_bfloat162 *d2 = reinterpret_cast<const __nv_bfloat162 *>(&dv);
            const __nv_bfloat162 *g2 = reinterpret_cast<const __nv_bfloat162 *>(&gv);
            const __nv_bfloat162 *u2 = reinterpret_cast<const __nv_bfloat162 *>(&uv);
            uint32_t dg[4], du[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 d = __bfloat1622float2(d2[i]), g = __bfloat1622float2(g2[i]), u = __bfloat1622float2(u2[i]);
                const float2 p = act_phi<ACT>(g);
                dg[i] = pack_bf16(d.x * u.x * fmaf(g.x, act_dphi<ACT>(g.x, p.x), p.x),
                                  d.y * u.y * fmaf(g.y, act_dphi<ACT>(g.y, p.y), p.y));
                du[i] = pack_bf16(d.x * (g.x * p.x), d.y * (g.y * p.y));
            }
            *reinterpret_cast<uint4 *>(dgu + row * 2 * F + c * 8) = make_uint4(dg[0], dg[1], dg[2], dg[3]);
            *reinterpret_cast<uint4 *>(dgu + row * 2 * F + F + c * 8) = make_uint4(du[0], du[1], du[2], du[3]);
        }
    }
}

}  // namespace

cudaError_t launch_gated_pair(bool e4m3, int act, const CUtensorMap &ta, const CUtensorMap &tw, const CUtensorMap &to,
                              const CUtensorMap &tg, const CUtensorMap &tu, const GatedParams &p, int grid,
                              cudaStream_t s)
{
    switch (act + (e4m3 ? 3 : 0)) {
    case ACT_SILU:
        return launch_gated_pair_t<false, ACT_SILU>(ta, tw, to, tg, tu, p, grid, s);
    case ACT_GELU:
        return launch_gated_pair_t<false, ACT_GELU>(ta, tw, to, tg, tu, p, grid, s);
    case ACT_GELU_TANH:
        return launch_gated_pair_t<false, ACT_GELU_TANH>(ta, tw, to, tg, tu, p, grid, s);
    case 3 + ACT_SILU:
        return launch_gated_pair_t<true, ACT_SILU>(ta, tw, to, tg, tu, p, grid, s);
    case 3 + ACT_GELU:
        return launch_gated_pair_t<true, ACT_GELU>(ta, tw, to, tg, tu, p, grid, s);
    case 3 + ACT_GELU_TANH:
        return launch_gated_pair_t<true, ACT_GELU_TANH>(ta, tw, to, tg, tu, p, grid, s);
    }
    return cudaErrorInvalidValue;
}

// Clusters of `split` few-token CTAs (one per SM) that the device holds at once:
// clusters stay within a group of SMs, so 152 SMs hold 76, 36 and 15 of two,
// four and eight, and a sixteenth cluster of eight would wait for a second wave.
static int skinny_clusters(int split, int num_sms)
{
    static std::atomic<int> known[4][64];
    int dev = 0;
    if (split == 1 || cudaGetDevice(&dev) != cudaSuccess)
        return num_sms;
    const int i = split == 2 ? 1 : split == 4 ? 2 : 3;
    std::atomic<int> &k = known[i][dev & 63];
    int n = k.load();
    if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(split), 1, 1);
        cfg.blockDim = dim3(S_THREADS, 1, 1);
        cfg.dynamicSmemBytes = S_SMEM_ONE;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(split);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaFuncSetAttribute(k_gated_skinny<false, ACT_SILU>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 S_SMEM_ONE) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, k_gated_skinny<false, ACT_SILU>, &cfg) != cudaSuccess || n < 1) {
            cudaGetLastError();
            n = 1;
        }
        k.store(n);
    }
    return n;
}

// 128 columns per tile keep the tensor cores fullest, and fewer fill the last wave
// better.  A K block then costs as much as its operands' way into shared memory, 128
// rows of x and `cols` rows of w per CTA (200 tokens of 5120 x 4096, one wave: 30.0 us
// with 128 columns, 28.9 with 112, 27.7 with 96, 26.9 with 80, 25.1 with 64), so
// waves x (128 + cols) orders the choices: 200 x 5120 x 13824 62.8 -> 57.6 us (96
// columns, two waves as with 128), 333 x 2048 x 5632 24.6 -> 21.6 (80), 1024 x 4096 x
// 8192 85.0 -> 82.3 (112), 200 x 520 x 1416 silu 8.0 -> 6.3 (64); 4096 x 5120 x 13824
// stays at 128 (584 us; 619 with 112).
int plan_gated_cols(int m_blocks, int64_t F, int pairs)
{
    int best = 0;
    int64_t least = 0;
    for (int cols = G_F; cols >= G_MIN_F; cols -= 16) {  // the MMA's N is a multiple of 32
        const int64_t tiles = (F + cols - 1) / cols * m_blocks;
        const int64_t t = (tiles + pairs - 1) / pairs * (BM + cols);
        if (best == 0 || t < least) {
            least = t;
            best = cols;
        }
    }
    return best;
}

GatedSkinny plan_gated_skinny(int64_t M, int64_t F, int num_k_blocks, int num_sms)
{
    GatedSkinny g;
    const int64_t groups = (M + BM - 1) / BM;
    g.tokens = groups == 1 ? static_cast<int>(M) : static_cast<int>(((M + groups - 1) / groups + 15) / 16 * 16);
    g.n = (g.tokens + 15) / 16 * 16;
    const int64_t tiles = (F + G_F - 1) / G_F * groups;
    // One CTA per SM with a deep ring, and the largest split that keeps all of them in
    // one wave (5120 x 13824, 48 tokens, 108 tiles: 48.6 us unsplit, 50.6 us split
    // in two with two CTAs per SM; 2048 x 5632, 64 tokens, 44 tiles: 14.8 us split in
    // two, 16.7 us in four with two CTAs per SM; 4096 x 2048, one token, 16 tiles: 11.0 us
    // split in four, 15.5 us in eight, whose sixteen clusters are two waves).
    // More tiles than SMs: two CTAs per SM while the sums of 64 tokens fit half an
    // SM's ring.
    const bool two = g.n <= 64 && tiles > num_sms;
    g.split = 1;
    while (g.split < 8 && num_k_blocks / (g.split * 2) >= 4 && tiles <= skinny_clusters(g.split * 2, num_sms))
        g.split *= 2;
    const int stage = S_W_BYTES + g.n * G_ROW;
    const int fit = ((two ? S_SMEM_TWO : S_SMEM_ONE) - S_MISC) / stage;
    g.stages = fit < S_MAX_STAGES ? fit : S_MAX_STAGES;
    g.smem = S_MISC + g.stages * stage;
    // The choice between this kernel and the pair kernel, which has no sums to exchange: one
    // rule for both types, over K blocks of 128 bytes.  (us, pair kernel / this one, bf16 and
    // then e4m3, which has twice the K in as many blocks [in brackets].)
    // Up to 16 tokens: always this one (16 x 256 x 4096 bf16 [4] 5.0 / 4.3, e4m3 [2] 5.7 / 3.7).
    // Up to 128: where the K loop is long for the tokens
    //   64 x .. x 1408   [8] 4.9 / 6.7, 6.1 / 6.8    [16] 6.5 / 6.2, 7.5 / 6.4
    //   128 x .. x 4096  [16] 8.3 / 10.7, 9.2 / 10.8  [32] bf16 12.3 / 13.1
    //   128 x .. x 1408  [32] 11.5 / 10.9, 12.2 / 10.9
    // or the tiles fill the device without a split
    //   .. x 11008 [8]   64 tokens 10.0 / 9.6, 10.8 / 10.0   96 10.2 / 10.8, 11.1 / 11.5   128 9.9 / 12.2, 10.8 / 13.1
    // so at the border of 96 tokens and at 128 x 2048 x 4096 the other kernel is up to 6 % faster.
    // More tokens, in groups: only where the tiles are few, and the K loops long enough
    // for the split to pay for its sums, which grow with the tokens of a group
    //   split in four or eight  144 x .. x 512 [16] 6.2 / 6.5, 7.0 / 6.8  [32] 9.0 / 7.4, 9.7 / 7.6
    //                           256 x .. x 512 [32] 9.0 / 9.6, 9.7 / 9.6  [64] 18.8 / 11.8, 19.6 / 11.8
    //   split in two            144 x .. x 4096 [80] 24.8 / 23.5, 26.1 / 23.9
    //                           256 x .. x 4096 [80] 25.0 / 26.5, 26.3 / 26.9  [128] 38.0 / 37.0, 39.6 / 37.3
    //   unsplit                 333 x .. x 4096 [80] 29.6 / 39.7, 31.0 / 40.9
    if (groups == 1)
        g.preferred = g.n <= 16 || 4 * num_k_blocks >= g.n || (g.n <= 96 && tiles > num_sms / 2);
    else
        g.preferred = (g.split >= 4 && 3 * num_k_blocks >= g.n) || (g.split == 2 && 4 * num_k_blocks >= 3 * g.n);
    return g;
}

cudaError_t launch_gated_skinny(bool e4m3, int act, const CUtensorMap &ta, const CUtensorMap &tw, const GatedParams &p,
                                const GatedSkinny &plan, void *gu, cudaStream_t s)
{
    switch (act + (e4m3 ? 3 : 0)) {
    case ACT_SILU:
        return launch_gated_skinny_t<false, ACT_SILU>(ta, tw, p, plan, gu, s);
    case ACT_GELU:
        return launch_gated_skinny_t<false, ACT_GELU>(ta, tw, p, plan, gu, s);
    case ACT_GELU_TANH:
        return launch_gated_skinny_t<false, ACT_GELU_TANH>(ta, tw, p, plan, gu, s);
    case 3 + ACT_SILU:
        return launch_gated_skinny_t<true, ACT_SILU>(ta, tw, p, plan, gu, s);
    case 3 + ACT_GELU:
        return launch_gated_skinny_t<true, ACT_GELU>(ta, tw, p, plan, gu, s);
    case 3 + ACT_GELU_TANH:
        return launch_gated_skinny_t<true, ACT_GELU_TANH>(ta, tw, p, plan, gu, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_gated_bwd(int act, const void *dout, const void *gu, void *dgu, int64_t M, int64_t F,
                             cudaStream_t s)
{
    const int64_t bx = (F / 8 + 255) / 256;
    const dim3 grid(static_cast<unsigned>(bx < 1024 ? bx : 1024), static_cast<unsigned>(M < 65535 ? M : 65535));
    const __nv_bfloat16 *d = static_cast<const __nv_bfloat16 *>(dout), *g = static_cast<const __nv_bfloat16 *>(gu);
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(dgu);
    const auto kernel = act == ACT_SILU   ? k_gated_bwd<ACT_SILU>
                        : act == ACT_GELU ? k_gated_bwd<ACT_GELU>
                                          : k_gated_bwd<ACT_GELU_TANH>;
    return launch_overlapped(kernel, grid, dim3(256), 0, 1, s, d, g, o, M, F);
}

}  // namespace lf
