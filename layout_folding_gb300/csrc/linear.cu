// linear.cu -- a projection with everything that follows it in its epilogue,
//   z = x w^T (times the scales of e4m3 operands) + bias,
//   out = act(z) + residual,
// and the elementwise part of its gradient, dz = dout act'(z) with its column sums.
//
// The product is the NT GEMM of gemm_nt_pair.cu on 256 x `cols` tiles (64 to 256
// columns, plan_linear_cols).  The accumulator leaves TMEM once, 64 columns of a
// warp's 32 rows at a time: bias, activation and residual are added in fp32 and the
// sum is rounded once, so neither z nor act(z) makes a trip through memory.  The
// residual arrives by the same boxes that the output leaves by, in the same staging
// buffer: its copy is started before the accumulator is complete and every thread
// replaces its own 16-byte pieces, which also makes an output over the residual safe.
//
// The roles, barriers and bounded waits are those of gemm_nt_pair.cu (whole
// tiles only: nothing here waits for another pair).
#include <atomic>

#include "activations.cuh"
#include "gated_common.cuh"

namespace lf {
namespace {

constexpr int L_CHUNK = 64;  // columns of one store
// The ring of gated_common.cuh, its barriers and one for each epilogue warp's residual.
constexpr int L_NUM_BARS = G_NUM_BARS + G_EPI_WARPS;
static_assert(G_SLOTS * G_SLOT_BYTES + L_NUM_BARS * 8 + 16 <= G_STG_OFF, "barriers before the staging buffers");

// 32 columns of the bias added to f; `valid` of them exist (N % 8 == 0).
__device__ __forceinline__ void l_add_bias(float (&f)[32], const LinearParams &lp, int col, int valid)
{
    if (!lp.bias)
        return;
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
        if (i < valid) {
            if (lp.bias_f32) {
                const float4 *b = reinterpret_cast<const float4 *>(static_cast<const float *>(lp.bias) + col + i);
                const float4 u = b[0], v = b[1];
                f[i] += u.x;
                f[i + 1] += u.y;
                f[i + 2] += u.z;
                f[i + 3] += u.w;
                f[i + 4] += v.x;
                f[i + 5] += v.y;
                f[i + 6] += v.z;
                f[i + 7] += v.w;
            } else {
                const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(lp.bias) + col + i);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f[i + 2 * j] += __uint_as_float(w[j] << 16);
                    f[i + 2 * j + 1] += __uint_as_float(w[j] & 0xffff0000u);
                }
            }
        }
    }
}

template <int ACT>
__device__ __forceinline__ void l_activate(float (&f)[32])
{
    if (ACT != ACT_NONE) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            const float2 v = make_float2(f[i], f[i + 1]);
            const float2 r = mul2(v, act_phi<ACT>(v));
            f[i] = r.x;
            f[i + 1] = r.y;
        }
    }
}

// Half 0 or 1 of this thread's 64 columns in the staging buffer added to f.
__device__ __forceinline__ void l_add_staged(float (&f)[32], const uint8_t *stg, int half)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 u = *reinterpret_cast<const uint4 *>(stg + lane * 128 + (((4 * half + j) ^ (lane & 7)) << 4));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[8 * j + 2 * i] += __uint_as_float(w[i] << 16);
            f[8 * j + 2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

template <bool E4M3, int ACT>
__global__ void __launch_bounds__(G_THREADS, 1)
    k_linear_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                  const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmP,
                  const __grid_constant__ CUtensorMap tmR, const __grid_constant__ LinearParams lp)
{
    const GemmParams &p = lp.g;
    constexpr int KELEMS = E4M3 ? 128 : 64;  // elements of K per block
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const uint32_t sA = base;
    const uint32_t sB = base + G_SLOTS * G_A_BYTES;
    const uint32_t bar0 = base + G_SLOTS * G_SLOT_BYTES;
    const uint32_t drain_bar = bar0 + 8u * (2 * G_STAGES + 2 * G_ACC_BUFS);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + G_SLOTS * G_SLOT_BYTES + L_NUM_BARS * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
#define FULL_BAR(s) (bar0 + 8u * (s))
#define EMPTY_BAR(s) (bar0 + 8u * (G_STAGES + (s)))
#define TFULL_BAR(b) (bar0 + 8u * (2 * G_STAGES + (b)))
#define TEMPTY_BAR(b) (bar0 + 8u * (2 * G_STAGES + G_ACC_BUFS + (b)))
#define RES_BAR(w) (bar0 + 8u * (G_NUM_BARS + (w)))

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1;
    const int num_pairs = gridDim.x >> 1;
    const int cols = lp.cols;

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
        for (int w = 0; w < G_EPI_WARPS; ++w)
            mbar_init(RES_BAR(w), 1);
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
            const uint32_t slot_bytes = 2u * static_cast<uint32_t>(G_A_BYTES + cols / 2 * G_ROW);
            uint32_t armed[G_STAGES];
#pragma unroll
            for (int s = 0; s < G_STAGES; ++s)
                armed[s] = 0;
            bool ok = true, first = true;
            for (int tile = pair; ok && tile < p.num_tiles; tile += num_pairs) {
                int mb, nb;
                g_tile_coords(p, tile, mb, nb);
                const int arow = mb * G_M + static_cast<int>(rank) * BM;
                const int brow = nb * cols + static_cast<int>(rank) * (cols / 2);
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
            const uint32_t idesc = E4M3 ? idesc_e4m3_f32(G_M, cols) : idesc_bf16_f32(G_M, cols);
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
        // warp w reads TMEM lanes 32 (w % 4) ..; warps 2..5 take the tile's even
        // chunks of 64 columns, warps 6..9 the odd ones
        const int q = warp & 3;
        const int first = warp >= 2 + G_EPI_WARPS / 2 ? L_CHUNK : 0;
        int acc = 0;
        uint32_t acc_phase = 0, res_phase = 0;
        uint8_t *stg = gbase + G_STG_OFF + (warp - 2) * G_STG_WARP;
        const uint32_t stg_s = base + static_cast<uint32_t>(G_STG_OFF + (warp - 2) * G_STG_WARP);
        const uint32_t res_bar = RES_BAR(warp - 2);
        bool ok = true;
        for (int tile = pair; ok && tile < p.num_tiles; tile += num_pairs) {
            int mb, nb;
            g_tile_coords(p, tile, mb, nb);
            const int row0 = mb * G_M + static_cast<int>(rank) * BM + q * 32;
            float sx = 1.f;  // the token's scale, loaded during the wait
            if (E4M3)
                sx = row0 + lane < p.M ? lp.x_scale[row0 + lane] : 0.f;
            // the residual of columns c .. c + 63, into the staging buffer
            const auto load_residual = [&](int c) {
                stage_begin();
                if (lane == 0) {
                    mbar_arrive_expect_tx(res_bar, G_STG_WARP);
                    tma_load_2d(stg_s, &tmR, nb * cols + c, row0, res_bar);
                }
            };
            const auto wanted = [&](int c) { return c < cols && nb * cols + c < p.N && row0 < p.M; };
            const bool early = lp.residual && !lp.save;
            if (early && wanted(first))
                load_residual(first);
            ok = __all_sync(0xffffffffu, wait_bar(TFULL_BAR(acc), acc_phase, abort_flag, p, ERR_EPI, peer_abort));
            if (!ok)
                break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + static_cast<uint32_t>(acc * BN) + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
            for (int c = first; ok && wanted(c); c += 2 * L_CHUNK) {
                const int col = nb * cols + c;
                float f[2][32];
                load_acc2(taddr + static_cast<uint32_t>(c), taddr + static_cast<uint32_t>(c + 32), f[0], f[1]);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    g_scale<E4M3>(f[half], sx, lp.w_scale + col + 32 * half, p.N - col - 32 * half);
                    l_add_bias(f[half], lp, col + 32 * half, p.N - col - 32 * half);
                }
                if (!E4M3 && lp.save) {
                    stage_begin();
                    stage_half(stg, 0, f[0]);
                    stage_half(stg, 1, f[1]);
                    stage_end(&tmP, stg_s, col, row0, p.M);
                }
                if (lp.residual && !(early && c == first))
                    load_residual(c);
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    l_activate<ACT>(f[half]);
                if (lp.residual) {
                    ok = __all_sync(0xffffffffu, wait_bar(res_bar, res_phase, abort_flag, p, ERR_EPI, peer_abort));
                    if (!ok)
                        break;
                    res_phase ^= 1u;
                    l_add_staged(f[0], stg, 0);
                    l_add_staged(f[1], stg, 1);
                } else {
                    stage_begin();
                }
                stage_half(stg, 0, f[0]);
                stage_half(stg, 1, f[1]);
                stage_end(&tmO, stg_s, col, row0, p.M);
            }
            if (!ok)
                break;
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
        __syncwarp();
    }
#undef FULL_BAR
#undef EMPTY_BAR
#undef TFULL_BAR
#undef TEMPTY_BAR
#undef RES_BAR

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
cudaError_t launch_linear_pair_t(const LinearMaps &m, const LinearParams &p, int grid, cudaStream_t s)
{
    static std::atomic<unsigned long long> done{0};  // the shared-memory opt-in, once per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load() & bit)) {
        e = cudaFuncSetAttribute(k_linear_pair<E4M3, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize, G_SMEM);
        if (e != cudaSuccess)
            return e;
        done.fetch_or(bit);
    }
    return launch_overlapped(k_linear_pair<E4M3, ACT>, dim3(static_cast<unsigned>(grid)), dim3(G_THREADS), G_SMEM, 2, s,
                             m.x, m.w, m.out, m.pre, m.residual, p);
}

// ---------------------------------------------------------------- gradient
// dz = dout act'(z) from the kept z, rounded to bf16 once for the products that read
// it, and the column sums of the unrounded dz, the bias's gradient: bound by HBM.  A
// block takes 128 columns (16 threads of 8) and every 16th row of its share of the
// rows; its sums over the 16 rows of threads are added in order and go to row
// blockIdx.y of `partial`, which k_linear_dbias adds up -- or to dbias, where one block
// has all rows.  Without an activation dz is dout itself and only the sums are left.
constexpr int DZ_COLS = 128, DZ_ROWS = 16;

template <class B>
__device__ __forceinline__ B bias_from(float v)
{
    return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 bias_from<__nv_bfloat16>(float v)
{
    return __float2bfloat16_rn(v);
}

template <int ACT>
__global__ void __launch_bounds__(256)
    k_linear_dz(const __nv_bfloat16 *dout, const __nv_bfloat16 *pre, __nv_bfloat16 *dz, float *partial, void *dbias,
                int bias_f32, int64_t M, int64_t N, int64_t rows)
{
    wait_previous_kernel();
    let_next_kernel_start();
    __shared__ float sh[DZ_ROWS][DZ_COLS];
    const int tx = threadIdx.x % (DZ_COLS / 8), ty = threadIdx.x / (DZ_COLS / 8);
    const int64_t c = static_cast<int64_t>(blockIdx.x) * DZ_COLS + tx * 8;
    const int64_t r0 = blockIdx.y * rows, r1 = r0 + rows < M ? r0 + rows : M;
    float sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        sum[i] = 0.f;
    if (c < N) {
#pragma unroll 2
        for (int64_t r = r0 + ty; r < r1; r += DZ_ROWS) {
            const uint4 dv = *reinterpret_cast<const uint4 *>(dout + r * N + c);
            const __nv_bfloat162 *d2 = reinterpret_cast<const __nv_bfloat162 *>(&dv);
            uint4 zv = make_uint4(0, 0, 0, 0);
            if (ACT != ACT_NONE)
                zv = *reinterpret_cast<const uint4 *>(pre + r * N + c);
            const __nv_bfloat162 *z2 = reinterpret_cast<const __nv_bfloat162 *>(&zv);
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 d = __bfloat1622float2(d2[i]);
                if (ACT != ACT_NONE) {
                    const float2 z = __bfloat1622float2(z2[i]);
                    const float2 p = act_phi<ACT>(z);
                    d.x *= fmaf(z.x, act_dphi<ACT>(z.x, p.x), p.x);
                    d.y *= fmaf(z.y, act_dphi<ACT>(z.y, p.y), p.y);
                    o[i] = pack_bf16(d.x, d.y);
                }
                sum[2 * i] += d.x;
                sum[2 * i + 1] += d.y;
            }
            if (ACT != ACT_NONE)
                *reinterpret_cast<uint4 *>(dz + r * N + c) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    if (!partial && !dbias)
        return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        sh[ty][tx * 8 + i] = sum[i];
    __syncthreads();
    const int64_t col = static_cast<int64_t>(blockIdx.x) * DZ_COLS + threadIdx.x;
    if (threadIdx.x >= DZ_COLS || col >= N)
        return;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < DZ_ROWS; ++i)
        s += sh[i][threadIdx.x];
    if (partial)
        partial[blockIdx.y * N + col] = s;
    else if (bias_f32)
        static_cast<float *>(dbias)[col] = s;
    else
        static_cast<__nv_bfloat16 *>(dbias)[col] = __float2bfloat16_rn(s);
}

// dbias[c] = the sum of the blocks' sums, in order.
template <class B>
__global__ void __launch_bounds__(256) k_linear_dbias(const float *partial, B *dbias, int64_t N, int blocks)
{
    wait_previous_kernel();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (c >= N)
        return;
    float s = 0.f;
#pragma unroll 8
    for (int b = 0; b < blocks; ++b)
        s += partial[b * N + c];
    dbias[c] = bias_from<B>(s);
}

}  // namespace

cudaError_t launch_linear_pair(bool e4m3, int act, const LinearMaps &m, const LinearParams &p, int grid, cudaStream_t s)
{
    switch (act + (e4m3 ? 4 : 0)) {
    case ACT_SILU:
        return launch_linear_pair_t<false, ACT_SILU>(m, p, grid, s);
    case ACT_GELU:
        return launch_linear_pair_t<false, ACT_GELU>(m, p, grid, s);
    case ACT_GELU_TANH:
        return launch_linear_pair_t<false, ACT_GELU_TANH>(m, p, grid, s);
    case ACT_NONE:
        return launch_linear_pair_t<false, ACT_NONE>(m, p, grid, s);
    case 4 + ACT_SILU:
        return launch_linear_pair_t<true, ACT_SILU>(m, p, grid, s);
    case 4 + ACT_GELU:
        return launch_linear_pair_t<true, ACT_GELU>(m, p, grid, s);
    case 4 + ACT_GELU_TANH:
        return launch_linear_pair_t<true, ACT_GELU_TANH>(m, p, grid, s);
    case 4 + ACT_NONE:
        return launch_linear_pair_t<true, ACT_NONE>(m, p, grid, s);
    }
    return cudaErrorInvalidValue;
}

// As plan_gated_cols: a K block costs 128 rows of x and cols / 2 rows of w for each CTA.
int plan_linear_cols(int m_blocks, int64_t N, int pairs)
{
    int best = 0;
    int64_t least = 0;
    for (int cols = BN; cols >= L_CHUNK; cols -= L_CHUNK) {
        const int64_t tiles = (N + cols - 1) / cols * m_blocks;
        const int64_t t = (tiles + pairs - 1) / pairs * (BM + cols / 2);
        if (best == 0 || t < least) {
            least = t;
            best = cols;
        }
    }
    return best;
}

// Rows of partial sums: none where one block takes all rows of its 128 columns.
int linear_dz_blocks(int64_t M, int64_t N)
{
    const int64_t strips = (N + DZ_COLS - 1) / DZ_COLS, want = (152 * 8 + strips - 1) / strips;
    const int64_t most = (M + 4 * DZ_ROWS - 1) / (4 * DZ_ROWS);  // four rows for each thread at least
    return static_cast<int>(want < most ? want : most);
}

cudaError_t launch_linear_dz(int act, const void *dout, const void *pre, void *dz, float *partial, void *dbias,
                             bool bias_f32, int64_t M, int64_t N, cudaStream_t s)
{
    const int blocks = linear_dz_blocks(M, N);
    const int64_t rows = ((M + blocks - 1) / blocks + DZ_ROWS - 1) / DZ_ROWS * DZ_ROWS;
    const dim3 grid(static_cast<unsigned>((N + DZ_COLS - 1) / DZ_COLS), static_cast<unsigned>(blocks));
    const auto kernel = act == ACT_SILU        ? k_linear_dz<ACT_SILU>
                        : act == ACT_GELU      ? k_linear_dz<ACT_GELU>
                        : act == ACT_GELU_TANH ? k_linear_dz<ACT_GELU_TANH>
                                               : k_linear_dz<ACT_NONE>;
    return launch_overlapped(kernel, grid, dim3(256), 0, 1, s, static_cast<const __nv_bfloat16 *>(dout),
                             static_cast<const __nv_bfloat16 *>(pre), static_cast<__nv_bfloat16 *>(dz),
                             dbias && blocks > 1 ? partial : nullptr, dbias, bias_f32 ? 1 : 0, M, N, rows);
}

cudaError_t launch_linear_dbias(const float *partial, void *dbias, bool bias_f32, int64_t M, int64_t N, cudaStream_t s)
{
    const int blocks = linear_dz_blocks(M, N);
    const dim3 grid(static_cast<unsigned>((N + 255) / 256));
    if (bias_f32)
        return launch_overlapped(k_linear_dbias<float>, grid, dim3(256), 0, 1, s, partial, static_cast<float *>(dbias), N,
                                 blocks);
    return launch_overlapped(k_linear_dbias<__nv_bfloat16>, grid, dim3(256), 0, 1, s, partial,
                             static_cast<__nv_bfloat16 *>(dbias), N, blocks);
}

}  // namespace lf
