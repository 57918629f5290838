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
// Where tiles are few and K is long, the K blocks of a tile are split over the two to
// four pairs of a cluster, which exchange their sums through shared memory.
//
// The roles, barriers and bounded waits are those of gemm_nt_pair.cu (whole
// tiles only: nothing here waits for a pair of another cluster).
#include <atomic>
#include <type_traits>

#include "activations.cuh"
#include "gated_common.cuh"

namespace lf {
namespace {

constexpr int L_CHUNK = 64;  // columns of one store
constexpr int L_MAX_SPLIT = 4;  // pairs that share a tile: clusters of up to eight CTAs
constexpr int64_t L_SPLIT_COST = 4500;  // of exchanging sums, in rows of one K block (plan_linear_pair)
// The ring: stages of G_KSUB slots of one K block each, 128 rows of x and cols / 2 rows
// of w; narrow tiles have a stage more.
constexpr int L_MAX_STAGES = 4;
constexpr int L_RING = G_SLOTS * G_SLOT_BYTES;
__host__ __device__ constexpr int l_slot_bytes(int cols) { return G_A_BYTES + cols / 2 * G_ROW; }
__host__ __device__ constexpr int l_stages(int cols)
{
    return L_RING / (G_KSUB * l_slot_bytes(cols)) < L_MAX_STAGES ? L_RING / (G_KSUB * l_slot_bytes(cols)) : L_MAX_STAGES;
}
static_assert(l_stages(BN) == G_STAGES && l_stages(L_CHUNK) == L_MAX_STAGES, "stages that fit the ring");
static_assert(BM * BN * 4 <= L_RING, "a tile's sums fit the idle ring");
// its barriers, and one for each epilogue warp's residual
constexpr int L_NUM_BARS = 2 * L_MAX_STAGES + 2 * G_ACC_BUFS + 1 + G_EPI_WARPS;
static_assert(L_RING + L_NUM_BARS * 8 + 16 <= G_STG_OFF, "barriers before the staging buffers");

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

// What an epilogue warp does with 32 rows x 64 columns of sums.
template <bool E4M3, int ACT>
struct LinearFinish {
    const LinearParams &lp;
    const CUtensorMap &tmO, &tmP, &tmR;
    uint8_t *stg;  // the warp's staging buffer
    uint32_t stg_s, res_bar, res_phase = 0;
    volatile int *abort_flag;
    uint32_t peer_abort;
    __device__ LinearFinish(const LinearParams &l, const CUtensorMap &o, const CUtensorMap &pre, const CUtensorMap &r,
                            uint8_t *s, uint32_t ss, uint32_t bar, volatile int *flag, uint32_t peer)
        : lp(l), tmO(o), tmP(pre), tmR(r), stg(s), stg_s(ss), res_bar(bar), abort_flag(flag), peer_abort(peer)
    {
    }
    __device__ bool wanted(int row0, int col) const { return col < lp.g.N && row0 < lp.g.M; }
    // The residual's copy into the staging buffer.
    __device__ void load_residual(int row0, int col) const
    {
        stage_begin();
        if ((threadIdx.x & 31) == 0) {
            mbar_arrive_expect_tx(res_bar, G_STG_WARP);
            tma_load_2d(stg_s, &tmR, col, row0, res_bar);
        }
    }
    // Before the sums are complete: starts that copy for the piece to come (if `any`),
    // unless z goes through the staging buffer first.  True if it did.
    __device__ bool begin(int row0, int col, bool any) const
    {
        const bool now = lp.residual && !lp.save && any && wanted(row0, col);
        if (now)
            load_residual(row0, col);
        return now;
    }
    // The piece at (row0, col): this thread's row is row0 + lane.  False after a wait that gave up.
    __device__ bool chunk(float (&f)[2][32], float sx, int row0, int col, bool begun)
    {
        const GemmParams &p = lp.g;
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
        if (lp.residual && !begun)
            load_residual(row0, col);
#pragma unroll
        for (int half = 0; half < 2; ++half)
            l_activate<ACT>(f[half]);
        if (lp.residual) {
            if (!__all_sync(0xffffffffu, wait_bar(res_bar, res_phase, abort_flag, p, ERR_EPI, peer_abort)))
                return false;
            res_phase ^= 1u;
            l_add_staged(f[0], stg, 0);
            l_add_staged(f[1], stg, 1);
        } else {
            stage_begin();
        }
        stage_half(stg, 0, f[0]);
        stage_half(stg, 1, f[1]);
        stage_end(&tmO, stg_s, col, row0, p.M);
        return true;
    }
};

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
    const uint32_t bar0 = base + L_RING;
    const uint32_t drain_bar = bar0 + 8u * (2 * L_MAX_STAGES + 2 * G_ACC_BUFS);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + L_RING + L_NUM_BARS * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
#define FULL_BAR(s) (bar0 + 8u * (s))
#define EMPTY_BAR(s) (bar0 + 8u * (L_MAX_STAGES + (s)))
#define TFULL_BAR(b) (bar0 + 8u * (2 * L_MAX_STAGES + (b)))
#define TEMPTY_BAR(b) (bar0 + 8u * (2 * L_MAX_STAGES + G_ACC_BUFS + (b)))
#define RES_BAR(w) (bar0 + 8u * (2 * L_MAX_STAGES + 2 * G_ACC_BUFS + 1 + (w)))

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t cta = cluster_ctarank();
    const uint32_t rank = cta & 1u;        // in the pair
    const uint32_t lead = cta & ~1u;       // the pair's leader in the cluster
    const bool leader = rank == 0;
    const int split = lp.split;
    const int part = static_cast<int>(cta >> 1);  // this pair's share of the K blocks
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.num_k_blocks) * part / split);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.num_k_blocks) * (part + 1) / split);
    const int first_tile = static_cast<int>(blockIdx.x >> 1) / split;
    const int tile_step = static_cast<int>(gridDim.x >> 1) / split;
    const int cols = lp.cols;
    const int stages = l_stages(cols);
    const uint32_t slot_bytes = static_cast<uint32_t>(l_slot_bytes(cols));

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
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
    const uint32_t peer_abort = mapa_shared(smem_u32(const_cast<int *>(abort_flag)), cta ^ 1u);

    LinearFinish<E4M3, ACT> finish(lp, tmO, tmP, tmR, gbase + G_STG_OFF + (warp - 2) * G_STG_WARP,
                                         base + static_cast<uint32_t>(G_STG_OFF + (warp - 2) * G_STG_WARP),
                                         RES_BAR(warp - 2), abort_flag, peer_abort);
    if (warp == 0) {
        // ------------------------------------------------ TMA producer (both CTAs)
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            uint32_t armed[L_MAX_STAGES];
#pragma unroll
            for (int s = 0; s < L_MAX_STAGES; ++s)
                armed[s] = 0;
            bool ok = true, first = true;
            for (int tile = first_tile; ok && tile < p.num_tiles; tile += tile_step) {
                int mb, nb;
                g_tile_coords(p, tile, mb, nb);
                const int arow = mb * G_M + static_cast<int>(rank) * BM;
                const int brow = nb * cols + static_cast<int>(rank) * (cols / 2);
                for (int kb = kb0; kb < kb1; kb += G_KSUB) {
                    const int nsub = min(G_KSUB, kb1 - kb);
                    if (!wait_bar(EMPTY_BAR(stage), phase ^ 1u, abort_flag, p, ERR_PRODUCER, peer_abort)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full_leader = mapa_shared(FULL_BAR(stage), lead);
                    const bool skip = first && p.inject == 1 && blockIdx.x == 0;  // test hook
                    first = false;
                    if (!skip) {
                        if (leader) {
                            mbar_arrive_expect_tx(FULL_BAR(stage), 2u * slot_bytes * static_cast<uint32_t>(nsub));
                            ++armed[stage];
                        }
#pragma unroll
                        for (int j = 0; j < G_KSUB; ++j) {
                            if (j >= nsub)
                                break;
                            const uint32_t slot = base + static_cast<uint32_t>(stage * G_KSUB + j) * slot_bytes;
                            tma_load_2d_pair(slot, &tmA, (kb + j) * KELEMS, arow, full_leader);
                            tma_load_2d_pair(slot + G_A_BYTES, &tmW, (kb + j) * KELEMS, brow, full_leader);
                        }
                    }
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (leader)
                for (int s = 0; s < stages; ++s)
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
            const uint16_t both_ctas = static_cast<uint16_t>(3u << lead);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool alive = true;
            const uint32_t idesc = E4M3 ? idesc_e4m3_f32(G_M, cols) : idesc_bf16_f32(G_M, cols);
            for (int tile = first_tile; tile < p.num_tiles; tile += tile_step) {
                if (alive)
                    alive = __all_sync(0xffffffffu, wait_bar(TEMPTY_BAR(acc), acc_phase ^ 1u, abort_flag, p, ERR_MMA_ACC,
                                                             peer_abort));
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
                for (int kb = kb0; kb < kb1; kb += G_KSUB) {
                    const int nsub = min(G_KSUB, kb1 - kb);
                    if (alive)
                        alive = __all_sync(0xffffffffu, wait_bar(FULL_BAR(stage), phase, abort_flag, p, ERR_MMA_FULL,
                                                                 peer_abort));
                    if (alive) {
                        tc_fence_after();
#pragma unroll
                        for (int j = 0; j < G_KSUB; ++j) {
                            if (j >= nsub)
                                break;
                            const uint32_t a0 = base + static_cast<uint32_t>(stage * G_KSUB + j) * slot_bytes;
                            const uint32_t b0 = a0 + G_A_BYTES;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {  // 32 bytes of K per MMA
                                const uint64_t da = smem_desc_k128(a0 + k * 32), db = smem_desc_k128(b0 + k * 32);
                                const uint32_t accumulate = (kb != kb0 || j != 0 || k != 0) ? 1u : 0u;
                                if (E4M3)
                                    umma_f8_pair_one(one, d_tmem, da, db, idesc, accumulate);
                                else
                                    umma_f16_pair_one(one, d_tmem, da, db, idesc, accumulate);
                            }
                        }
                        umma_commit_pair_mc_one(one, EMPTY_BAR(stage), both_ctas);
                    }
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (alive)
                    umma_commit_pair_mc_one(one, TFULL_BAR(acc), both_ctas);
                if (++acc == G_ACC_BUFS) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
            umma_commit_pair_mc_one(one, drain_bar, static_cast<uint16_t>(1u << lead));
            if (lane == 0)
                wait_bar_drain(drain_bar, 0u, abort_flag, p, peer_abort);
        }
        __syncwarp();
    } else if (split == 1) {
        // ------------------------------------------------ epilogue (both CTAs)
        // warp w reads TMEM lanes 32 (w % 4) ..; warps 2..5 take the tile's even
        // chunks of 64 columns, warps 6..9 the odd ones
        const int q = warp & 3;
        const int first = warp >= 2 + G_EPI_WARPS / 2 ? L_CHUNK : 0;
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        for (int tile = first_tile; tile < p.num_tiles; tile += tile_step) {
            int mb, nb;
            g_tile_coords(p, tile, mb, nb);
            const int row0 = mb * G_M + static_cast<int>(rank) * BM + q * 32;
            const float sx = E4M3 && row0 + lane < p.M ? lp.x_scale[row0 + lane] : 0.f;  // loaded during the wait
            bool begun = finish.begin(row0, nb * cols + first, first < cols);
            ok = __all_sync(0xffffffffu, wait_bar(TFULL_BAR(acc), acc_phase, abort_flag, p, ERR_EPI, peer_abort));
            if (!ok)
                break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + static_cast<uint32_t>(acc * BN) + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
            for (int c = first; ok && c < cols && finish.wanted(row0, nb * cols + c); c += 2 * L_CHUNK, begun = false) {
                float f[2][32];
                load_acc2(taddr + static_cast<uint32_t>(c), taddr + static_cast<uint32_t>(c + 32), f[0], f[1]);
                ok = finish.chunk(f, sx, row0, nb * cols + c, begun);
            }
            if (!ok)
                break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(mapa_shared(TEMPTY_BAR(acc), lead));
            if (++acc == G_ACC_BUFS) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
    } else {
        // ------------------------------------------------ sums to shared memory (the cluster's one tile)
        // [column / 4][row][4], in the idle ring
        const int q = warp & 3;
        const bool ok = __all_sync(0xffffffffu, wait_bar(TFULL_BAR(0), 0u, abort_flag, p, ERR_EPI, peer_abort));
        tc_fence_after();
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
        float4 *sums = reinterpret_cast<float4 *>(gbase) + q * 32 + lane;
#pragma unroll 1
        for (int c = warp >= 2 + G_EPI_WARPS / 2 ? L_CHUNK : 0; ok && c < cols; c += 2 * L_CHUNK) {
            float f[2][32];
            load_acc2(taddr + static_cast<uint32_t>(c), taddr + static_cast<uint32_t>(c + 32), f[0], f[1]);
#pragma unroll
            for (int i = 0; i < 64; i += 4)
                sums[(c + i) / 4 * BM] = make_float4(f[i / 32][i % 32], f[i / 32][i % 32 + 1], f[i / 32][i % 32 + 2],
                                                     f[i / 32][i % 32 + 3]);
        }
        tc_fence_before();
        __syncwarp();
    }
    if (split > 1) {
        // Every pair's sums are in place: the 32-row, 64-column pieces of this CTA's rows
        // go round the pairs, each added up from its pair's sums on, round the cluster.
        int mb, nb;
        g_tile_coords(p, first_tile, mb, nb);
        const int pieces = 4 * (cols / L_CHUNK);
        const auto row_of = [&](int i) { return mb * G_M + static_cast<int>(rank) * BM + (i & 3) * 32; };
        const auto col_of = [&](int i) { return nb * cols + (i >> 2) * L_CHUNK; };
        int piece = part + split * (warp - 2);
        bool begun = warp >= 2 && finish.begin(row_of(piece), col_of(piece), piece < pieces);
        __syncwarp();
        cluster_sync();
        bool ok = __all_sync(0xffffffffu, !*abort_flag);
        for (; warp >= 2 && ok && piece < pieces; piece += split * G_EPI_WARPS, begun = false) {
            const int row0 = row_of(piece), col = col_of(piece);
            if (!finish.wanted(row0, col))
                continue;
            const float sx = E4M3 && row0 + lane < p.M ? lp.x_scale[row0 + lane] : 0.f;
            float f[2][32];
            const uint32_t at = base + static_cast<uint32_t>(((piece >> 2) * (L_CHUNK / 4) * BM + (piece & 3) * 32 + lane) * 16);
            for (int r = 0; r < split; ++r) {
                const int of = part + r < split ? part + r : part + r - split;
                const uint32_t from = mapa_shared(at, 2u * static_cast<uint32_t>(of) + rank);
#pragma unroll
                for (int i = 0; i < 64; i += 4) {
                    const float4 v = ld_cluster_f32x4(from + static_cast<uint32_t>(i / 4 * BM * 16));
                    float *o = &f[i / 32][i % 32];
                    o[0] = r ? o[0] + v.x : v.x;
                    o[1] = r ? o[1] + v.y : v.y;
                    o[2] = r ? o[2] + v.z : v.z;
                    o[3] = r ? o[3] + v.w : v.w;
                }
            }
            ok = finish.chunk(f, sx, row0, col, begun);
        }
    }
    if (warp >= 2 && lane == 0)
        bulk_wait_group_all();
    __syncwarp();
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
    return launch_overlapped(k_linear_pair<E4M3, ACT>, dim3(static_cast<unsigned>(grid)), dim3(G_THREADS), G_SMEM,
                             2 * p.split, s, m.x, m.w, m.out, m.pre, m.residual, p);
}

// ---------------------------------------------------------------- few tokens
// Up to 128 tokens (and groups of them where tiles are few and K long, see
// plan_linear_skinny): the weights' bytes bound the call, so the operands are swapped --
// 128 rows of w are the A operand of a 128 x n MMA whose B operand is the tokens (n:
// M rounded up to 16) -- and a CTA only streams its share of w through a ring of
// stages, one K block of 128 bytes each.  The K blocks of a tile of 128 output columns
// are split over a cluster of up to eight CTAs, so that most SMs stream: each leaves
// its fp32 sums in its own shared memory, and after a cluster barrier every CTA adds its
// part of the tokens from all of them, its own first and then round the cluster (so they
// do not all read the same CTA at once).
constexpr int LS_THREADS = 192;  // producer, MMA, 4 epilogue warps
constexpr int LS_WARPS = LS_THREADS / 32;
constexpr int LS_MAX_STAGES = 12;
constexpr int LS_BATCH = 4;
constexpr int LS_W_BYTES = BM * G_ROW;
constexpr int LS_MISC = 1024 + (2 * LS_MAX_STAGES + 1) * 8 + 32;  // alignment, barriers, TMEM address, abort flag
constexpr int LS_SMEM_ONE = 220 * 1024, LS_SMEM_TWO = 113 * 1024;  // with one / two CTAs per SM

__device__ __forceinline__ float4 bf16x4(uint2 u)
{
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}

// Four output columns of one token, from their sums z: `at` is where they go.
template <bool E4M3, int ACT>
__device__ __forceinline__ void s_finish(const LinearParams &lp, float4 z, float sx, float4 w4, float4 b4,
                                         bool residual, uint2 res, __nv_bfloat16 *pre, size_t at)
{
    if (E4M3)
        z = make_float4(z.x * sx * w4.x, z.y * sx * w4.y, z.z * sx * w4.z, z.w * sx * w4.w);
    z = make_float4(z.x + b4.x, z.y + b4.y, z.z + b4.z, z.w + b4.w);
    if (!E4M3 && pre)
        *reinterpret_cast<uint2 *>(pre + at) = make_uint2(pack_bf16(z.x, z.y), pack_bf16(z.z, z.w));
    if (ACT != ACT_NONE) {
        const float2 u = act_phi<ACT>(make_float2(z.x, z.y)), v = act_phi<ACT>(make_float2(z.z, z.w));
        z = make_float4(z.x * u.x, z.y * u.y, z.z * v.x, z.w * v.y);
    }
    if (residual) {
        const float4 t = bf16x4(res);
        z = make_float4(z.x + t.x, z.y + t.y, z.z + t.z, z.w + t.w);
    }
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(lp.g.out) + at) =
        make_uint2(pack_bf16(z.x, z.y), pack_bf16(z.z, z.w));
}

template <bool E4M3, int ACT>
__global__ void __launch_bounds__(LS_THREADS, 2)
    k_linear_skinny(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                    const __grid_constant__ LinearParams lp, const LinearSkinny plan, const __nv_bfloat16 *residual,
                    __nv_bfloat16 *pre)
{
    const GemmParams &p = lp.g;
    constexpr int KELEMS = E4M3 ? 128 : 64;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const uint32_t stage_bytes = LS_W_BYTES + static_cast<uint32_t>(plan.n) * G_ROW;
    const uint32_t bar0 = base + static_cast<uint32_t>(plan.stages) * stage_bytes;
    const uint32_t done_bar = bar0 + 8u * (2 * LS_MAX_STAGES);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + (done_bar + 8u - base));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
#define FULL_BAR(s) (bar0 + 8u * (s))
#define EMPTY_BAR(s) (bar0 + 8u * (LS_MAX_STAGES + (s)))
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int split = plan.split;
    const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int f0 = static_cast<int>(blockIdx.x) / split * BM;
    const int m0 = static_cast<int>(blockIdx.y) * plan.tokens;  // this CTA's tokens: m0 .. m0 + M - 1
    const int M = min(plan.tokens, p.M - m0);
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.num_k_blocks) * rank / split);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.num_k_blocks) * (rank + 1) / split);
    uint32_t cols = 32;
    while (cols < static_cast<uint32_t>(plan.n))
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
    // What this thread finishes with, loaded while the weights stream: the scales and
    // the bias of its four output columns, the scales of the warp's tokens m_first + 6 i
    // (in lane i), the residual of the first four of them.
    const int f = f0 + 4 * lane;
    const int m_first = M * rank / split + warp, m_end = M * (rank + 1) / split;
    float4 w4 = make_float4(1.f, 1.f, 1.f, 1.f), b4 = make_float4(0.f, 0.f, 0.f, 0.f);
    float sx_lane = 1.f;
    uint2 res[LS_BATCH];
    if (f < p.N) {  // N % 8 == 0
        if (E4M3)
            w4 = *reinterpret_cast<const float4 *>(lp.w_scale + f);
        if (lp.bias)
            b4 = lp.bias_f32 ? *reinterpret_cast<const float4 *>(static_cast<const float *>(lp.bias) + f)
                             : bf16x4(*reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(lp.bias) + f));
    }
    const auto load_residual = [&](int i0) {
#pragma unroll
        for (int j = 0; j < LS_BATCH; ++j) {
            const int m = m_first + LS_WARPS * (i0 + j);
            if (residual && f < p.N && m < m_end)
                res[j] = *reinterpret_cast<const uint2 *>(residual + static_cast<size_t>(m0 + m) * p.N + f);
        }
    };
    load_residual(0);
    if (E4M3 && m_first + LS_WARPS * lane < m_end)
        sx_lane = lp.x_scale[m0 + m_first + LS_WARPS * lane];

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
                    tma_load_2d(dst + LS_W_BYTES, &tmX, kb * KELEMS, m0, FULL_BAR(stage));
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
                const uint32_t ws = base + stage * stage_bytes, xs = ws + LS_W_BYTES;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t accumulate = (kb != kb0 || k != 0) ? 1u : 0u;
                    if (E4M3)
                        umma_f8(tmem_base, smem_desc_k128(ws + k * 32), smem_desc_k128(xs + k * 32), idesc, accumulate);
                    else
                        umma_f16(tmem_base, smem_desc_k128(ws + k * 32), smem_desc_k128(xs + k * 32), idesc, accumulate);
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
        float *part = reinterpret_cast<float *>(gbase) + q * 32 + lane;  // the ring is idle: [M][128] sums
        for (int c = 0; ok && c < M; c += 16) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(taddr + static_cast<uint32_t>(c), v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c + i < M)
                    part[(c + i) * BM] = __uint_as_float(v[i]);
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
    // (LS_BATCH tokens' sums are on their way at a time, or one token's from four CTAs)
    const int tokens = m_first < m_end ? (m_end - m_first + LS_WARPS - 1) / LS_WARPS : 0;  // of this warp
    const auto finish = [&](auto batch, int i0) {
        constexpr int B = decltype(batch)::value;
        float4 z[B];
#pragma unroll
        for (int j = 0; j < B; ++j)
            z[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll(B == 1 ? 4 : 1)
        for (int i = 0; i < split; ++i) {
            const uint32_t r = static_cast<uint32_t>(rank + i < split ? rank + i : rank + i - split);
#pragma unroll
            for (int j = 0; j < B; ++j) {
                const int m = min(m_first + LS_WARPS * (i0 + j), m_end - 1);
                const uint32_t a = base + static_cast<uint32_t>((m * BM + 4 * lane) * 4);
                const float4 d = ld_cluster_f32x4(split > 1 ? mapa_shared(a, r) : a);
                z[j] = make_float4(z[j].x + d.x, z[j].y + d.y, z[j].z + d.z, z[j].w + d.w);
            }
        }
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const int m = m_first + LS_WARPS * (i0 + j);
            const float sx = E4M3 ? __shfl_sync(0xffffffffu, sx_lane, i0 + j) : 1.f;
            if (m < m_end && f < p.N)
                s_finish<E4M3, ACT>(lp, z[j], sx, w4, b4, residual != nullptr, res[j], pre,
                                    static_cast<size_t>(m0 + m) * p.N + f);
        }
    };
    for (int i0 = 0; i0 < tokens; i0 += LS_BATCH) {
        if (i0 > 0)
            load_residual(i0);
        if (tokens - i0 == 1)
            finish(std::integral_constant<int, 1>(), i0);
        else
            finish(std::integral_constant<int, LS_BATCH>(), i0);
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
cudaError_t launch_linear_skinny_t(const LinearMaps &m, const LinearParams &p, const LinearSkinny &plan,
                                   const void *residual, void *pre, cudaStream_t s)
{
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load() & bit)) {
        e = cudaFuncSetAttribute(k_linear_skinny<E4M3, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize, LS_SMEM_ONE);
        if (e != cudaSuccess)
            return e;
        done.fetch_or(bit);
    }
    return launch_overlapped(k_linear_skinny<E4M3, ACT>,
                             dim3(static_cast<unsigned>(p.g.num_n_blocks * plan.split),
                                  static_cast<unsigned>((p.g.M + plan.tokens - 1) / plan.tokens)),
                             dim3(LS_THREADS), static_cast<size_t>(plan.smem), plan.split, s, m.x, m.w, p, plan,
                             static_cast<const __nv_bfloat16 *>(residual), static_cast<__nv_bfloat16 *>(pre));
}

// ---------------------------------------------------------------- gradient
// dz = dout act'(z) from the kept z, rounded to bf16 once for the products that read
// it, and the column sums of the unrounded dz, the bias's gradient: bound by HBM.  A
// block takes 128 columns (16 threads of 8) and every 16th row of its share of the
// rows; its sums over the 16 rows of threads are added in order.  Where up to eight blocks
// share the rows they are a cluster, which adds up their sums through shared memory
// (`shared`; blockIdx.x is then the share, blockIdx.y the columns); more write them to rows
// of `partial`, which k_linear_dbias adds up (333 x 5632 without an activation, with both
// products: 32.0 us with that kernel, 30.3 in clusters).  Without an activation dz is dout
// itself and only the sums are left.
constexpr int DZ_COLS = 128, DZ_ROWS = 16, DZ_CLUSTER = 8;

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
                int bias_f32, int64_t M, int64_t N, int64_t rows, int shared)
{
    wait_previous_kernel();
    let_next_kernel_start();
    __shared__ float sh[DZ_ROWS][DZ_COLS];
    __shared__ float total[DZ_COLS];
    const int tx = threadIdx.x % (DZ_COLS / 8), ty = threadIdx.x / (DZ_COLS / 8);
    const int64_t strip = shared ? blockIdx.y : blockIdx.x, share = shared ? blockIdx.x : blockIdx.y;
    const int64_t c = strip * DZ_COLS + tx * 8;
    const int64_t r0 = share * rows, r1 = r0 + rows < M ? r0 + rows : M;
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
    const int64_t col = strip * DZ_COLS + threadIdx.x;
    const bool mine = threadIdx.x < DZ_COLS && col < N;
    float s = 0.f;
    if (mine) {
#pragma unroll
        for (int i = 0; i < DZ_ROWS; ++i)
            s += sh[i][threadIdx.x];
    }
    const auto put = [&](float v) {
        if (bias_f32)
            static_cast<float *>(dbias)[col] = v;
        else
            static_cast<__nv_bfloat16 *>(dbias)[col] = __float2bfloat16_rn(v);
    };
    if (shared > 1) {
        if (mine)
            total[threadIdx.x] = s;
        cluster_sync();
        if (mine && threadIdx.x % shared == share) {  // every block finishes a part of the columns
            s = 0.f;
            for (int b = 0; b < shared; ++b)
                s += ld_cluster_f32(mapa_shared(smem_u32(&total[threadIdx.x]), b));
            put(s);
        }
        cluster_sync();  // no block leaves while its sums are read
        return;
    }
    if (!mine)
        return;
    if (partial)
        partial[share * N + col] = s;
    else
        put(s);
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

// Clusters of `size` CTAs with `smem` bytes of shared memory each that the device holds at
// once, -1 if it holds none.
template <class K>
static int max_clusters(K kernel, int size, int threads, int smem)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(size), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(size);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = -1;
    }
    return n;
}

// Clusters of `split` pairs that the device holds at once (k_linear_pair).
static int linear_pair_clusters(int split, int pairs)
{
    static std::atomic<int> known[L_MAX_SPLIT + 1][64];
    int dev = 0;
    if (split == 1 || cudaGetDevice(&dev) != cudaSuccess)
        return pairs;
    std::atomic<int> &k = known[split][dev & 63];
    int n = k.load();
    if (n == 0) {
        n = max_clusters(k_linear_pair<false, ACT_NONE>, 2 * split, G_THREADS, G_SMEM);
        k.store(n);
    }
    return n;
}

// Columns of a tile and pairs that share its K blocks.  A K block costs 128 rows of x
// and cols / 2 rows of w for each CTA, however many tensor operations that feeds (one wave
// of narrow tiles moves about 100 GB/s into every SM), and exchanging sums as much as
// L_SPLIT_COST of those rows, 3 us:
//   256 x 5120 x 13824 47.0 us unsplit, 35.9 in three; 256 x 2048 x 5632 19.8 and 16.0;
//   512 x 4096 x 4096 18.8 and, in two, 20.8; 256 x 2048 x 2048 10.5 and, in two, 11.6.
void plan_linear_pair(int m_blocks, int64_t N, int num_k_blocks, int pairs, int *best_cols, int *best_split)
{
    int64_t least = 0;
    *best_cols = 0;
    for (int split = 1; split <= L_MAX_SPLIT; ++split) {
        if (split > 1 && num_k_blocks < 4 * split)
            break;
        for (int cols = BN; cols >= L_CHUNK; cols -= L_CHUNK) {
            const int64_t tiles = (N + cols - 1) / cols * m_blocks;
            if (split > 1 && tiles > linear_pair_clusters(split, pairs))
                break;
            const int64_t waves = split > 1 ? 1 : (tiles + pairs - 1) / pairs;
            const int64_t t = waves * ((num_k_blocks + split - 1) / split) * (BM + cols / 2) + (split > 1 ? L_SPLIT_COST : 0);
            if (*best_cols == 0 || t < least) {
                least = t;
                *best_cols = cols;
                *best_split = split;
            }
        }
    }
}

// Clusters of `split` few-token CTAs (one per SM) that the device holds at once.
static int linear_clusters(int split, int num_sms)
{
    static std::atomic<int> known[9][64];
    int dev = 0;
    if (split == 1 || cudaGetDevice(&dev) != cudaSuccess)
        return num_sms;
    std::atomic<int> &k = known[split][dev & 63];
    int n = k.load();
    if (n == 0) {
        n = max_clusters(k_linear_skinny<false, ACT_NONE>, split, LS_THREADS, LS_SMEM_ONE);
        k.store(n);
    }
    return n;
}

LinearSkinny plan_linear_skinny(int64_t M, int64_t N, int num_k_blocks, int num_sms)
{
    LinearSkinny g;
    const int64_t groups = (M + BM - 1) / BM;
    g.tokens = groups == 1 ? static_cast<int>(M) : static_cast<int>(((M + groups - 1) / groups + 15) / 16 * 16);
    g.n = (g.tokens + 15) / 16 * 16;
    const int64_t tiles = (N + BM - 1) / BM * groups;
    // The largest split whose clusters are one wave, with four K blocks for each CTA at
    // least.  More tiles than SMs: two CTAs per SM while the sums fit half an SM's ring.
    const bool two = g.n <= 64 && tiles > num_sms;
    g.split = 1;
    for (int split = 2; split <= 8 && num_k_blocks / split >= 4; ++split)
        if (tiles <= linear_clusters(split, num_sms))
            g.split = split;
    const int stage = LS_W_BYTES + g.n * G_ROW;
    // Half the ring for few tokens and short shares of K, too: the next call's CTAs can start
    // beside this one's (us with all / half of it, K to N [K blocks of a CTA], one token: 5120 to
    // 5120 [27] 13.1 / 12.5, 4096 to 4096 [16] 10.0 / 9.3, 2048 to 5632 [11] 8.6 / 8.1, e4m3 5120 to 13824 [40]
    // 15.9 / 15.4; longer ones 13824 to 5120 [72] 26.0 / 26.7; 64 tokens 5120 to 5120 14.1 / 15.4).
    const bool lean = g.n <= 32 && (num_k_blocks + g.split - 1) / g.split <= 40;
    const int fit = ((two || lean ? LS_SMEM_TWO : LS_SMEM_ONE) - LS_MISC) / stage;
    g.stages = fit < LS_MAX_STAGES ? fit : LS_MAX_STAGES;
    g.smem = LS_MISC + g.stages * stage;
    // The choice between this kernel and the pair kernel (us, this one / the pair kernel,
    // bf16; e4m3 with twice the K alike).  Up to 16 tokens always this one.  Up to 128
    // where the K loop [K blocks] is long for the tokens:
    //   64 x .. x 512 [8] 5.2 / 4.9    64 x .. x 1024 [16] 6.3 / 7.3   64 x .. x 13824 [80] 29.2 / 33.7
    //   128 x .. x 1024 [16] 7.7 / 7.5  128 x .. x 2048 [32] 8.8 / 10.4  128 x .. x 5120 [216] 29.6 / 35.1
    // More, in groups, where a split makes up for reading w once for each group:
    //   split in four or more  144 x .. x 1024 [16] 6.4 / 7.5  256 x .. x 1024 [16] 7.8 / 7.6
    //                          256 x .. x 2048 [32] 9.7 / 10.5  512 x .. x 512 [128] 13.3 / 14.1
    //   in two or three        256 x .. x 4096 [64] 16.6 / 16.7  384 x .. x 2048 [88] 19.5 / 18.2
    //   unsplit                144 x .. x 5120 [80] 28.1 / 20.4
    if (groups == 1)
        g.preferred = g.n <= 16 || 4 * num_k_blocks >= g.n;
    else
        g.preferred = 6 * num_k_blocks >= g.n && (g.split >= 4 || (g.split >= 2 && groups == 2));
    return g;
}

cudaError_t launch_linear_skinny(bool e4m3, int act, const LinearMaps &m, const LinearParams &p,
                                 const LinearSkinny &plan, const void *residual, void *pre, cudaStream_t s)
{
    switch (act + (e4m3 ? 4 : 0)) {
    case ACT_SILU:
        return launch_linear_skinny_t<false, ACT_SILU>(m, p, plan, residual, pre, s);
    case ACT_GELU:
        return launch_linear_skinny_t<false, ACT_GELU>(m, p, plan, residual, pre, s);
    case ACT_GELU_TANH:
        return launch_linear_skinny_t<false, ACT_GELU_TANH>(m, p, plan, residual, pre, s);
    case ACT_NONE:
        return launch_linear_skinny_t<false, ACT_NONE>(m, p, plan, residual, pre, s);
    case 4 + ACT_SILU:
        return launch_linear_skinny_t<true, ACT_SILU>(m, p, plan, residual, pre, s);
    case 4 + ACT_GELU:
        return launch_linear_skinny_t<true, ACT_GELU>(m, p, plan, residual, pre, s);
    case 4 + ACT_GELU_TANH:
        return launch_linear_skinny_t<true, ACT_GELU_TANH>(m, p, plan, residual, pre, s);
    case 4 + ACT_NONE:
        return launch_linear_skinny_t<true, ACT_NONE>(m, p, plan, residual, pre, s);
    }
    return cudaErrorInvalidValue;
}

// Blocks that share the rows of a strip of columns.
static int dz_blocks(int64_t M, int64_t N)
{
    const int64_t strips = (N + DZ_COLS - 1) / DZ_COLS, want = (152 * 8 + strips - 1) / strips;
    const int64_t most = (M + 4 * DZ_ROWS - 1) / (4 * DZ_ROWS);  // four rows for each thread at least
    return static_cast<int>(want < most ? want : most);
}
int linear_dz_blocks(int64_t M, int64_t N)
{
    const int blocks = dz_blocks(M, N);
    return blocks > DZ_CLUSTER ? blocks : 1;
}

cudaError_t launch_linear_dz(int act, const void *dout, const void *pre, void *dz, float *partial, void *dbias,
                             bool bias_f32, int64_t M, int64_t N, cudaStream_t s)
{
    const int blocks = dz_blocks(M, N);
    const int64_t rows = ((M + blocks - 1) / blocks + DZ_ROWS - 1) / DZ_ROWS * DZ_ROWS;
    const int shared = dbias && blocks > 1 && blocks <= DZ_CLUSTER ? blocks : 0;  // (strips: fewer than 1216 then)
    const unsigned strips = static_cast<unsigned>((N + DZ_COLS - 1) / DZ_COLS), shares = static_cast<unsigned>(blocks);
    const auto kernel = act == ACT_SILU        ? k_linear_dz<ACT_SILU>
                        : act == ACT_GELU      ? k_linear_dz<ACT_GELU>
                        : act == ACT_GELU_TANH ? k_linear_dz<ACT_GELU_TANH>
                                               : k_linear_dz<ACT_NONE>;
    return launch_overlapped(kernel, shared ? dim3(shares, strips) : dim3(strips, shares), dim3(256), 0, shared ? shared : 1,
                             s, static_cast<const __nv_bfloat16 *>(dout), static_cast<const __nv_bfloat16 *>(pre),
                             static_cast<__nv_bfloat16 *>(dz), dbias && blocks > DZ_CLUSTER ? partial : nullptr, dbias,
                             bias_f32 ? 1 : 0, M, N, rows, shared);
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
