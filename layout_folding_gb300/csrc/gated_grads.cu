// gated_grads.cu -- the two products of the gated projections' gradient,
//   dx[M, K] = dgu[M, 2F] . w[2F, K]      and      dw[2F, K] = dgu^T . x[M, K],
// in one persistent launch on CTA pairs (256 x 256 tiles, cta_group::2); and the same
// two of a plain projection's, with dz[M, N] in the place of dgu.
//
// No operand is transposed in memory: dgu is the K-major A operand of dx and the
// MN-major A operand of dw; w and x are MN-major B operands.
//
// Why one launch: each product alone leaves pairs idle in its last wave -- dx
// most of all, whose tiles are few and long (4096 x 5120 x 13824: 320 tiles of 432
// K blocks are 4.2 waves of 76 pairs, so a fifth wave for a fifth of the pairs).
// Here the pairs without a tile of that last wave start on the other product, whose
// tiles are short, and all of them end within one short tile of each other: 1240 us
// in a burst (1.87 PFLOP/s) where two launches took 685 + 636.  The schedule is
// fixed (GradIter), so no pair waits for another, replays of a captured call are
// the same, and every output is summed in the same order every time.  What
// bounds it: the tensor cores, and over many calls the power limit.
//
// A product with too few tiles to go round has its K blocks split: each part
// leaves its sums in fp32 in the caller's scratch, and a last, elementwise kernel
// adds the parts in their order.
#include <atomic>

#include "gated_common.cuh"

namespace lf {
namespace {

constexpr uint32_t GR_MN_HALF = G_A_BYTES / 2;  // an MN-major operand: two 64 x 64 boxes per K block
constexpr uint32_t GR_MN_KSTEP = 2 * 1024;      // 16 rows of K in it
// an MN-major descriptor of the ring's last slot can reach 8 KiB past the ring: barriers and staging follow it
static_assert(G_EPI_WARPS * G_STG_WARP >= 8192, "room past the ring for MN-major descriptors");

struct GradItem {
    int side, mb, nb, kb0, kb1, part;
};

// The items of one pair.  The side with the longer items first: pair, pair +
// pairs, ...; while the `extra` pairs that have one more of those run it, the
// others take `rounds` rounds of the other side's items; then all pairs take
// what is left, in turn.
struct GradIter {
    const GradsParams &p;
    int pair, pairs, phase = 0, i;
    int extra, head;  // items of the second side taken in the middle phase
    __device__ GradIter(const GradsParams &gp, int pr, int n) : p(gp), pair(pr), pairs(n), i(pr)
    {
        const GradSide &a = p.side[p.first], &b = p.side[p.first ^ 1];
        extra = a.items % pairs;
        head = extra ? min(b.items, p.rounds * (pairs - extra)) : 0;
    }
    __device__ bool next(GradItem &it)
    {
        for (;;) {
            const int s = phase == 0 ? p.first : p.first ^ 1;
            const int end = phase == 0 ? p.side[s].items : phase == 1 ? head : p.side[s].items;
            if (i < end) {
                decode(s, i, it);
                i += phase == 1 ? pairs - extra : pairs;
                return true;
            }
            if (phase == 2)
                return false;
            ++phase;
            if (phase == 1)
                i = extra && pair >= extra ? pair - extra : end + head;  // the pairs still on the first side skip it
            else
                i = head + pair;
        }
    }
    // (Kept to a few 32-bit divisions: the producer decodes between two items,
    // with only the ring's slack to hide it.)
    __device__ void decode(int s, int item, GradItem &it) const
    {
        const GradSide &g = p.side[s];
        unsigned part = 0, tile = static_cast<unsigned>(item);
        it.kb0 = 0;
        it.kb1 = g.k_blocks;
        if (g.split > 1) {  // the parts of a tile run side by side with its neighbours' same part
            part = tile / static_cast<unsigned>(g.tiles);
            tile -= part * static_cast<unsigned>(g.tiles);
            const unsigned kb = static_cast<unsigned>(g.k_blocks), n = static_cast<unsigned>(g.split);
            it.kb0 = static_cast<int>(kb * part / n);  // k_blocks < 2^25, split <= 16
            it.kb1 = static_cast<int>(kb * (part + 1) / n);
        }
        const unsigned per_band = static_cast<unsigned>(g.band * g.n_blocks);
        const unsigned band = tile / per_band;
        const unsigned local = tile - band * per_band;
        const unsigned rows = static_cast<unsigned>(min(g.band, g.m_blocks - static_cast<int>(band) * g.band));
        const unsigned col = local / rows;
        it.side = s;
        it.part = static_cast<int>(part);
        it.mb = static_cast<int>(band) * g.band + static_cast<int>(local - col * rows);
        it.nb = static_cast<int>(col);
    }
};

// Both 64-row halves of this CTA's 128 rows of an MN-major operand.
__device__ __forceinline__ void load_mn(uint32_t dst, const CUtensorMap *m, bool three_d, int row, int k, uint32_t bar)
{
    if (three_d) {
        tma_load_3d_pair(dst, m, 0, k, row / 64, bar);
    } else {
        tma_load_2d_pair(dst, m, row, k, bar);
        tma_load_2d_pair(dst + GR_MN_HALF, m, row + 64, k, bar);
    }
}

// What the producer and the MMA issuer keep across items.
struct RingPos {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void advance()
    {
        if (++stage == G_STAGES) {
            stage = 0;
            phase ^= 1u;
        }
    }
};

// Two K blocks per ring stage: 1381 us for the whole call against 1392 with one.
// After a wait that gave up (`alive` false) the producer and the MMA issuer walk
// through their remaining steps without doing any: loops that never leave early
// keep their indexes, and so the MMA descriptors, warp-uniform (with early exits
// the call took 1525 us).
// One item's copies (one thread of each CTA).  A_MN: side 1, whose A operand is MN-major.
template <bool A_MN>
__device__ __forceinline__ void produce_item(const GemmParams &p, const GradItem &it, const CUtensorMap *tA,
                                             const CUtensorMap *tB, bool a_3d, bool b_3d, RingPos &pos,
                                             uint32_t (&armed)[G_STAGES], bool &alive, bool &skip_next, uint32_t sA, uint32_t sB,
                                             uint32_t bar0, uint32_t rank, volatile int *abort_flag, uint32_t peer_abort)
{
    const int arow = it.mb * G_M + static_cast<int>(rank) * BM;
    const int brow = it.nb * BN + static_cast<int>(rank) * (BN / 2);
    for (int kb = it.kb0; kb < it.kb1; kb += G_KSUB) {
        const int nsub = min(G_KSUB, it.kb1 - kb);
        if (alive)
            alive = wait_bar(bar0 + 8u * (G_STAGES + pos.stage), pos.phase ^ 1u, abort_flag, p, ERR_PRODUCER, peer_abort);
        const uint32_t full = bar0 + 8u * pos.stage;
        const uint32_t full_leader = mapa_shared(full, 0u);
        if (alive && !skip_next) {
            if (rank == 0) {
                mbar_arrive_expect_tx(full, 2u * G_SLOT_BYTES * static_cast<uint32_t>(nsub));
                ++armed[pos.stage];
            }
#pragma unroll
            for (int j = 0; j < G_KSUB; ++j) {
                if (j >= nsub)
                    break;
                const uint32_t slot = static_cast<uint32_t>(pos.stage * G_KSUB + j);
                const int k = (kb + j) * BK;
                if (A_MN)
                    load_mn(sA + slot * G_A_BYTES, tA, a_3d, arow, k, full_leader);
                else
                    tma_load_2d_pair(sA + slot * G_A_BYTES, tA, k, arow, full_leader);
                load_mn(sB + slot * G_B_BYTES, tB, b_3d, brow, k, full_leader);
            }
        }
        skip_next = false;
        pos.advance();
    }
}

// One item's MMAs (the leader's whole MMA warp, converged; `one` set in the thread that issues).
template <bool A_MN>
__device__ __forceinline__ void multiply_item(const GemmParams &p, const GradItem &it, uint32_t d_tmem, RingPos &pos,
                                              bool &alive, uint32_t one, uint32_t sA, uint32_t sB, uint32_t bar0, volatile int *abort_flag,
                                              uint32_t peer_abort)
{
    constexpr uint32_t idesc = idesc_bf16_f32_major(G_M, BN, A_MN, true);
    for (int kb = it.kb0; kb < it.kb1; kb += G_KSUB) {
        const int nsub = min(G_KSUB, it.kb1 - kb);
        if (alive)
            alive = __all_sync(0xffffffffu,
                               wait_bar(bar0 + 8u * pos.stage, pos.phase, abort_flag, p, ERR_MMA_FULL, peer_abort));
        if (alive) {
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < G_KSUB; ++j) {
                if (j >= nsub)
                    break;
                const uint32_t a0 = sA + (pos.stage * G_KSUB + j) * G_A_BYTES;
                const uint32_t b0 = sB + (pos.stage * G_KSUB + j) * G_B_BYTES;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint64_t da =
                        A_MN ? smem_desc_mn128(a0 + k * GR_MN_KSTEP, GR_MN_HALF) : smem_desc_k128(a0 + k * 32);
                    const uint64_t db = smem_desc_mn128(b0 + k * GR_MN_KSTEP, GR_MN_HALF);
                    umma_f16_pair_one(one, d_tmem, da, db, idesc, (kb != it.kb0 || j != 0 || k != 0) ? 1u : 0u);
                }
            }
            umma_commit_pair_mc_one(one, bar0 + 8u * (G_STAGES + pos.stage), 0x3);
        }
        pos.advance();
    }
}

__global__ void __launch_bounds__(G_THREADS, 1)
    k_gated_grads(const __grid_constant__ GradMaps maps, const __grid_constant__ GradsParams gp)
{
    const GemmParams &p = gp.wait;
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
    if (warp == 0 && lane == 0)
        for (int s = 0; s < 2; ++s)
            if (gp.side[s].items) {
                prefetch_tmap(&maps.a[s]);
                prefetch_tmap(&maps.b[s]);
                prefetch_tmap(&maps.o[s]);
            }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), G_TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any cross-CTA signal
    tc_fence_after();
    // everything above touches no global memory and overlaps the kernel before
    wait_previous_kernel();
    let_next_kernel_start();
    const uint32_t tmem_base = *tmem_slot;
    const uint32_t peer_abort = mapa_shared(smem_u32(const_cast<int *>(abort_flag)), rank ^ 1u);

    if (warp == 0) {
        // ------------------------------------------------ TMA producer (both CTAs)
        if (lane == 0) {
            RingPos pos;
            uint32_t armed[G_STAGES];
#pragma unroll
            for (int s = 0; s < G_STAGES; ++s)
                armed[s] = 0;
            bool alive = true, skip_next = p.inject == 1 && blockIdx.x == 0;  // test hook
            GradIter iter(gp, pair, num_pairs);
            for (GradItem it; iter.next(it);) {
                const GradSide &g = gp.side[it.side];
                if (it.side == 0)
                    produce_item<false>(p, it, &maps.a[0], &maps.b[0], false, g.b_3d != 0, pos, armed, alive, skip_next,
                                        sA, sB, bar0, rank, abort_flag, peer_abort);
                else
                    produce_item<true>(p, it, &maps.a[1], &maps.b[1], g.a_3d != 0, g.b_3d != 0, pos, armed, alive,
                                       skip_next, sA, sB, bar0, rank, abort_flag, peer_abort);
            }
            if (leader)
                for (int s = 0; s < G_STAGES; ++s)
                    if (armed[s])
                        wait_bar_drain(FULL_BAR(s), (armed[s] - 1u) & 1u, abort_flag, p, peer_abort);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (leader only)
        if (leader) {
            const uint32_t one = elect_one();
            RingPos pos;
            int acc = 0;
            uint32_t acc_phase = 0;
            GradIter iter(gp, pair, num_pairs);
            bool alive = true;
            for (GradItem it; iter.next(it);) {
                if (alive)
                    alive = __all_sync(0xffffffffu, wait_bar(TEMPTY_BAR(acc), acc_phase ^ 1u, abort_flag, p, ERR_MMA_ACC,
                                                             peer_abort));
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
                if (it.side == 0)
                    multiply_item<false>(p, it, d_tmem, pos, alive, one, sA, sB, bar0, abort_flag, peer_abort);
                else
                    multiply_item<true>(p, it, d_tmem, pos, alive, one, sA, sB, bar0, abort_flag, peer_abort);
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
        // warp w reads TMEM lanes 32 (w % 4) ..; warps 2..5 take the tile's first
        // 128 columns, warps 6..9 the rest
        const int q = warp & 3;
        const int c0 = ((warp - 2) >> 2) * (BN / 2), c1 = c0 + BN / 2;
        int acc = 0;
        uint32_t acc_phase = 0;
        uint8_t *stg = gbase + G_STG_OFF + (warp - 2) * G_STG_WARP;
        const uint32_t stg_s = base + static_cast<uint32_t>(G_STG_OFF + (warp - 2) * G_STG_WARP);
        GradIter iter(gp, pair, num_pairs);
        for (GradItem it; iter.next(it);) {
            const GradSide &g = gp.side[it.side];
            const int row0 = it.mb * G_M + static_cast<int>(rank) * BM + q * 32;
            const uint32_t taddr = tmem_base + static_cast<uint32_t>(acc * BN) + (static_cast<uint32_t>(q * 32) << 16);
            const bool ok = wait_bar(TFULL_BAR(acc), acc_phase, abort_flag, p, ERR_EPI, peer_abort);
            if (!__all_sync(0xffffffffu, ok))
                break;
            tc_fence_after();
            // 64 columns at a time, read before the wait for the staging buffer (the two overlap)
#pragma unroll 1
            for (int c = c0; c < c1; c += 64) {
                const int col = it.nb * BN + c;
                if (col >= g.N)
                    break;  // warp-uniform
                float f[2][32];
                load_acc2(taddr + static_cast<uint32_t>(c), taddr + static_cast<uint32_t>(c + 32), f[0], f[1]);
                stage_begin();
                if (g.split == 1) {
                    stage_half(stg, 0, f[0]);
                    stage_half(stg, 1, f[1]);
                    stage_end(&maps.o[it.side], stg_s, col, row0, g.M);
                    continue;
                }
                // fp32 into the part's matrix (the map's third coordinate), 32 columns a store
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (half)
                        stage_begin();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        stage_piece(stg, j,
                                    make_uint4(__float_as_uint(f[half][4 * j]), __float_as_uint(f[half][4 * j + 1]),
                                               __float_as_uint(f[half][4 * j + 2]), __float_as_uint(f[half][4 * j + 3])));
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && row0 < g.M && col + 32 * half < g.N) {
                        tma_store_3d(&maps.o[it.side], stg_s, col + 32 * half, row0, it.part);
                        bulk_commit_group();
                    }
                }
            }
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

// out = bf16_rn(the sum of the parts, in order), 8 columns per thread and step;
// N % 8 == 0.
__global__ void __launch_bounds__(256)
    k_add_parts(const float *parts0, __nv_bfloat16 *out0, int split0, int64_t n0, const float *parts1,
                __nv_bfloat16 *out1, int split1, int64_t n1)
{
    wait_previous_kernel();
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x * 8;
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * 8; i < n0 + n1; i += step) {
        const bool second = i >= n0;
        const int64_t at = second ? i - n0 : i, n = second ? n1 : n0;
        const float *p = (second ? parts1 : parts0) + at;
        const int split = second ? split1 : split0;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
#pragma unroll 4
        for (int s = 0; s < split; ++s) {
            const float4 u = __ldcg(reinterpret_cast<const float4 *>(p + s * n));
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(p + s * n + 4));
            a = make_float4(a.x + u.x, a.y + u.y, a.z + u.z, a.w + u.w);
            b = make_float4(b.x + v.x, b.y + v.y, b.z + v.z, b.w + v.w);
        }
        *reinterpret_cast<uint4 *>((second ? out1 : out0) + at) =
            make_uint4(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w), pack_bf16(b.x, b.y), pack_bf16(b.z, b.w));
    }
}

// K blocks that an item costs besides its own (the epilogue of a short item is
// not hidden by its MMAs).
constexpr int GR_ITEM_COST = 4;
constexpr int GR_MAX_SPLIT = 16;

}  // namespace

// Sides, splits and schedule.  Where there are more tiles than pairs, a side's K
// blocks are split while an item would be longer than 3/4 of what each of `pairs`
// pairs has to do (and than 8 K blocks): the other side's items fill the rest (1/2
// measured 33.9 us at 1000 x 1024 x 4096 and 122 us at 2048 x 2048 x 5632, 3/4 31.4
// and 110).  Fewer tiles are split into at most one item for each pair (2323 x 144 x
// 1000: 80 items by the first rule 21.2 us, 72 by this one 18.1).  Both products are
// planned, wanted or not, so that one is summed the same way with and without the other.
void plan_gated_grads(GradsParams *p, bool want_dx, bool want_dw, int64_t M, int64_t N, int64_t K, int pairs)
{
    const int64_t rows[2] = {M, N}, kg[2] = {N, M};
    const bool want[2] = {want_dx, want_dw};
    double total = 0;
    for (int s = 0; s < 2; ++s) {
        GradSide &g = p->side[s];
        g = GradSide{};
        g.split = 1;
        g.M = static_cast<int>(rows[s]);
        g.N = static_cast<int>(K);
        g.m_blocks = static_cast<int>((rows[s] + G_M - 1) / G_M);
        g.n_blocks = static_cast<int>((K + BN - 1) / BN);
        g.k_blocks = static_cast<int>((kg[s] + BK - 1) / BK);
        // Bands of M blocks whose A rows stay in L2, and at least eight: 76 tiles at a
        // time read the fewest operand bytes as eight to ten M blocks by as many N
        // blocks (4096 x 5120 x 13824, 14 MB of A rows per block: 1385 us in bands of
        // two, 1345 in eight).
        const double a_bytes = static_cast<double>(G_M) * static_cast<double>(kg[s]) * 2.0;
        const double fit = 32.0 * 1024 * 1024 / a_bytes;
        const int band = fit < 8 ? 8 : fit > g.m_blocks ? g.m_blocks : static_cast<int>(fit);
        const int nbands = (g.m_blocks + band - 1) / band;
        g.band = (g.m_blocks + nbands - 1) / nbands;
        g.tiles = g.m_blocks * g.n_blocks;
        total += static_cast<double>(g.tiles) * (g.k_blocks + GR_ITEM_COST);
    }
    const double share = 0.75 * total / pairs;
    const double most = share < 8 ? 8 : share;
    if (p->side[0].tiles + p->side[1].tiles > pairs) {
        for (int s = 0; s < 2; ++s)
            while (p->side[s].split < GR_MAX_SPLIT && p->side[s].k_blocks > most * p->side[s].split)
                ++p->side[s].split;
    } else {
        // one item for each pair at most: split the side with the longer items while
        // that leaves 8 K blocks to an item and no pair with two
        for (;;) {
            GradSide &a = p->side[0], &b = p->side[1];
            const bool first = static_cast<int64_t>(a.k_blocks) * b.split >= static_cast<int64_t>(b.k_blocks) * a.split;
            GradSide &g = first ? a : b;
            if (g.split >= GR_MAX_SPLIT || g.k_blocks <= 8 * g.split ||
                a.tiles * a.split + b.tiles * b.split + g.tiles > pairs)
                break;
            ++g.split;
        }
    }
    int64_t floats = 0;
    for (int s = 0; s < 2; ++s) {
        GradSide &g = p->side[s];
        g.items = want[s] ? g.tiles * g.split : 0;
        g.parts = floats;
        if (g.split > 1)
            floats += static_cast<int64_t>(g.split) * g.M * g.N;
    }
    p->part_floats = floats;
    const auto cost = [&](int s) {
        return (p->side[s].k_blocks + p->side[s].split - 1) / p->side[s].split + GR_ITEM_COST;
    };
    p->first = !p->side[0].items || (p->side[1].items && cost(1) > cost(0)) ? 1 : 0;
    p->rounds = (cost(p->first) + cost(p->first ^ 1) / 2) / cost(p->first ^ 1);
}

cudaError_t launch_gated_grads(const GradMaps &maps, const GradsParams &p, int pairs, cudaStream_t s)
{
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load() & bit)) {
        e = cudaFuncSetAttribute(k_gated_grads, cudaFuncAttributeMaxDynamicSharedMemorySize, G_SMEM);
        if (e != cudaSuccess)
            return e;
        done.fetch_or(bit);
    }
    const int64_t items = static_cast<int64_t>(p.side[0].items) + p.side[1].items;
    return launch_overlapped(k_gated_grads, dim3(static_cast<unsigned>(2 * (items < pairs ? items : pairs))),
                             dim3(G_THREADS), G_SMEM, 2, s, maps, p);
}

cudaError_t launch_add_parts(const GradsParams &p, const float *parts, void *dx, void *dw, int num_sms, cudaStream_t s)
{
    const GradSide &a = p.side[0], &b = p.side[1];
    const int64_t n0 = a.items && a.split > 1 ? static_cast<int64_t>(a.M) * a.N : 0;
    const int64_t n1 = b.items && b.split > 1 ? static_cast<int64_t>(b.M) * b.N : 0;
    const int64_t blocks = ((n0 + n1) / 8 + 255) / 256, most = static_cast<int64_t>(num_sms) * 8;
    return launch_overlapped(k_add_parts, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(256), 0, 1, s,
                             parts + a.parts, static_cast<__nv_bfloat16 *>(dx), a.split, n0, parts + b.parts,
                             static_cast<__nv_bfloat16 *>(dw), b.split, n1);
}

}  // namespace lf
