// gated_common.cuh -- what the CTA-pair kernels of the gated projections and of
// their gradient share: the tile and ring constants, and the store of a finished
// 32 x 32 chunk.  Roles, barriers and bounded waits are those of gemm_nt_pair.cu.
#pragma once
#include "lf_gemm_common.cuh"

namespace lf {
namespace {

constexpr int G_M = 2 * BM;                // 256 rows of x per pair tile
constexpr int G_F = BN / 2;                // 128 output columns per pair tile
// The ring: G_SLOTS slots of one K block (128 bytes of K), G_KSUB consecutive
// slots per stage -- one wait, one commit and one barrier arm per two K blocks.
constexpr int G_SLOTS = 6;
constexpr int G_KSUB = 2;
constexpr int G_STAGES = G_SLOTS / G_KSUB;
constexpr int G_ROW = 128;                 // bytes of K per row and block
constexpr int G_A_BYTES = BM * G_ROW;      // this CTA's 128 rows of x
constexpr int G_B_BYTES = G_F * G_ROW;     // this CTA's 128 rows of w (gate in the leader, up in its peer)
constexpr int G_SLOT_BYTES = G_A_BYTES + G_B_BYTES;
constexpr int G_ACC_BUFS = 2;
constexpr int G_TMEM_COLS = G_ACC_BUFS * BN;
constexpr int G_NUM_BARS = 2 * G_STAGES + 2 * G_ACC_BUFS + 1;
constexpr int G_EPI_WARPS = 8;
constexpr int G_THREADS = 64 + 32 * G_EPI_WARPS;
constexpr int G_STG_SLOT = 32 * 64;        // 32 rows x 32 bf16 columns
constexpr int G_STG_WARP = 2 * G_STG_SLOT;
constexpr int G_STG_OFF = ((G_SLOTS * G_SLOT_BYTES + G_NUM_BARS * 8 + 16 + 1023) / 1024) * 1024;
constexpr int G_SMEM = 1024 + G_STG_OFF + G_EPI_WARPS * G_STG_WARP;
static_assert(G_SMEM <= 232448, "shared memory per CTA");
constexpr uint64_t G_ABORT_SETTLE_NS = 100000;

// One 32 x 32 chunk of output (this thread's row as 16 packed pairs) through
// staging slot k & 1 and a TMA store, as tma_store_chunk of gemm_nt_pair.cu.
__device__ __forceinline__ void g_store_chunk(const CUtensorMap *tm, uint8_t *stg, uint32_t stg_s, int k,
                                              const uint32_t (&pk)[16], int col, int row0, int M)
{
    const int lane = threadIdx.x & 31;
    const int slot = k & 1;
    if (k >= 2) {
        if (lane == 0)
            bulk_wait_group_read<1>();
        __syncwarp();
    }
    uint8_t *buf = stg + slot * G_STG_SLOT;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4 *>(buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
            make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && row0 < M) {
        tma_store_2d(tm, stg_s + static_cast<uint32_t>(slot * G_STG_SLOT), col, row0);
        bulk_commit_group();
    }
}

}  // namespace
}  // namespace lf
