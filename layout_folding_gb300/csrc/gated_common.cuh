// gated_common.cuh -- what the CTA-pair kernels of the gated projections and of
// their gradient share: the tile and ring constants, and the store of a finished
// tile by boxes of 32 rows x 128 bytes (64 bf16 or 32 fp32 columns).  Roles, barriers and bounded waits are those of gemm_nt_pair.cu.
#pragma once
#include "lf_gemm_common.cuh"
#include "lf_ptx_ffn.cuh"

namespace lf {
namespace {

constexpr int G_M = 2 * BM;                // 256 rows of x per pair tile
constexpr int G_F = BN / 2;                // output columns per pair tile: at most 128,
constexpr int G_MIN_F = 64;                // and at least what half the epilogue's warps store
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
constexpr int G_STG_WARP = 32 * 128;       // a warp's staging: 32 rows x 64 bf16 (or 32 fp32) columns
constexpr int G_STG_OFF = ((G_SLOTS * G_SLOT_BYTES + G_NUM_BARS * 8 + 16 + 1023) / 1024) * 1024;
constexpr int G_SMEM = 1024 + G_STG_OFF + G_EPI_WARPS * G_STG_WARP;
static_assert(G_SMEM <= 232448, "shared memory per CTA");
constexpr uint64_t G_ABORT_SETTLE_NS = 100000;

// Stores of a finished tile go through a warp's staging buffer, 32 rows of 128
// bytes whose 16-byte pieces are XOR-swizzled by row (the 128-byte swizzle of the
// output's tensor map), and leave as one box.  (64-byte rows -- 32 bf16 columns a
// store -- made the tensor-copy unit the bottleneck of tiles with short K loops.)
//
// Before the buffer is written again: the store issued from it has read it.
__device__ __forceinline__ void stage_begin()
{
    if ((threadIdx.x & 31) == 0)
        bulk_wait_group_read<0>();
    __syncwarp();
}
// 16-byte piece j (0..7) of this thread's row.
__device__ __forceinline__ void stage_piece(uint8_t *stg, int j, uint4 v)
{
    const int lane = threadIdx.x & 31;
    *reinterpret_cast<uint4 *>(stg + lane * 128 + ((j ^ (lane & 7)) << 4)) = v;
}
// 32 values of this thread's row as bf16: half 0 or 1 of its 64 columns.
__device__ __forceinline__ void stage_half(uint8_t *stg, int half, const float (&f)[32])
{
#pragma unroll
    for (int j = 0; j < 4; ++j)
        stage_piece(stg, 4 * half + j,
                    make_uint4(pack_bf16(f[8 * j], f[8 * j + 1]), pack_bf16(f[8 * j + 2], f[8 * j + 3]),
                               pack_bf16(f[8 * j + 4], f[8 * j + 5]), pack_bf16(f[8 * j + 6], f[8 * j + 7])));
}
// The buffer is full: lane 0 stores it at (col, row0); rows and columns outside
// the map are left out.
__device__ __forceinline__ void stage_end(const CUtensorMap *tm, uint32_t stg_s, int col, int row0, int M)
{
    fence_proxy_async_smem();
    __syncwarp();
    if ((threadIdx.x & 31) == 0 && row0 < M) {
        tma_store_2d(tm, stg_s, col, row0);
        bulk_commit_group();
    }
}

// Two runs of 32 accumulator columns of this thread's row.
__device__ __forceinline__ void load_acc2(uint32_t t0, uint32_t t1, float (&f)[32], float (&g)[32])
{
    uint32_t v[32], w[32];
    tmem_ld_32x32b_x32(t0, v);
    tmem_ld_32x32b_x32(t1, w);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        f[i] = __uint_as_float(v[i]);
        g[i] = __uint_as_float(w[i]);
    }
}

}  // namespace
}  // namespace lf
