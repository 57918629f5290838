// lf_internal.h -- declarations shared by the translation units of
// liblayoutfold.so (not part of the public C ABI).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#ifdef LF_NVTX
#include <nvtx3/nvToolsExt.h>
#endif

#include "lf_kernel_params.h"

namespace lf {

// Launchers (host).  Return cudaSuccess or the launch error.
cudaError_t launch_gemm_nt(int epi, const CUtensorMap &ta, const CUtensorMap &tb, const GemmParams &p,
                           int grid, cudaStream_t s);
int gemm_smem_bytes();

// CTA-pair variant (cta_group::2, 256x256 tiles; p.num_m_blocks counts
// 256-row blocks; grid even).  layout bit 0: X stored [K,M] (tensor map over
// [K rows, M columns], 64x64 boxes), else [M,K] (64-column x 128-row boxes);
// bit 1: W stored [K,N] likewise, else [N,K]; bit 2: batched (3-D tensor
// maps, batch outermost; p.batch, p.w_batched, p.ldo, p.stride_o).  Layouts
// 1..3 take the EPI_STORE and cross-entropy epilogues, batched layouts
// EPI_STORE only.  `to`: the output as a
// bf16 tensor map (2-D [M rows, N columns], row pitch p.ldo; 3-D with the
// batch outermost when batched), 32 x 32 boxes, 64-byte swizzle -- read only
// when p.tma_store is set.
cudaError_t launch_gemm_nt_pair(int epi, int layout, const CUtensorMap &ta, const CUtensorMap &tb,
                                const CUtensorMap &to, const GemmParams &p, int grid, cudaStream_t s);
int gemm_pair_smem_bytes();
int gemm_pair_max_active_clusters();

// One-pass GEMM + cross-entropy + gradient on CTA pairs (no recompute GEMM,
// no combine kernel).  Requires op_k * op_Q co-resident pairs; grid = 2 * op_k * op_Q.
// `to`: the gradient (p.out) as a 2-D bf16 map, 32 x 32 boxes, 64-byte swizzle.
// layout bit 0: X stored [K,M] (ta as for the pair kernel: 64 x 64 boxes); bit
// 1: W stored [K,N] (tb with 64 x 64 boxes; op_tile 128 or 256), else tb's box
// is op_tile / 2 rows of W [N,K].
cudaError_t launch_xent_onepass(int layout, const CUtensorMap &ta, const CUtensorMap &tb, const CUtensorMap &to,
                                const GemmParams &p, int grid, cudaStream_t s);

cudaError_t launch_xent_combine(const float *part_max, const float *part_sum, const float *label_logit,
                                const int32_t *labels, int M, int N, int num_n_blocks, float *loss,
                                float *row_max, float *row_logsum, cudaStream_t s);

// Second pass of the cross-entropy gradient after EPI_XENT_EXP: per row, the
// combine (lse from the tile partials, loss), then grad rewritten in place
// from the fp16 e = exp(z - tile max) it holds: grad = bf16_rn(e * exp(tile
// max - lse)), the label column from the fp32 label logit.
cudaError_t launch_xent_rescale(const float *part_max, const float *part_sum, const float *label_logit,
                                const int32_t *labels, int M, int N, int num_n_blocks, float *loss, void *grad,
                                cudaStream_t s);

cudaError_t launch_matmul_k1_f32(const float *a, const float *b, float *out, int64_t M, int64_t N,
                                 int num_sms, cudaStream_t s);
cudaError_t launch_matmul_k1_bf16(const void *x, const void *w, void *out, int64_t M, int64_t N,
                                  int num_sms, cudaStream_t s);
cudaError_t launch_rope_cos_sin(const void *inv_freq, const int64_t *pos, void *cos_out, void *sin_out, int64_t H,
                                int64_t S, int num_sms, cudaStream_t s);
cudaError_t launch_fp8_cast_dual(const void *x, const float *scale, void *out, void *out_t, int64_t M, int64_t K,
                                 int num_sms, cudaStream_t s);
// Launch with programmatic stream serialisation (and clusters of `cluster` CTAs):
// the kernel may be set up while its predecessor in the stream ends, so it has to
// call wait_previous_kernel (lf_ptx_ffn.cuh) before it touches global memory.
template <class... P, class... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t s,
                              A &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<A &&>(args)...);
}

// Where a kernel's bounded waits report, and their limit.
struct WaitLimit {
    int *err;
    unsigned long long timeout_ns;
    int inject;  // test hook: 1 = the first wait is never satisfied
};

// Residual addition + RMS norm (rms_norm.cu).  dtype / wdtype as lf_dtype;
// wdtype is dtype or fp32.  ldx, ldr: row pitches in elements; h and y are [M,D].
struct NormParams {
    const void *x, *residual, *weight;  // residual may be null: then h is x and is not written
    void *h, *y;
    float *scale;  // [M], the e4m3 form only
    int64_t M, D, ldx, ldr;
    float eps;
    WaitLimit limit;
};
cudaError_t launch_rms_norm(const NormParams &p, int dtype, int wdtype, bool fp8, int num_sms, cudaStream_t s);

// Its gradient.  partial: fp32 [rms_norm_bwd_blocks(M)][D] at most, or null with
// dweight null; dweight has the weight's type.  dh may be null.
struct NormBwdParams {
    const void *dy, *h, *weight, *dh;
    void *dx;
    float *partial;
    int64_t M, D;
    float eps;
    WaitLimit limit;
};
constexpr int RMS_BWD_BLOCKS = 304;  // two blocks for each of 152 SMs
int rms_norm_bwd_blocks(int64_t M);
cudaError_t launch_rms_norm_bwd(const NormBwdParams &p, void *dweight, int dtype, int wdtype, int num_sms,
                                cudaStream_t s);

// The norms after and before a block with its gate and scales (block_norm.cu).  dtype /
// wdtype as above; post, pre and gate may be null.  gate: [M / gate_tokens, D] of dtype or
// (gate_f32) fp32; gate_tokens is M without a gate.  ldx, ldr: row pitches in elements; h
// and y are [M,D].
struct BlockNormParams {
    const void *x, *residual, *post, *pre, *gate;
    void *h, *y;   // y null without pre
    float *scale;  // [M], the e4m3 form only
    int64_t M, D, ldx, ldr, gate_tokens;
    float eps, branch_scale, residual_scale;
    int gate_f32;
    WaitLimit limit;
};
cudaError_t launch_block_norm(const BlockNormParams &p, int dtype, int wdtype, bool fp8, int num_sms, cudaStream_t s);

// Its gradient (block_norm_grads.cu).  dy and h are read with pre, x with post or a gate (null otherwise), dh may
// be null with pre.  part_pre, part_sum and counters: the three parts of the scratch, in
// this order; part_pre is null with dpre, part_sum with dpost and dgate, and counters with
// dpost.  dpost and dpre have wdtype, dgate the gate's type.
struct BlockNormBwdParams {
    const void *dy, *x, *h, *post, *pre, *gate, *dh;
    void *dx, *dres;
    float *part_pre, *part_sum;
    unsigned *counters;
    int64_t M, D, gate_tokens, gate_rows;  // gate_rows: M / gate_tokens, or 0 without a gate
    int64_t lanes, residues;               // set by launch_block_norm_bwd
    float eps, branch_scale, residual_scale;
    int gate_f32;
    WaitLimit limit;
};
constexpr int BLOCK_NORM_BWD_BLOCKS = 152;  // of the ring kernel at most
struct BlockNormScratch {
    int64_t pre_floats, sum_floats, counters;  // (words of four bytes, the first two multiples of four)
};
BlockNormScratch block_norm_bwd_scratch(int64_t M, int64_t D, int dtype, int64_t gate_rows);
cudaError_t launch_block_norm_bwd(const BlockNormBwdParams &p, void *dpost, void *dpre, void *dgate, int dtype, int wdtype,
                                  int num_sms, cudaStream_t s);

// Gated projections on CTA pairs (gated_ffn.cu): out = act(x Wg^T) * (x Wu^T).
// g: M, N = F, K, block counts (256-row M blocks, N blocks of cols, 128-byte
// K blocks), num_tiles, band_m, err, timeout_ns, inject.
struct GatedParams {
    GemmParams g;
    const float *x_scale, *w_scale;  // e4m3 operands: [M] and [2F]
    int save;                        // also store gate and up (tg, tu)
    int cols;                        // output columns of a pair tile (plan_gated_cols)
};
// ta: x, boxes of 128 rows; tw: w [2F, K], boxes of cols rows (both 128-byte
// rows, 128-byte swizzle); to: out; tg, tu: the two halves of gu (64 x 32
// boxes, 128-byte swizzle).
cudaError_t launch_gated_pair(bool e4m3, int act, const CUtensorMap &ta, const CUtensorMap &tw, const CUtensorMap &to,
                              const CUtensorMap &tg, const CUtensorMap &tu, const GatedParams &p, int grid,
                              cudaStream_t s);
// The output columns of a pair tile for m_blocks blocks of 256 tokens on `pairs` CTA pairs.
int plan_gated_cols(int m_blocks, int64_t F, int pairs);
// The same for few tokens (operands swapped, the K loop split over clusters).
struct GatedSkinny {
    bool preferred;  // to the pair kernel

    int tokens;  // of one CTA (at most 128)
    int n;       // the MMA's N: tokens rounded up to 16
    int split;   // CTAs per cluster, each with its share of the K blocks: 1, 2, 4 or 8
    int stages;  // ring stages
    int smem;    // dynamic shared memory per CTA
};
// How a call with M tokens would run (in groups of at most 128); num_k_blocks counts 128-byte K blocks.
GatedSkinny plan_gated_skinny(int64_t M, int64_t F, int num_k_blocks, int num_sms);
// ta: x, boxes of plan.n rows; tw: boxes of 128 rows.  gu may be null.
cudaError_t launch_gated_skinny(bool e4m3, int act, const CUtensorMap &ta, const CUtensorMap &tw, const GatedParams &p,
                                const GatedSkinny &plan, void *gu, cudaStream_t s);
// dgu = [dout u act'(g), dout act(g)] from gu = [g, u]; F % 8 == 0, 16-byte
// aligned.
cudaError_t launch_gated_bwd(int act, const void *dout, const void *gu, void *dgu, int64_t M, int64_t F,
                             cudaStream_t s);

// The products of the gradient (gated_grads.cu).  Side 0: dx[M, K] = dgu . w;
// side 1: dw[N, K] = dgu^T . x, dgu [M, N] (N = 2F for the gated projections).
struct GradSide {
    int M, N;                                    // the output's rows and columns
    int m_blocks, n_blocks, k_blocks, band;      // 256-row, 256-column and 64-wide K blocks; M blocks per band
    int tiles, split, items;                     // K parts per tile; items = tiles * split (0: not wanted)
    int64_t parts;                               // where its parts start, in floats: [split][M][N] (split > 1)
    int a_3d, b_3d;                              // the MN-major operands' maps are 3-D views
};
struct GradsParams {
    GemmParams wait;  // err, timeout_ns, inject
    GradSide side[2];
    int first, rounds;    // the schedule (GradIter)
    int64_t part_floats;  // of all parts
};
// o: the output (bf16, 64 x 32 boxes, 128-byte swizzle) or, where the side is split, its parts
// (fp32, 3-D: N, M, split; 32 x 32 x 1 boxes, 128-byte swizzle).
struct GradMaps {
    CUtensorMap a[2], b[2], o[2];
};
// Pairs that the splits (and so the scratch) are planned for, whatever the device has.
constexpr int GRAD_PLAN_PAIRS = 76;
void plan_gated_grads(GradsParams *p, bool want_dx, bool want_dw, int64_t M, int64_t N, int64_t K, int pairs);
cudaError_t launch_gated_grads(const GradMaps &maps, const GradsParams &p, int pairs, cudaStream_t s);
// The wanted split sides' parts added up.
cudaError_t launch_add_parts(const GradsParams &p, const float *parts, void *dx, void *dw, int num_sms, cudaStream_t s);

// A projection with bias, activation and residual in its epilogue, on CTA pairs
// (linear.cu): out = act(x w^T + bias) + residual.  g: M, N, K, block counts (256-row M
// blocks, N blocks of cols, 128-byte K blocks), num_tiles, band_m, err, timeout_ns, inject.
struct LinearParams {
    GemmParams g;
    const float *x_scale, *w_scale;  // e4m3 operands: [M] and [N]
    const void *bias;                // [N] or null
    int bias_f32;                    // it is fp32 (else bf16)
    int residual, save;              // add the residual (map residual), store z (map pre)
    int cols, split;                 // columns of a tile, pairs that share its K blocks (plan_linear_pair)
};
// x: boxes of 128 rows; w: boxes of cols / 2 rows (both 128-byte rows, 128-byte
// swizzle); out, pre, residual: bf16 [M, N], 64 x 32 boxes, 128-byte swizzle.
struct LinearMaps {
    CUtensorMap x, w, out, pre, residual;
};
cudaError_t launch_linear_pair(bool e4m3, int act, const LinearMaps &m, const LinearParams &p, int grid, cudaStream_t s);
void plan_linear_pair(int m_blocks, int64_t N, int num_k_blocks, int pairs, int *cols, int *split);
// The same for few tokens (operands swapped, the K loop split over clusters).
struct LinearSkinny {
    bool preferred;  // to the pair kernel
    int tokens;      // of one CTA (at most 128)
    int n;           // the MMA's N: tokens rounded up to 16
    int split;       // CTAs per cluster, each with its share of the K blocks: 1 to 8
    int stages;      // ring stages
    int smem;        // dynamic shared memory per CTA
};
// How a call with M tokens would run (in groups of at most 128); num_k_blocks counts 128-byte K blocks.
LinearSkinny plan_linear_skinny(int64_t M, int64_t N, int num_k_blocks, int num_sms);
// m.x: boxes of plan.n rows; m.w: boxes of 128 rows; the other maps are not read.
// p.g.num_n_blocks counts blocks of 128 columns.  residual and pre: [M, N] or null.
cudaError_t launch_linear_skinny(bool e4m3, int act, const LinearMaps &m, const LinearParams &p,
                                 const LinearSkinny &plan, const void *residual, void *pre, cudaStream_t s);
// dz = dout act'(pre) (not written without an activation) and its column sums: to
// dbias, or to `partial` (fp32 [linear_dz_blocks][N]) where that is more than one row (of blocks that no cluster holds),
// and from there by launch_linear_dbias.  dbias may be null.  N % 8 == 0, 16-byte aligned.
int linear_dz_blocks(int64_t M, int64_t N);
cudaError_t launch_linear_dz(int act, const void *dout, const void *pre, void *dz, float *partial, void *dbias,
                             bool bias_f32, int64_t M, int64_t N, cudaStream_t s);
cudaError_t launch_linear_dbias(const float *partial, void *dbias, bool bias_f32, int64_t M, int64_t N, cudaStream_t s);

// Test hook: `ctas` CTAs, each holding 200 KiB of shared memory (one per SM),
// that wait `ns` nanoseconds on the global timer and exit.
cudaError_t launch_occupy_sms(int ctas, unsigned long long ns, cudaStream_t s);

// A profiling range around one entry-point call: an NVTX range named after
// the call when the library is built with LF_NVTX defined, nothing otherwise.
struct CallRange {
    explicit CallRange(const char *name)
    {
#ifdef LF_NVTX
        nvtxRangePushA(name);
#else
        (void)name;
#endif
    }
    ~CallRange()
    {
#ifdef LF_NVTX
        nvtxRangePop();
#endif
    }
    CallRange(const CallRange &) = delete;
    CallRange &operator=(const CallRange &) = delete;
};

// Library state and helpers shared by the entry points of every translation
// unit (defined in api.cu).
unsigned long long wait_timeout_ns();  // device-side wait limit (lf_set_test_hooks; 2 s by default)
bool cooperative_launches();           // false after lf_set_cooperative(0)
int stall_injection();                 // 1 while lf_set_test_hooks asks for a stalled first stage
void count_launches(int n);            // adds n to the lf_launch_count total
bool debug_sync_enabled();             // LF_DEBUG_SYNC is set in the environment
// 2-D bf16 tensor [rows, K] (K contiguous) as a TMA map: boxes of 64 columns x
// box_rows rows, 128-byte swizzle, zero fill out of bounds.  False if the
// driver entry point is missing or rejects the layout.
bool make_tmap_kmajor(CUtensorMap *m, const void *ptr, int64_t rows, int64_t K, uint32_t box_rows);

}  // namespace lf
