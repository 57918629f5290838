// block_norm.cu -- the norm after a block, its gate, the scaled addition to the stream
// and the norm before the next block.  One row (token) of D channels; x is the block's
// output, u its gate row:
//   r1 = 1 / sqrt(mean_d x^2 + eps),  p = (x r1) (post u)    (what there is of them)
//   h  = rn(alpha residual + beta p)                          the stream, kept in its own type
//   r2 = 1 / sqrt(mean_d h^2 + eps),  f = (h r2) pre,  y = rn(f) or e4m3(f / scale)
// Two row reductions, one after the other: h is rounded before its own norm reads it.
// Bound by memory: every element of x and the residual is read once, h and y are written
// once.  Few rows take a block each, with the row in its registers; many rows the rings of
// bulk copies of rms_norm_common.cuh.
#include "block_norm_common.cuh"

namespace lf {
namespace {

// VEC columns of the stream from x, the residual and the columns' factors.
template <class T, int VEC>
__device__ __forceinline__ void enter_stream(const BlockNormParams &p, const Pack<T, VEC> &x, const Pack<T, VEC> &res,
                                             float r1, const float2 (&cf)[PAIRS<VEC>], Pack<T, VEC> &h)
{
    float2 f[PAIRS<VEC>], v[PAIRS<VEC>];
    pairs_of<T, VEC>(x, f);
    pairs_of<T, VEC>(res, v);
#pragma unroll
    for (int i = 0; i < PAIRS<VEC>; ++i)
        f[i] = fma2(v[i], both(p.residual_scale), mul2(mul2(mul2(f[i], both(r1)), cf[i]), both(p.branch_scale)));
    from_pairs<T, VEC>(h, f);
}

// wide_rows' view of the second norm.
__device__ __forceinline__ NormParams second_norm(const BlockNormParams &p)
{
    NormParams n;
    n.x = p.h;
    n.residual = nullptr;
    n.weight = p.pre;
    n.h = nullptr;
    n.y = p.y;
    n.scale = p.scale;
    n.M = p.M;
    n.D = p.D;
    n.ldx = p.D;
    n.ldr = 0;
    n.eps = p.eps;
    n.limit = p.limit;
    return n;
}

// One row per block; thread t holds the row's packs t, t + threads, ...  Latency bounds it: two
// reductions, one after the other (one token of 5120 2.8 us, 100 x 4096 2.5, both in L2; 600 x
// 5120 6.6 of 3.6).  Without a loop over rows it needs ten registers fewer (600 x 5120 9.5 us with
// one); the loads stand in a loop of their own, before the sums (one token 3.04 us, so 2.91).
template <class T, class W, int VEC, int NV, bool FP8>
__global__ void __launch_bounds__(NV <= 2 ? 512 : 1024) k_block_norm(const __grid_constant__ BlockNormParams p)
{
    wait_previous_kernel();
    let_next_kernel_start();
    __shared__ float2 sh[2][MAX_WARPS];
    __shared__ uint32_t wide_sh[MAX_WARPS];
    const int packs = static_cast<int>(p.D / VEC);
    const T *x = static_cast<const T *>(p.x), *res = static_cast<const T *>(p.residual);
    const W *pre = static_cast<const W *>(p.pre);
    const int64_t row = blockIdx.x;
    Pack<T, VEC> h[NV], rs[NV];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = threadIdx.x + j * blockDim.x;
        if (c < packs) {
            h[j] = load_pack<T, VEC>(x + row * p.ldx + static_cast<int64_t>(c) * VEC);
            rs[j] = load_pack<T, VEC>(res + row * p.ldr + static_cast<int64_t>(c) * VEC);
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = threadIdx.x + j * blockDim.x;
        if (c < packs) {
            float v[VEC];
            h[j].get(v);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                ss = fmaf(v[i], v[i], ss);
        }
    }
    float r1 = 1.f;
    if (p.post)
        r1 = rsqrtf(block_reduce<false>(ss, 0u, sh[0]).x / static_cast<float>(p.D) + p.eps);
    const int64_t gate_row = p.gate ? row / p.gate_tokens * p.D : 0;
    ss = 0.f;
    float mx = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = threadIdx.x + j * blockDim.x;
        if (c < packs) {
            const int64_t at = static_cast<int64_t>(c) * VEC;
            float2 cf[PAIRS<VEC>];
            float v[VEC];
            column_factors<T, W, VEC>(p, gate_row, at, cf);
            enter_stream<T, VEC>(p, h[j], rs[j], r1, cf, h[j]);
            h[j].store(static_cast<T *>(p.h) + row * p.D + at);
            h[j].get(v);
            if (FP8) {
                float w[VEC];
                load_pack<W, VEC>(pre + at).get(w);
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    mx = max_mag(mx, v[i] * w[i]);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                ss = fmaf(v[i], v[i], ss);
        }
    }
    if (!pre)
        return;
    const float2 sums = block_reduce<true>(ss, mag_bits(mx), sh[1]);
    const float r2 = rsqrtf(sums.x / static_cast<float>(p.D) + p.eps);
    const RowScale scale(sums.y, sums.x, r2);
    if (FP8 && threadIdx.x == 0)
        p.scale[row] = scale.scale;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = threadIdx.x + j * blockDim.x;
        if (c < packs) {
            const int64_t at = static_cast<int64_t>(c) * VEC;
            float f[VEC], w[VEC];
            h[j].get(f);
            load_pack<W, VEC>(pre + at).get(w);
            if (FP8) {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    f[i] *= w[i];
                scale.apply(f);
                store_e4m3<VEC>(static_cast<uint8_t *>(p.y) + row * p.D + at, f);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    f[i] = f[i] * r2 * w[i];
                Pack<T, VEC> y;
                y.set(f);
                y.store(static_cast<T *>(p.y) + row * p.D + at);
            }
        }
    }
    if constexpr (FP8)
        if (scale.wide)  // the same for every thread
            wide_rows<T, W>(second_norm(p), wide_sh, blockDim.x, 1);
}

// Rows that do not fit the registers of a block: x is read twice, and h, which each
// thread wrote itself, once more (element by element, 16 x 40000 fp32 18.4 us, 4 x 70000 bf16 30.2;
// with blockDim.x for the step of the loops 20.3 and 31.2).
constexpr int LONG_THREADS = 1024;
template <class T, class W, bool FP8>
__global__ void __launch_bounds__(LONG_THREADS) k_block_norm_long(const __grid_constant__ BlockNormParams p)
{
    wait_previous_kernel();
    let_next_kernel_start();
    __shared__ float2 sh[2][MAX_WARPS];
    __shared__ uint32_t wide_sh[MAX_WARPS];
    const W *pre = static_cast<const W *>(p.pre);
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.ldx, *res = static_cast<const T *>(p.residual) + row * p.ldr;
    T *h = static_cast<T *>(p.h) + row * p.D;
    const int64_t gate_row = p.gate ? row / p.gate_tokens * p.D : 0;
    float r1 = 1.f, ss = 0.f, mx = 0.f;
    if (p.post) {
#pragma unroll 4
        for (int64_t c = threadIdx.x; c < p.D; c += LONG_THREADS)
            ss = fmaf(to_f(x[c]), to_f(x[c]), ss);
        r1 = rsqrtf(block_reduce<false>(ss, 0u, sh[0]).x / static_cast<float>(p.D) + p.eps);
    }
    ss = 0.f;
#pragma unroll 4
    for (int64_t c = threadIdx.x; c < p.D; c += LONG_THREADS) {
        Pack<T, 1> k;
        float2 cf[1];
        column_factors<T, W, 1>(p, gate_row, c, cf);
        enter_stream<T, 1>(p, load_pack<T, 1>(x + c), load_pack<T, 1>(res + c), r1, cf, k);
        h[c] = k.v;
        const float v = to_f(k.v);
        ss = fmaf(v, v, ss);
        if (FP8)
            mx = max_mag(mx, v * to_f(pre[c]));
    }
    if (!pre)
        return;
    const float2 sums = block_reduce<true>(ss, mag_bits(mx), sh[1]);
    const float r2 = rsqrtf(sums.x / static_cast<float>(p.D) + p.eps);
    const RowScale scale(sums.y, sums.x, r2);
    if (FP8 && threadIdx.x == 0)
        p.scale[row] = scale.scale;
    for (int64_t c = threadIdx.x; c < p.D; c += LONG_THREADS) {
        const float v = to_f(h[c]);
        if (FP8) {
            float f[1] = {v * to_f(pre[c])};
            scale.apply(f);
            store_e4m3<1>(static_cast<uint8_t *>(p.y) + row * p.D + c, f);
        } else {
            static_cast<T *>(p.y)[row * p.D + c] = from_f<T>(v * r2 * to_f(pre[c]));
        }
    }
    if constexpr (FP8)
        if (scale.wide)  // the same for every thread
            wide_rows<T, W>(second_norm(p), wide_sh, LONG_THREADS, 1);
}

// ---------------------------------------------------------------- many rows
// Where a ring kernel has the parameters.
enum Params { PARAMS_GLOBAL, PARAMS_SHARED, PARAMS_SHARED_GATES };
__host__ __device__ constexpr int block_norm_threads(bool fp8, bool phased) { return fp8 || phased ? 640 : 512; }

// In rings of bulk copies (rms_norm_common.cuh).  The parameters lie in shared memory where
// they fit: beta post (times a gate of one row) in fp32, then pre, in fp32 too (in its own
// type for e4m3, which reads it twice, and for phased rows, which leave less room), so that a
// pack takes few conversions and one product for them.  A gate of several rows is read where
// it is, before the wait for the row if it is of the stream's type.  Between its two
// reductions a row is kept in fp32, in its type where the gate or the codes need the
// registers.
// 8192 x 5120 bf16 takes 58 to 60 us (335 MB: 5.7 TB/s, 84 % of the copy rate), with no gate,
// one or four; without pre 44.7; with 640 threads, and so spills, 82.  Into e4m3, at 640
// threads, 52.2, with four gates 59.5.  8188 x 4097 55.4, at 512 threads 63.
template <class T, class W, bool FP8, bool PH, Params PARAMS>
__global__ void __launch_bounds__(block_norm_threads(FP8, PH))
    k_block_norm_ring(const __grid_constant__ BlockNormParams p, const RingPlan r)
{
    constexpr int VEC = 16 / static_cast<int>(sizeof(T)), N = VEC / 2;
    constexpr bool SHARED = PARAMS != PARAMS_GLOBAL, EARLY_GATE = PARAMS == PARAMS_SHARED_GATES;
    constexpr bool KEEP_F32 = !FP8 && !EARLY_GATE && !PH;
    using Pre = typename std::conditional<FP8 || PH, W, float>::type;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ RingSync sy;
    __shared__ __align__(16) float scales[8];  // beta
    const int group = threadIdx.x / r.group_threads, t = threadIdx.x % r.group_threads;
    const int warps = r.group_threads >> 5, first_warp = group * warps;
    const RowSpan<T, PH> span(p.M, p.D);
    const int packs = span.packs;
    const T *x = static_cast<const T *>(p.x), *res = static_cast<const T *>(p.residual);
    const int64_t step = static_cast<int64_t>(gridDim.x) * r.groups;
    // neighbouring rows go to neighbouring SMs
    const int64_t row0 = static_cast<int64_t>(group) * gridDim.x + blockIdx.x;
    Ring ring(r, smem, sy, group);
    const auto fill = [&](int slot, int64_t row) {
        ring.fill(span, slot, row, x, p.ldx, res, p.ldr, static_cast<const T *>(nullptr), 0);
    };
    if (t == 0)
        ring.init();
    if (FP8 && threadIdx.x == 0)
        sy.wide = 0;
    wait_previous_kernel();
    let_next_kernel_start();
    if (t == 0) {
        // (test hook: the first block's first group never loads its first row)
        for (int i = p.limit.inject && blockIdx.x == 0 && group == 0 ? 1 : 0; i < r.slots && row0 + i * step < p.M; ++i)
            fill(i, row0 + i * step);
    }
    const bool one_gate = p.gate && p.gate_tokens == p.M, gates = p.gate && !one_gate, factors = p.post || one_gate;
    const W *const post = static_cast<const W *>(p.post), *const pre = static_cast<const W *>(p.pre);
    if (threadIdx.x < 8)
        scales[threadIdx.x] = p.branch_scale;
    float *const s_factor = reinterpret_cast<float *>(smem + r.w_off);
    Pre *const s_pre = reinterpret_cast<Pre *>(s_factor + (factors ? packs * VEC : 0));
    if (SHARED) {
#pragma unroll 4
        for (int i = threadIdx.x; i < packs * VEC; i += blockDim.x) {
            const int k = i - span.phase;
            const bool inside = !PH || (k >= 0 && k < span.D);
            if (factors) {
                float f = inside && post ? to_f(post[k]) : 1.f;
                if (inside && one_gate)
                    f *= gate_one<T>(p.gate, p.gate_f32, k);
                s_factor[i] = inside ? f * p.branch_scale : 0.f;
            }
            if (pre)
                s_pre[i] = from_f<Pre>(inside ? to_f(pre[k]) : 0.f);
        }
    }
    __syncthreads();
    const uint32_t factor = factors ? smem_u32(s_factor) : smem_u32(scales), factor_apart = factors ? 4u * VEC : 0u;
    const uint32_t pre_at = smem_u32(s_pre);
    const auto second_weights = [&](int c, float2 (&w)[N]) {
        if constexpr (SHARED)
            get2<Pre, VEC>(lds_pack<Pre, VEC>(pre_at + c * static_cast<uint32_t>(VEC * sizeof(Pre))), w);
        else
            get2<W, VEC>(load_pack<W, VEC>(pre + c * VEC), w);
    };
    bool ok = true;
    for (int64_t row = row0; row < p.M; row += step) {
        // every thread of the group has read the slot: it takes the row `slots` steps ahead
        const auto refill = [&] {
            if (t == 0 && row + r.slots * step < p.M)
                fill(ring.slot, row + r.slots * step);
            ring.advance();
        };
        const int64_t gate_row = gates ? row / p.gate_tokens * p.D : 0;
        Pack<T, VEC> u[RING_NV];
        if (EARLY_GATE) {
#pragma unroll
            for (int j = 0; j < RING_NV; ++j) {
                const int c = t + j * r.group_threads;
                if (c < packs)
                    u[j] = load_pack<T, VEC>(static_cast<const T *>(p.gate) + gate_row + c * VEC);
            }
        }
        // post times the gate times beta
        const auto first_weights = [&](int j, int c, float2 (&w)[N]) {
            if constexpr (!SHARED) {
                column_factors<T, W, VEC>(p, gate_row, c * VEC, w);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    w[i] = mul2(w[i], both(p.branch_scale));
                return;
            }
            get2<float, VEC>(lds_pack<float, VEC>(factor + c * factor_apart), w);
            if (!gates)
                return;
            float2 g[N];
            if constexpr (PH) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float v = span.inside(c, i) ? gate_one<T>(p.gate, p.gate_f32, gate_row + c * VEC + i - span.phase) : 0.f;
                    (i % 2 ? g[i / 2].y : g[i / 2].x) = v;
                }
            } else if (!EARLY_GATE) {
                gate_at<T, VEC>(p.gate, p.gate_f32, gate_row + c * VEC, g);
            } else {
                get2<T, VEC>(u[j], g);
            }
#pragma unroll
            for (int i = 0; i < N; ++i)
                w[i] = mul2(w[i], g[i]);
        };
        ok = ring_wait(ring.full_s + 8u * ring.slot, ring.phase, p.limit);
        const uint32_t in = ring.slots_s + ring.slot * ring.slot_bytes;
        Pack<T, VEC> xs[RING_NV], rs[RING_NV];
        float2 ss = both(0.f);
#pragma unroll
        for (int j = 0; j < RING_NV; ++j) {
            const int c = t + j * r.group_threads;
            if (c < packs) {
                xs[j] = lds_pack<T, VEC>(in + c * 16u);
                rs[j] = lds_pack<T, VEC>(in + ring.row_bytes + c * 16u);
                if (PH) {
                    const uint4 keep = span.words(c);
                    xs[j].keep(keep);
                    rs[j].keep(keep);
                }
                float2 f[N];
                get2<T, VEC>(xs[j], f);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    ss = fma2(f[i], f[i], ss);
            }
        }
        float r1 = 1.f;
        if (!p.post && p.pre) {
            group_barrier(1 + group, r.group_threads);
            if (ok)
                refill();
        } else {
            const float2 sums = group_reduce<false>(ss.x + ss.y, 0u, ok, sy, 0, first_warp, warps, 1 + group);
            if (!ok)
                break;
            refill();
            if (p.post)
                r1 = rsqrtf(sums.x / static_cast<float>(p.D) + p.eps);
        }
        float2 h[KEEP_F32 ? RING_NV : 1][N];  // the stream as it is kept, in fp32 (else in xs)
        ss = both(0.f);
        float mx = 0.f;
#pragma unroll
        for (int j = 0; j < RING_NV; ++j) {
            const int c = t + j * r.group_threads;
            if (c < packs) {
                float2 w[N], f[N], v[N];
                first_weights(j, c, w);
                get2<T, VEC>(xs[j], f);
                get2<T, VEC>(rs[j], v);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    f[i] = mul2(mul2(f[i], both(r1)), w[i]);
                    f[i] = make_float2(fmaf(v[i].x, p.residual_scale, f[i].x), fmaf(v[i].y, p.residual_scale, f[i].y));
                }
                Pack<T, VEC> kept;
                set2<T, VEC>(kept, f);
                span.store(static_cast<T *>(p.h), row, c, kept);
                float2 (&k)[N] = h[KEEP_F32 ? j : 0];
                get2<T, VEC>(kept, k);
                if (!KEEP_F32)
                    xs[j] = kept;
                if (FP8) {
                    second_weights(c, w);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const float2 m = mul2(k[i], w[i]);
                        mx = max_mag3(mx, m.x, m.y);
                    }
                }
#pragma unroll
                for (int i = 0; i < N; ++i)
                    ss = fma2(k[i], k[i], ss);
            }
        }
        if (!p.pre) {
            group_barrier(1 + group, r.group_threads);  // sy.sums[0] is written again
            continue;
        }
        const float2 sums = group_reduce<true>(ss.x + ss.y, mag_bits(mx), ok, sy, 1, first_warp, warps, 1 + group);
        if (!ok)
            break;
        const float r2 = rsqrtf(sums.x / static_cast<float>(p.D) + p.eps);
        const RowScale scale(sums.y, sums.x, r2);
        if (FP8 && t == 0)
            p.scale[row] = scale.scale;
        if (FP8 && scale.wide)
            sy.wide = 1;
#pragma unroll
        for (int j = 0; j < RING_NV; ++j) {
            const int c = t + j * r.group_threads;
            if (c < packs) {
                float2 w[N];
                second_weights(c, w);
                float2 (&k)[N] = h[KEEP_F32 ? j : 0];
                if (!KEEP_F32)
                    get2<T, VEC>(xs[j], k);
                if (FP8) {
                    float q[VEC];
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const float2 m = mul2(k[i], w[i]);
                        q[2 * i] = m.x;
                        q[2 * i + 1] = m.y;
                    }
                    scale.apply(q);
                    span.store_codes(static_cast<uint8_t *>(p.y), row, c, q);
                } else {
                    float2 f[N];
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        f[i] = mul2(mul2(k[i], both(r2)), w[i]);
                    Pack<T, VEC> y;
                    set2<T, VEC>(y, f);
                    span.store(static_cast<T *>(p.y), row, c, y);
                }
            }
        }
    }
    if (!ok) {  // copies of this group may still be in flight: give them time to land
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < RING_SETTLE_NS) {
        }
    }
    if constexpr (FP8) {
        __syncthreads();
        if (ok && sy.wide)
            ring_wide_rows<T, W>(second_norm(p), sy.wide_max, r.group_threads, r.groups);
    }
}

// ---------------------------------------------------------------- launches
template <class T, class W, int VEC, bool FP8>
bool launch_block_regs(const BlockNormParams &p, cudaStream_t s, cudaError_t *e)
{
    const int64_t packs = p.D / VEC;
    const dim3 grid(static_cast<unsigned>(p.M));  // < 2^31
    int t;
    if ((t = threads_for(packs, 1)) && t <= 512)
        *e = launch_overlapped(k_block_norm<T, W, VEC, 1, FP8>, grid, dim3(t), 0, 1, s, p);
    else if ((t = threads_for(packs, 2)) && t <= 512)
        *e = launch_overlapped(k_block_norm<T, W, VEC, 2, FP8>, grid, dim3(t), 0, 1, s, p);
    else if ((t = threads_for(packs, 4)))
        *e = launch_overlapped(k_block_norm<T, W, VEC, 4, FP8>, grid, dim3(t), 0, 1, s, p);
    else
        return false;
    return true;
}

template <class T, class W, bool FP8, bool PH, Params PARAMS>
cudaError_t launch_block_ring(const BlockNormParams &p, const RingPlan &r, int num_sms, cudaStream_t s)
{
    static std::atomic<unsigned long long> opted{0};
    const cudaError_t e = ring_opt_in(k_block_norm_ring<T, W, FP8, PH, PARAMS>, opted);
    if (e != cudaSuccess)
        return e;
    return launch_overlapped(k_block_norm_ring<T, W, FP8, PH, PARAMS>, dim3(ring_blocks(p.M, num_sms)),
                             dim3(r.groups * r.group_threads), r.bytes, 1, s, p, r);
}

template <class T, class W, bool FP8>
cudaError_t launch_block_t(const BlockNormParams &p, Rows rows, int num_sms, cudaStream_t s)
{
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    RingPlan r;
    const bool one_gate = p.gate && p.gate_tokens == p.M;
    const int param_bytes = (p.pre ? static_cast<int>(FP8 || rows == ROWS_PHASED ? sizeof(W) : sizeof(float)) : 0) + (p.post || one_gate ? 4 : 0);
    if (num_sms >= 8 && use_ring(rows, p.M, p.D) &&
        plan_ring(&r, rows == ROWS_PHASED, p.D, sizeof(T), param_bytes, 2, block_norm_threads(FP8, rows == ROWS_PHASED)))
        return rows == ROWS_PHASED ? launch_block_ring<T, W, FP8, true, PARAMS_SHARED>(p, r, num_sms, s)
               : !r.w_shared       ? launch_block_ring<T, W, FP8, false, PARAMS_GLOBAL>(p, r, num_sms, s)
               : p.gate && !one_gate && (!p.gate_f32 || sizeof(T) == sizeof(float))
                   ? launch_block_ring<T, W, FP8, false, PARAMS_SHARED_GATES>(p, r, num_sms, s)
                   : launch_block_ring<T, W, FP8, false, PARAMS_SHARED>(p, r, num_sms, s);
    cudaError_t e = cudaSuccess;
    if (rows == ROWS_VEC ? launch_block_regs<T, W, V, FP8>(p, s, &e) : launch_block_regs<T, W, 1, FP8>(p, s, &e))
        return e;
    return launch_overlapped(k_block_norm_long<T, W, FP8>, dim3(static_cast<unsigned>(p.M)), dim3(LONG_THREADS), 0, 1,
                            s, p);
}

template <class T, class W>
cudaError_t launch_block_tw(const BlockNormParams &p, Rows rows, bool fp8, int num_sms, cudaStream_t s)
{
    return fp8 ? launch_block_t<T, W, true>(p, rows, num_sms, s) : launch_block_t<T, W, false>(p, rows, num_sms, s);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormParams &p, int dtype, int wdtype, bool fp8, int num_sms, cudaStream_t s)
{
    const int64_t v = dtype == 2 ? 4 : 8;
    const bool based = al16(p.x) && al16(p.residual) && al16(p.h) && al16(p.y) && al16(p.post) && al16(p.pre) && al16(p.gate);
    const bool packed = p.D % v == 0 && p.ldx % v == 0 && p.ldr % v == 0;
    const bool contiguous = p.ldx == p.D && p.ldr == p.D;
    const Rows rows = !based ? ROWS_ANY : packed ? ROWS_VEC : contiguous && p.D >= PHASED_MIN_D ? ROWS_PHASED : ROWS_ANY;
    if (dtype == 0)
        return wdtype == 0 ? launch_block_tw<__nv_bfloat16, __nv_bfloat16>(p, rows, fp8, num_sms, s)
                           : launch_block_tw<__nv_bfloat16, float>(p, rows, fp8, num_sms, s);
    if (dtype == 1)
        return wdtype == 1 ? launch_block_tw<__half, __half>(p, rows, fp8, num_sms, s)
                           : launch_block_tw<__half, float>(p, rows, fp8, num_sms, s);
    return launch_block_tw<float, float>(p, rows, fp8, num_sms, s);
}

}  // namespace lf
