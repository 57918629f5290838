// rms_norm.cu -- the residual addition with its root-mean-square norm, the
// 8-bit form of its output, and the gradient of both.
//
// Forward, one row (token) of D channels:
//   h = rn(x + residual)                      the stream, kept in its own type
//   r = 1 / sqrt(mean_d h^2 + eps),  f = h r weight
//   y = rn(f),  or  scale = max_d |f| / 448 (1 if that is 0),  y = e4m3(f / scale)
// (f as (h r) weight: h r is of order one, where r weight may leave fp32's range)
// Backward, with g = dy weight and the same r (recomputed from the h that the
// forward pass kept, so nothing but h has to be saved):
//   dx = r g - h r^3 mean_d(g h) + dh         the gradient of x and of residual
//   dweight = sum over rows of dy h r
//
// Both passes are bound by memory: every element of the row is read once and
// held in registers between the reduction and the output (rows too long for
// that take the *_long kernels, which read the row again from L2).  In replays of a
// captured call one row takes 2.3 us; 8192 x 4096 bf16 44.5 us (6.0 TB/s, 89 % of the
// copy rate), 8192 x 5120 into e4m3 49.6 us, the gradient of 8192 x 4096 47.4 us with
// dweight.
#include "rms_norm_common.cuh"

namespace lf {
namespace {

// One row per block and step; thread t holds the row's packs t, t + threads, ...
// (NV of them at most).
template <class T, class W, int VEC, int NV, bool FP8>
__global__ void __launch_bounds__(NV <= 2 ? 512 : 1024) k_rms_norm(const __grid_constant__ NormParams p)
{
    wait_previous_kernel();
    let_next_kernel_start();
    __shared__ float2 sh[2][MAX_WARPS];
    __shared__ uint32_t wide_sh[MAX_WARPS];
    const int packs = static_cast<int>(p.D / VEC);
    const T *x = static_cast<const T *>(p.x);
    const T *res = static_cast<const T *>(p.residual);
    const W *w = static_cast<const W *>(p.weight);
    int buf = 0;
    bool wide = false;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, buf ^= 1) {
        Pack<T, VEC> h[NV];
        float ss = 0.f;
        float mx = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c < packs)
                h[j] = load_pack<T, VEC>(x + row * p.ldx + static_cast<int64_t>(c) * VEC);
        }
        if (res) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = threadIdx.x + j * blockDim.x;
                if (c < packs) {
                    h[j].add(load_pack<T, VEC>(res + row * p.ldr + static_cast<int64_t>(c) * VEC));
                    h[j].store(static_cast<T *>(p.h) + row * p.D + static_cast<int64_t>(c) * VEC);
                }
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
                if (FP8) {
                    float wv[VEC];
                    load_pack<W, VEC>(w + static_cast<int64_t>(c) * VEC).get(wv);
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        mx = max_mag(mx, v[i] * wv[i]);
                }
            }
        }
        const float2 sums = block_reduce<true>(ss, mag_bits(mx), sh[buf]);
        const float r = rsqrtf(sums.x / static_cast<float>(p.D) + p.eps);
        const RowScale rs(sums.y, sums.x, r);
        if (FP8 && threadIdx.x == 0)
            p.scale[row] = rs.scale;
        wide |= FP8 && rs.wide;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c < packs) {
                const int64_t o = row * p.D + static_cast<int64_t>(c) * VEC;
                float f[VEC], wv[VEC];
                h[j].get(f);
                load_pack<W, VEC>(w + static_cast<int64_t>(c) * VEC).get(wv);
                if (FP8) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        f[i] *= wv[i];
                    rs.apply(f);
                    store_e4m3<VEC>(static_cast<uint8_t *>(p.y) + o, f);
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        f[i] = f[i] * r * wv[i];
                    Pack<T, VEC> yv;
                    yv.set(f);
                    yv.store(static_cast<T *>(p.y) + o);
                }
            }
        }
    }
    if constexpr (FP8)
        if (wide)  // the same for every thread
            wide_rows<T, W>(p, wide_sh, blockDim.x, 1);
}

// Rows that do not fit the registers of a block: the row is read a second time
// (h, which each thread wrote itself, or x where nothing is added).
template <class T, class W, bool FP8>
__global__ void __launch_bounds__(1024) k_rms_norm_long(const __grid_constant__ NormParams p)
{
    wait_previous_kernel();
    let_next_kernel_start();
    __shared__ float2 sh[2][MAX_WARPS];
    __shared__ uint32_t wide_sh[MAX_WARPS];
    const T *res = static_cast<const T *>(p.residual);
    const W *w = static_cast<const W *>(p.weight);
    int buf = 0;
    bool wide = false;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, buf ^= 1) {
        const T *x = static_cast<const T *>(p.x) + row * p.ldx;
        T *h = res ? static_cast<T *>(p.h) + row * p.D : nullptr;
        float ss = 0.f;
        float mx = 0.f;
        for (int64_t c = threadIdx.x; c < p.D; c += blockDim.x) {
            T t = x[c];
            if (res) {
                t = from_f<T>(to_f(t) + to_f(res[row * p.ldr + c]));
                h[c] = t;
            }
            const float v = to_f(t);
            ss = fmaf(v, v, ss);
            if (FP8)
                mx = max_mag(mx, v * to_f(w[c]));
        }
        const float2 sums = block_reduce<true>(ss, mag_bits(mx), sh[buf]);
        const float r = rsqrtf(sums.x / static_cast<float>(p.D) + p.eps);
        const RowScale rs(sums.y, sums.x, r);
        if (FP8 && threadIdx.x == 0)
            p.scale[row] = rs.scale;
        wide |= FP8 && rs.wide;
        for (int64_t c = threadIdx.x; c < p.D; c += blockDim.x) {
            const float v = to_f(res ? h[c] : x[c]);
            if (FP8) {
                float f[1] = {v * to_f(w[c])};
                rs.apply(f);
                store_e4m3<1>(static_cast<uint8_t *>(p.y) + row * p.D + c, f);
            } else {
                static_cast<T *>(p.y)[row * p.D + c] = from_f<T>(v * r * to_f(w[c]));
            }
        }
    }
    if constexpr (FP8)
        if (wide)  // the same for every thread
            wide_rows<T, W>(p, wide_sh, blockDim.x, 1);
}

// Backward: block b takes rows b, b + blocks, ...; thread t keeps the weight
// gradient of its own columns (packs t, t + threads, ...) in fp32 registers
// over all of them and writes it to row b of `partial` at the end; the sum over
// blocks is k_rms_norm_dweight's, in block order: no atomics, one result.
template <class T, class W, int VEC, int NV>
__global__ void __launch_bounds__(VEC * NV <= 8 ? 512 : 1024) k_rms_norm_bwd(const NormBwdParams p)
{
    wait_previous_kernel();
    let_next_kernel_start();
    __shared__ float2 sh[2][MAX_WARPS];
    const int packs = static_cast<int>(p.D / VEC);
    const W *w = static_cast<const W *>(p.weight);
    const float inv_d = 1.f / static_cast<float>(p.D);
    float acc[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            acc[j][i] = 0.f;
    int buf = 0;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, buf ^= 1) {
        const int64_t o = row * p.D;
        Pack<T, VEC> h[NV], dy[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c < packs) {
                h[j] = load_pack<T, VEC>(static_cast<const T *>(p.h) + o + static_cast<int64_t>(c) * VEC);
                dy[j] = load_pack<T, VEC>(static_cast<const T *>(p.dy) + o + static_cast<int64_t>(c) * VEC);
            }
        }
        float ss = 0.f, gh = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c < packs) {
                float v[VEC], d[VEC], wv[VEC];
                h[j].get(v);
                dy[j].get(d);
                load_pack<W, VEC>(w + static_cast<int64_t>(c) * VEC).get(wv);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    ss = fmaf(v[i], v[i], ss);
                    gh = fmaf(d[i] * wv[i], v[i], gh);
                }
            }
        }
        const float2 sums = block_reduce<false>(ss, __float_as_uint(gh), sh[buf]);
        const float r = rsqrtf(sums.x * inv_d + p.eps);
        const float k = (sums.y * inv_d) * r * r;  // dx = r (g - h k) + dh
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c < packs) {
                const int64_t oc = o + static_cast<int64_t>(c) * VEC;
                float v[VEC], d[VEC], wv[VEC], o2[VEC];
                h[j].get(v);
                dy[j].get(d);
                load_pack<W, VEC>(w + static_cast<int64_t>(c) * VEC).get(wv);
                if (p.dh) {
                    load_pack<T, VEC>(static_cast<const T *>(p.dh) + oc).get(o2);
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        o2[i] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    acc[j][i] = fmaf(d[i], v[i] * r, acc[j][i]);
                    o2[i] = fmaf(r, fmaf(d[i], wv[i], -v[i] * k), o2[i]);
                }
                Pack<T, VEC> dx;
                dx.set(o2);
                dx.store(static_cast<T *>(p.dx) + oc);
            }
        }
    }
    if (p.partial) {
        float *out = p.partial + static_cast<int64_t>(blockIdx.x) * p.D;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c < packs) {
                Pack<float, VEC> a;
                a.set(acc[j]);
                a.store(out + static_cast<int64_t>(c) * VEC);
            }
        }
    }
}

// Rows too long for the registers: the row is read twice, and the block's
// weight gradient is kept in its row of `partial` (each thread updates its own
// columns only).
template <class T, class W>
__global__ void __launch_bounds__(1024) k_rms_norm_bwd_long(const NormBwdParams p)
{
    wait_previous_kernel();
    let_next_kernel_start();
    __shared__ float2 sh[2][MAX_WARPS];
    const W *w = static_cast<const W *>(p.weight);
    const float inv_d = 1.f / static_cast<float>(p.D);
    float *part = p.partial ? p.partial + static_cast<int64_t>(blockIdx.x) * p.D : nullptr;
    int buf = 0;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, buf ^= 1) {
        const T *h = static_cast<const T *>(p.h) + row * p.D;
        const T *dy = static_cast<const T *>(p.dy) + row * p.D;
        const T *dh = p.dh ? static_cast<const T *>(p.dh) + row * p.D : nullptr;
        T *dx = static_cast<T *>(p.dx) + row * p.D;
        float ss = 0.f, gh = 0.f;
        for (int64_t c = threadIdx.x; c < p.D; c += blockDim.x) {
            const float v = to_f(h[c]);
            ss = fmaf(v, v, ss);
            gh = fmaf(to_f(dy[c]) * to_f(w[c]), v, gh);
        }
        const float2 sums = block_reduce<false>(ss, __float_as_uint(gh), sh[buf]);
        const float r = rsqrtf(sums.x * inv_d + p.eps);
        const float k = (sums.y * inv_d) * r * r;
        for (int64_t c = threadIdx.x; c < p.D; c += blockDim.x) {
            const float v = to_f(h[c]), d = to_f(dy[c]);
            const float g = r * (d * to_f(w[c]) - v * k);
            if (part)
                part[c] = row == blockIdx.x ? d * (v * r) : fmaf(d, v * r, part[c]);
            dx[c] = from_f<T>(dh ? g + to_f(dh[c]) : g);
        }
    }
}

// dweight[c] = sum over blocks of partial[b][c]: 32 columns per block, 32 rows of
// threads that each sum every 32nd block's row (at most 10, all in flight at
// once); then warp y adds the 32 sums of column y as a tree.
constexpr int DW_ROWS = 32;
constexpr int DW_STEPS = (RMS_BWD_BLOCKS + DW_ROWS - 1) / DW_ROWS;
template <class W>
__global__ void __launch_bounds__(32 * DW_ROWS)
    k_rms_norm_dweight(const float *partial, W *dweight, int64_t D, int blocks)
{
    wait_previous_kernel();
    __shared__ float sh[DW_ROWS][33];
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    float v[DW_STEPS];
#pragma unroll
    for (int i = 0; i < DW_STEPS; ++i) {
        const int b = threadIdx.y + i * DW_ROWS;
        v[i] = c < D && b < blocks ? partial[b * D + c] : 0.f;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < DW_STEPS; ++i)
        s += v[i];
    sh[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    s = sh[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, o);
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.y;
    if (threadIdx.x == 0 && col < D)
        dweight[col] = from_f<W>(s);
}

// Threads of a forward block: the e4m3 form keeps the row's products in fp32 and
// gets 72 registers for it instead of 64.
__host__ __device__ constexpr int ring_threads(bool fp8) { return fp8 ? 896 : 1024; }

template <class T, class W, bool FP8, bool PH>
__global__ void __launch_bounds__(ring_threads(FP8)) k_rms_norm_ring(const __grid_constant__ NormParams p, const RingPlan r)
{
    constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ RingSync sy;
    const int group = threadIdx.x / r.group_threads, t = threadIdx.x % r.group_threads;
    const int warps = r.group_threads >> 5, first_warp = group * warps;
    const RowSpan<T, PH> span(p.M, p.D);
    const int packs = span.packs;
    const T *x = static_cast<const T *>(p.x);
    const T *res = static_cast<const T *>(p.residual);
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
    const W *w = ring_weights<W, PH>(smem, r, static_cast<const W *>(p.weight), span);
    bool ok = true;
    int buf = 0;
    for (int64_t row = row0; row < p.M; row += step, buf ^= 1) {
        ok = ring_wait(ring.full_s + 8u * ring.slot, ring.phase, p.limit);
        // what the second half needs of the row: h, or for e4m3 its products with the weights
        Pack<T, VEC> h[FP8 ? 1 : RING_NV];
        float2 hw[FP8 ? RING_NV : 1][VEC / 2];
        float2 ss2 = both(0.f);
        float mx = 0.f;
#pragma unroll
        for (int j = 0; j < RING_NV; ++j) {
            const int c = t + j * r.group_threads;
            if (c < packs) {
                Pack<T, VEC> v = load_pack<T, VEC>(reinterpret_cast<const T *>(ring.input(0)) + c * VEC);
                if (res) {
                    v.add(load_pack<T, VEC>(reinterpret_cast<const T *>(ring.input(1)) + c * VEC));
                    span.store(static_cast<T *>(p.h), row, c, v);
                }
                span.mask(v, c);
                float2 f[VEC / 2];
                get2<T, VEC>(v, f);
                if (FP8) {
                    float2 wv[VEC / 2];
                    get2<W, VEC>(load_pack<W, VEC>(w + c * VEC), wv);
#pragma unroll
                    for (int i = 0; i < VEC / 2; ++i) {
                        ss2 = fma2(f[i], f[i], ss2);
                        const float2 m = mul2(f[i], wv[i]);
                        hw[FP8 ? j : 0][i] = m;
                        mx = max_mag3(mx, m.x, m.y);
                    }
                } else {
                    h[FP8 ? 0 : j] = v;
#pragma unroll
                    for (int i = 0; i < VEC / 2; ++i)
                        ss2 = fma2(f[i], f[i], ss2);
                }
            }
        }
        const float2 sums = group_reduce<true>(ss2.x + ss2.y, mag_bits(mx), ok, sy, buf, first_warp, warps, 1 + group);
        if (!ok)
            break;
        if (t == 0 && row + r.slots * step < p.M)
            fill(ring.slot, row + r.slots * step);  // every thread of the group has read the slot
        ring.advance();
        const float rr = rsqrtf(sums.x / static_cast<float>(p.D) + p.eps);
        const RowScale rs(sums.y, sums.x, rr);
        if (FP8 && t == 0)
            p.scale[row] = rs.scale;
        if (FP8 && rs.wide)
            sy.wide = 1;
#pragma unroll
        for (int j = 0; j < RING_NV; ++j) {
            const int c = t + j * r.group_threads;
            if (c < packs) {
                if (FP8) {
                    float f[VEC];
#pragma unroll
                    for (int i = 0; i < VEC / 2; ++i) {
                        f[2 * i] = hw[FP8 ? j : 0][i].x;
                        f[2 * i + 1] = hw[FP8 ? j : 0][i].y;
                    }
                    rs.apply(f);
                    span.store_codes(static_cast<uint8_t *>(p.y), row, c, f);
                } else {
                    float2 f[VEC / 2], wv[VEC / 2];
                    get2<T, VEC>(h[FP8 ? 0 : j], f);
                    get2<W, VEC>(load_pack<W, VEC>(w + c * VEC), wv);
#pragma unroll
                    for (int i = 0; i < VEC / 2; ++i)
                        f[i] = mul2(mul2(f[i], both(rr)), wv[i]);
                    Pack<T, VEC> yv;
                    set2<T, VEC>(yv, f);
                    span.store(static_cast<T *>(p.y), row, c, yv);
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
            ring_wide_rows<T, W>(p, sy.wide_max, r.group_threads, r.groups);
    }
}

// Backward: as above with the rows of h, dy (and dh); each thread keeps the
// weight gradient of its columns in registers over its group's rows, the block's
// groups are added in order through shared memory, and the block writes one row
// of `partial`.
template <class T, class W, bool DH, bool PH>
__global__ void __launch_bounds__(512) k_rms_norm_bwd_ring(const NormBwdParams p, const RingPlan r)
{
    constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ RingSync sy;
    const int group = threadIdx.x / r.group_threads, t = threadIdx.x % r.group_threads;
    const int warps = r.group_threads >> 5, first_warp = group * warps;
    const RowSpan<T, PH> span(p.M, p.D);
    const int packs = span.packs;
    const T *hg = static_cast<const T *>(p.h), *yg = static_cast<const T *>(p.dy), *dg = static_cast<const T *>(p.dh);
    const float inv_d = 1.f / static_cast<float>(p.D);
    const int64_t step = static_cast<int64_t>(gridDim.x) * r.groups;
    const int64_t row0 = static_cast<int64_t>(group) * gridDim.x + blockIdx.x;
    Ring ring(r, smem, sy, group);
    const auto fill = [&](int slot, int64_t row) {
        ring.fill(span, slot, row, hg, p.D, yg, p.D, DH ? dg : static_cast<const T *>(nullptr), p.D);
    };
    if (t == 0)
        ring.init();
    wait_previous_kernel();
    let_next_kernel_start();
    if (t == 0) {
        // (test hook: the first block's first group never loads its first row)
        for (int i = p.limit.inject && blockIdx.x == 0 && group == 0 ? 1 : 0; i < r.slots && row0 + i * step < p.M; ++i)
            fill(i, row0 + i * step);
    }
    const W *w = ring_weights<W, PH>(smem, r, static_cast<const W *>(p.weight), span);
    float2 acc[RING_NV][VEC / 2];
#pragma unroll
    for (int j = 0; j < RING_NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i)
            acc[j][i] = both(0.f);
    bool ok = true;
    int buf = 0;
    for (int64_t row = row0; row < p.M; row += step, buf ^= 1) {
        ok = ring_wait(ring.full_s + 8u * ring.slot, ring.phase, p.limit);
        Pack<T, VEC> h[RING_NV], dy[RING_NV], dh[DH ? RING_NV : 1];
        float2 ss = both(0.f), gh = both(0.f);
#pragma unroll
        for (int j = 0; j < RING_NV; ++j) {
            const int c = t + j * r.group_threads;
            if (c < packs) {
                h[j] = load_pack<T, VEC>(reinterpret_cast<const T *>(ring.input(0)) + c * VEC);
                dy[j] = load_pack<T, VEC>(reinterpret_cast<const T *>(ring.input(1)) + c * VEC);
                span.mask(h[j], c);
                span.mask(dy[j], c);
                if (DH)
                    dh[DH ? j : 0] = load_pack<T, VEC>(reinterpret_cast<const T *>(ring.input(2)) + c * VEC);
                float2 v[VEC / 2], d[VEC / 2], wv[VEC / 2];
                get2<T, VEC>(h[j], v);
                get2<T, VEC>(dy[j], d);
                get2<W, VEC>(load_pack<W, VEC>(w + c * VEC), wv);
#pragma unroll
                for (int i = 0; i < VEC / 2; ++i) {
                    ss = fma2(v[i], v[i], ss);
                    gh = fma2(mul2(d[i], wv[i]), v[i], gh);
                }
            }
        }
        const float2 sums = group_reduce<false>(ss.x + ss.y, __float_as_uint(gh.x + gh.y), ok, sy, buf, first_warp, warps,
                                                1 + group);
        if (!ok)
            break;
        if (t == 0 && row + r.slots * step < p.M)
            fill(ring.slot, row + r.slots * step);
        ring.advance();
        const float rr = rsqrtf(sums.x * inv_d + p.eps);
        const float k = (sums.y * inv_d) * rr * rr;  // dx = r (g - h k) + dh
#pragma unroll
        for (int j = 0; j < RING_NV; ++j) {
            const int c = t + j * r.group_threads;
            if (c < packs) {
                float2 v[VEC / 2], d[VEC / 2], wv[VEC / 2], o[VEC / 2];
                get2<T, VEC>(h[j], v);
                get2<T, VEC>(dy[j], d);
                get2<W, VEC>(load_pack<W, VEC>(w + c * VEC), wv);
                if (DH)
                    get2<T, VEC>(dh[DH ? j : 0], o);
#pragma unroll
                for (int i = 0; i < VEC / 2; ++i) {
                    acc[j][i] = fma2(d[i], mul2(v[i], both(rr)), acc[j][i]);
                    const float2 g = fma2(d[i], wv[i], mul2(v[i], both(-k)));
                    o[i] = DH ? fma2(both(rr), g, o[i]) : mul2(both(rr), g);
                }
                Pack<T, VEC> dx;
                set2<T, VEC>(dx, o);
                span.store(static_cast<T *>(p.dx), row, c, dx);
            }
        }
    }
    if (!ok) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < RING_SETTLE_NS) {
        }
    }
    if (!p.partial)
        return;
    // the rings are idle: the first group stores its sums there, the others add
    // theirs in turn, the last one writes the block's row
    __syncthreads();
    float *dw = reinterpret_cast<float *>(smem + r.slot_off);
    for (int g = 0; g < r.groups; ++g) {
        if (group == g) {
#pragma unroll
            for (int j = 0; j < RING_NV; ++j) {
                const int c = t + j * r.group_threads;
                if (c < packs) {
                    Pack<float, VEC> a;
                    set2<float, VEC>(a, acc[j]);
                    if (g > 0)
                        a.add(load_pack<float, VEC>(dw + c * VEC));
                    if (PH || g + 1 < r.groups)
                        a.store(dw + c * VEC);
                    else
                        a.store(p.partial + static_cast<int64_t>(blockIdx.x) * p.D + c * VEC);
                }
            }
        }
        __syncthreads();
    }
    if (PH)
        for (int c = threadIdx.x; c < p.D; c += blockDim.x)
            p.partial[static_cast<int64_t>(blockIdx.x) * p.D + c] = dw[span.phase + c];
}

template <class T, class W, int VEC, bool FP8>
bool launch_norm_regs(const NormParams &p, cudaStream_t s, cudaError_t *e)
{
    const int64_t packs = p.D / VEC;
    const unsigned grid = static_cast<unsigned>(p.M);  // < 2^31
    int t;
    if ((t = threads_for(packs, 1)) && t <= 512)
        *e = launch_overlapped(k_rms_norm<T, W, VEC, 1, FP8>, dim3(grid), dim3(t), 0, 1, s, p);
    else if ((t = threads_for(packs, 2)) && t <= 512)
        *e = launch_overlapped(k_rms_norm<T, W, VEC, 2, FP8>, dim3(grid), dim3(t), 0, 1, s, p);
    else if ((t = threads_for(packs, 4)))
        *e = launch_overlapped(k_rms_norm<T, W, VEC, 4, FP8>, dim3(grid), dim3(t), 0, 1, s, p);
    else if ((t = threads_for(packs, 8)))
        *e = launch_overlapped(k_rms_norm<T, W, VEC, 8, FP8>, dim3(grid), dim3(t), 0, 1, s, p);
    else
        return false;
    return true;
}

template <class T, class W, bool FP8, bool PH>
cudaError_t launch_norm_ring(const NormParams &p, const RingPlan &r, int num_sms, cudaStream_t s)
{
    static std::atomic<unsigned long long> opted{0};
    const cudaError_t e = ring_opt_in(k_rms_norm_ring<T, W, FP8, PH>, opted);
    if (e != cudaSuccess)
        return e;
    return launch_overlapped(k_rms_norm_ring<T, W, FP8, PH>, dim3(ring_blocks(p.M, num_sms)),
                             dim3(r.groups * r.group_threads), r.bytes, 1, s, p, r);
}

template <class T, class W, bool FP8>
cudaError_t launch_norm_t(const NormParams &p, Rows rows, int num_sms, cudaStream_t s)
{
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    RingPlan r;
    if (num_sms >= 8 && use_ring(rows, p.M, p.D) &&
        plan_ring(&r, rows == ROWS_PHASED, p.D, sizeof(T), sizeof(W), p.residual ? 2 : 1, ring_threads(FP8)))
        return rows == ROWS_PHASED ? launch_norm_ring<T, W, FP8, true>(p, r, num_sms, s)
                                   : launch_norm_ring<T, W, FP8, false>(p, r, num_sms, s);
    cudaError_t e = cudaSuccess;
    if (rows == ROWS_VEC ? launch_norm_regs<T, W, V, FP8>(p, s, &e) : launch_norm_regs<T, W, 1, FP8>(p, s, &e))
        return e;
    return launch_overlapped(k_rms_norm_long<T, W, FP8>, dim3(static_cast<unsigned>(p.M)), dim3(1024), 0, 1, s, p);
}

template <class T, class W>
cudaError_t launch_norm_tw(const NormParams &p, Rows rows, bool fp8, int num_sms, cudaStream_t s)
{
    return fp8 ? launch_norm_t<T, W, true>(p, rows, num_sms, s) : launch_norm_t<T, W, false>(p, rows, num_sms, s);
}

template <class T, class W, int VEC>
bool launch_bwd_regs(const NormBwdParams &p, int grid, cudaStream_t s, cudaError_t *e)
{
    constexpr int PER = 16 / VEC;  // at most 16 columns per thread
    const int64_t packs = p.D / VEC;
    int t;
    if constexpr (PER >= 2)
        if ((t = threads_for(packs, PER / 2)) && t <= 512) {
            *e = launch_overlapped(k_rms_norm_bwd<T, W, VEC, PER / 2>, dim3(grid), dim3(t), 0, 1, s, p);
            return true;
        }
    if ((t = threads_for(packs, PER))) {
        *e = launch_overlapped(k_rms_norm_bwd<T, W, VEC, PER>, dim3(grid), dim3(t), 0, 1, s, p);
        return true;
    }
    return false;
}

template <class T, class W, bool DH, bool PH>
cudaError_t launch_bwd_ring(const NormBwdParams &p, const RingPlan &r, int blocks, cudaStream_t s)
{
    static std::atomic<unsigned long long> opted{0};
    const cudaError_t e = ring_opt_in(k_rms_norm_bwd_ring<T, W, DH, PH>, opted);
    if (e != cudaSuccess)
        return e;
    return launch_overlapped(k_rms_norm_bwd_ring<T, W, DH, PH>, dim3(blocks), dim3(r.groups * r.group_threads), r.bytes, 1,
                             s, p, r);
}

template <class T, class W>
cudaError_t launch_bwd_tw(const NormBwdParams &p, Rows rows, void *dweight, int num_sms, cudaStream_t s)
{
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    int blocks = static_cast<int>(p.M < RMS_BWD_BLOCKS ? p.M : RMS_BWD_BLOCKS);
    cudaError_t e = cudaSuccess;
    RingPlan r;
    if (num_sms >= 8 && num_sms <= RMS_BWD_BLOCKS && use_ring(rows, p.M, p.D) &&
        plan_ring(&r, rows == ROWS_PHASED, p.D, sizeof(T), sizeof(W), p.dh ? 3 : 2, 512)) {
        blocks = ring_blocks(p.M, num_sms);
        if (rows == ROWS_PHASED)
            e = p.dh ? launch_bwd_ring<T, W, true, true>(p, r, blocks, s)
                     : launch_bwd_ring<T, W, false, true>(p, r, blocks, s);
        else
            e = p.dh ? launch_bwd_ring<T, W, true, false>(p, r, blocks, s)
                     : launch_bwd_ring<T, W, false, false>(p, r, blocks, s);
    } else {
        if (!(rows == ROWS_VEC ? launch_bwd_regs<T, W, V>(p, blocks, s, &e) : launch_bwd_regs<T, W, 1>(p, blocks, s, &e)))
            e = launch_overlapped(k_rms_norm_bwd_long<T, W>, dim3(blocks), dim3(1024), 0, 1, s, p);
    }
    if (e != cudaSuccess || !dweight)
        return e;
    return launch_overlapped(k_rms_norm_dweight<W>, dim3(static_cast<unsigned>((p.D + 31) / 32)), dim3(32, DW_ROWS), 0, 1,
                             s, static_cast<const float *>(p.partial), static_cast<W *>(dweight), p.D, blocks);
}

}  // namespace

// dtype / wdtype: 0 bf16, 1 fp16, 2 fp32; wdtype is dtype or 2.
cudaError_t launch_rms_norm(const NormParams &p, int dtype, int wdtype, bool fp8, int num_sms, cudaStream_t s)
{
    const int64_t v = dtype == 2 ? 4 : 8;
    const bool based = al16(p.x) && al16(p.y) && al16(p.weight) && (!p.residual || (al16(p.residual) && al16(p.h)));
    const bool packed = p.D % v == 0 && p.ldx % v == 0 && (!p.residual || p.ldr % v == 0);
    const bool contiguous = p.ldx == p.D && (!p.residual || p.ldr == p.D);
    const Rows rows = !based ? ROWS_ANY : packed ? ROWS_VEC : contiguous && p.D >= PHASED_MIN_D ? ROWS_PHASED : ROWS_ANY;
    if (dtype == 0)
        return wdtype == 0 ? launch_norm_tw<__nv_bfloat16, __nv_bfloat16>(p, rows, fp8, num_sms, s)
                           : launch_norm_tw<__nv_bfloat16, float>(p, rows, fp8, num_sms, s);
    if (dtype == 1)
        return wdtype == 1 ? launch_norm_tw<__half, __half>(p, rows, fp8, num_sms, s)
                           : launch_norm_tw<__half, float>(p, rows, fp8, num_sms, s);
    return launch_norm_tw<float, float>(p, rows, fp8, num_sms, s);
}

int rms_norm_bwd_blocks(int64_t M)
{
    return static_cast<int>(M < RMS_BWD_BLOCKS ? (M + 7) / 8 * 8 : RMS_BWD_BLOCKS);  // (304 is a multiple of eight)
}

cudaError_t launch_rms_norm_bwd(const NormBwdParams &p, void *dweight, int dtype, int wdtype, int num_sms,
                                cudaStream_t s)
{
    const int64_t v = dtype == 2 ? 4 : 8;
    const bool based = al16(p.dy) && al16(p.h) && al16(p.weight) && al16(p.dx) && (!p.dh || al16(p.dh)) &&
                       (!p.partial || al16(p.partial));
    const Rows rows = !based ? ROWS_ANY : p.D % v == 0 ? ROWS_VEC : p.D >= PHASED_MIN_D ? ROWS_PHASED : ROWS_ANY;
    if (dtype == 0)
        return wdtype == 0 ? launch_bwd_tw<__nv_bfloat16, __nv_bfloat16>(p, rows, dweight, num_sms, s)
                           : launch_bwd_tw<__nv_bfloat16, float>(p, rows, dweight, num_sms, s);
    if (dtype == 1)
        return wdtype == 1 ? launch_bwd_tw<__half, __half>(p, rows, dweight, num_sms, s)
                           : launch_bwd_tw<__half, float>(p, rows, dweight, num_sms, s);
    return launch_bwd_tw<float, float>(p, rows, dweight, num_sms, s);
}

}  // namespace lf
