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
#include <atomic>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math_constants.h>
#include <type_traits>

#include "lf_internal.h"
#include "lf_ptx_ffn.cuh"

namespace lf {
namespace {

constexpr float E4M3_MAX = 448.f;
constexpr int MAX_WARPS = 32;

// VEC consecutive elements as they lie in memory: 32-bit words moved 16 bytes at
// a time, or (VEC = 1) one element with no alignment beyond its own.  get() and
// set() convert to and from fp32 a pair at a time.
template <class T, int VEC>
struct Pack {
    static constexpr int WORDS = VEC * static_cast<int>(sizeof(T)) / 4;
    uint32_t u[WORDS];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i) {
            const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
            u[4 * i] = v.x;
            u[4 * i + 1] = v.y;
            u[4 * i + 2] = v.z;
            u[4 * i + 3] = v.w;
        }
    }
    __device__ __forceinline__ void store(T *p) const
    {
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i)
            reinterpret_cast<uint4 *>(p)[i] = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
    }
    __device__ __forceinline__ void get(float (&f)[VEC]) const
    {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            if constexpr (sizeof(T) == 4) {
                f[i] = __uint_as_float(u[i]);
            } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                f[2 * i] = __uint_as_float(u[i] << 16);
                f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            } else {
                const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
                f[2 * i] = v.x;
                f[2 * i + 1] = v.y;
            }
        }
    }
    __device__ __forceinline__ void set(const float (&f)[VEC])
    {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            if constexpr (sizeof(T) == 4) {
                u[i] = __float_as_uint(f[i]);
            } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t *>(&v);
            } else {
                const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t *>(&v);
            }
        }
    }
    // this += o, each sum rounded once to T.  (For the 16-bit types that is also
    // what an fp32 addition rounded to T gives: fp32 has more than twice their
    // digits, so its own rounding cannot move a sum across one of theirs.)
    __device__ __forceinline__ void add(const Pack &o)
    {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            if constexpr (sizeof(T) == 4) {
                u[i] = __float_as_uint(__uint_as_float(u[i]) + __uint_as_float(o.u[i]));
            } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                const __nv_bfloat162 v = __hadd2_rn(*reinterpret_cast<const __nv_bfloat162 *>(&u[i]),
                                                    *reinterpret_cast<const __nv_bfloat162 *>(&o.u[i]));
                u[i] = *reinterpret_cast<const uint32_t *>(&v);
            } else {
                const __half2 v = __hadd2_rn(*reinterpret_cast<const __half2 *>(&u[i]),
                                             *reinterpret_cast<const __half2 *>(&o.u[i]));
                u[i] = *reinterpret_cast<const uint32_t *>(&v);
            }
        }
    }
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f(float v)
{
    if constexpr (std::is_same<T, float>::value)
        return v;
    else if constexpr (std::is_same<T, __half>::value)
        return __float2half_rn(v);
    else
        return __float2bfloat16_rn(v);
}

template <class T>
struct Pack<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ void store(T *p) const { *p = v; }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = to_f(v); }
    __device__ __forceinline__ void set(const float (&f)[1]) { v = from_f<T>(f[0]); }
    __device__ __forceinline__ void add(const Pack &o) { v = from_f<T>(to_f(v) + to_f(o.v)); }
};

template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T *p)
{
    Pack<T, VEC> r;
    r.load(p);
    return r;
}

// max(|a|, |b|, |c|), a NaN kept
__device__ __forceinline__ float max_mag3(float a, float b, float c)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// The values of a pack, two at a time.
template <class T, int VEC>
__device__ __forceinline__ void get2(const Pack<T, VEC> &p, float2 (&f)[VEC / 2])
{
    float v[VEC];
    p.get(v);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i)
        f[i] = make_float2(v[2 * i], v[2 * i + 1]);
}
template <class T, int VEC>
__device__ __forceinline__ void set2(Pack<T, VEC> &p, const float2 (&f)[VEC / 2])
{
    float v[VEC];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
        v[2 * i] = f[i].x;
        v[2 * i + 1] = f[i].y;
    }
    p.set(v);
}

// max(|m|, |a|), a NaN kept: the running maximum of magnitudes (its sign is not
// meaningful until mag() clears it).
__device__ __forceinline__ float max_mag(float m, float a)
{
    float r;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(a));
    return r;
}
// |v| as an unsigned integer: ordered like the magnitudes, infinity above
// every number and a NaN above infinity, so an integer maximum keeps a NaN.
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Sum of `a` (and of `b`, or the maximum of the magnitude bits in `b`) over the
// block; every thread gets both.  `sh` holds one pair per warp; callers that
// reduce row after row alternate between two such buffers, so one barrier per
// row is enough (a warp can be at most one barrier ahead).
template <bool MAXB>
__device__ __forceinline__ float2 block_reduce(float a, uint32_t b, float2 *sh)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        const uint32_t c = __shfl_xor_sync(0xffffffffu, b, o);
        b = MAXB ? max(b, c) : __float_as_uint(__uint_as_float(b) + __uint_as_float(c));
    }
    const int warps = blockDim.x >> 5;
    if (warps == 1)
        return make_float2(a, __uint_as_float(b));
    if ((threadIdx.x & 31) == 0)
        sh[threadIdx.x >> 5] = make_float2(a, __uint_as_float(b));
    __syncthreads();
    a = 0.f;
    b = 0u;
    const int lane = threadIdx.x & 31;
    if (lane < warps) {
        const float2 t = sh[lane];
        a = t.x;
        b = __float_as_uint(t.y);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        const uint32_t c = __shfl_xor_sync(0xffffffffu, b, o);
        b = MAXB ? max(b, c) : __float_as_uint(__uint_as_float(b) + __uint_as_float(c));
    }
    return make_float2(a, __uint_as_float(b));
}

// The e4m3 scale of a row and the factor that takes h weight to its code: f is
// h weight r, and its largest magnitude r times mx = max |h weight|, so
// f / scale = h weight (448 / mx).  A scale that would be 0 is 1; NaN stays NaN.
// `wide`: a product h weight overflowed, or they are so small that they lose bits or
// 448 / mx could overflow, although (h r) weight may be an ordinary number: its scale
// is left as -r for wide_rows, which does the row again.  Rows of zeros stay here: h or
// the weights are 0, h so small that its squares are, or products below 2^-150 with
// r <= 2^8, whose f / 448 is 0 as well.
struct RowScale {
    float scale, factor;
    bool wide;
    __device__ __forceinline__ RowScale(float mx, float ss, float r)
    {
        const float q = mx * r / E4M3_MAX;
        const bool zeros = mx == 0.f && (ss == 0.f || r <= 256.f);
        wide = !zeros && (mx < 0x1p-100f || q < 0x1p-120f || mx == CUDART_INF_F);
        scale = wide ? -r : q == 0.f ? 1.f : q;
        factor = q == 0.f ? r : q != q ? q : E4M3_MAX / mx;
    }
    // f: h weight, N of them, to what is converted to e4m3
    template <int N>
    __device__ __forceinline__ void apply(float (&f)[N]) const
    {
        if constexpr (N % 2 == 0) {
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const float2 v = mul2(make_float2(f[i], f[i + 1]), both(factor));
                f[i] = v.x;
                f[i + 1] = v.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                f[i] *= factor;
        }
    }
};

__device__ __forceinline__ uint32_t e4m3_pair(float a, float b)
{
    return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}

template <int VEC>
__device__ __forceinline__ void store_e4m3(uint8_t *p, const float (&f)[VEC])
{
    if constexpr (VEC == 8) {
        uint2 q;
        q.x = e4m3_pair(f[0], f[1]) | (e4m3_pair(f[2], f[3]) << 16);
        q.y = e4m3_pair(f[4], f[5]) | (e4m3_pair(f[6], f[7]) << 16);
        *reinterpret_cast<uint2 *>(p) = q;
    } else if constexpr (VEC == 4) {
        *reinterpret_cast<uint32_t *>(p) = e4m3_pair(f[0], f[1]) | (e4m3_pair(f[2], f[3]) << 16);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            p[i] = static_cast<uint8_t>(e4m3_pair(f[i], 0.f) & 0xffu);
    }
}

__device__ __forceinline__ void group_barrier(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// This thread's group's rows (group g of the block's `groups` of group_threads each:
// rows g gridDim + blockIdx, and so on in steps of all groups) whose scale says wide:
// f = (h r) weight and f / scale, element by element from their h in memory.  `sh`
// holds one word per warp of the block.  Done after a kernel's own rows, with nothing
// kept for it but that there is one: inside their loop it makes the ring kernel keep some
// fifty bytes of a thread's registers in local memory.
template <class T, class W>
__device__ __forceinline__ void wide_rows(const NormParams &p, uint32_t *sh, int group_threads, int groups)
{
    const int group = threadIdx.x / group_threads, t = threadIdx.x % group_threads;
    const int warps = group_threads >> 5, first_warp = group * warps, lane = t & 31;
    const T *h = static_cast<const T *>(p.residual ? p.h : p.x);
    const int64_t ld = p.residual ? p.D : p.ldx, D = p.D;
    const W *w = static_cast<const W *>(p.weight);
    const auto sync = [&] {
        if (warps > 1)
            group_barrier(1 + group, group_threads);
        else
            __syncwarp();
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
#pragma unroll 1
    for (int64_t row = static_cast<int64_t>(group) * gridDim.x + blockIdx.x; row < p.M; row += step) {
        sync();  // the row's h, codes and scale are written, the last row's words read
        const float mark = p.scale[row];
        if (static_cast<int>(__float_as_uint(mark)) >= 0 || mark != mark)
            continue;
        const float r = -mark;
        const T *hr = h + row * ld;
        float m = 0.f;
#pragma unroll 1
        for (int64_t c = t; c < D; c += group_threads)
            m = max_mag(m, to_f(hr[c]) * r * to_f(w[c]));
        uint32_t b = __reduce_max_sync(0xffffffffu, mag_bits(m));
        if (lane == 0)
            sh[first_warp + (t >> 5)] = b;
        sync();
        b = __reduce_max_sync(0xffffffffu, lane < warps ? sh[first_warp + lane] : 0u);
        const float q = __uint_as_float(b) / E4M3_MAX, s = q == 0.f ? 1.f : q;
        if (t == 0)
            p.scale[row] = s;
#pragma unroll 1
        for (int64_t c = t; c < D; c += group_threads)
            static_cast<uint8_t *>(p.y)[row * D + c] =
                static_cast<uint8_t>(e4m3_pair(to_f(hr[c]) * r * to_f(w[c]) / s, 0.f) & 0xffu);
    }
}

// The same for the ring kernel, out of the way of its code (8192 x 5120 49.4 us, in line
// 50.4; the kernels of one block per row need eight registers more for a call).
template <class T, class W>
__device__ __noinline__ void ring_wide_rows(const NormParams &p, uint32_t *sh, int group_threads, int groups)
{
    wide_rows<T, W>(p, sh, group_threads, groups);
}

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

// ---------------------------------------------------------------- many rows
// With many rows the kernels are bound by HBM, which wants some 70 KB in flight
// on every SM at all times.  So one persistent block per SM splits into groups of
// warps, each with its own ring of row slots in shared memory that bulk copies
// (cp.async.bulk, one per input row) fill: group g of the grid takes rows g,
// g + groups, ...  A group moves a landed row into registers, reduces it over its
// own warps -- a named barrier, after which every thread has read the slot, so
// one thread refills it with the row `slots` steps ahead -- and writes its
// outputs while the copies run.  Registers hold one row only; the latency is
// covered by the rings.
//
// Rows whose length is not a multiple of 16 bytes (PH, "phased") are moved in
// 16-byte granules all the same: contiguous rows lie one after another, so the
// granules that cover row r start `phase` = r D mod VEC elements before it.  The
// grid is a multiple of VEC, so every row of a block has the phase of its first,
// and a thread's columns, the shifted weights in shared memory and the places
// of the row's two ragged granules stay the same for the whole block.
constexpr int RING_NV = 4;            // packs per thread: a group has ceil(packs / 128) warps
constexpr int RING_MAX_GROUPS = 15;   // named barriers 1..15
constexpr int RING_MAX_SLOTS = 8;
// Fewer rows than four per SM: one block per row.  Around the border both take about
// the same (us by blocks / in rings: 608 x 5120 bf16 4.7 / 5.0, into e4m3 5.1 / 5.0, 608 x
// 1024 into e4m3 2.4 / 2.8, 1000 x 5120 bf16 7.4 / 7.4); 8192 x 5120 into e4m3 takes 54.4 /
// 49.7.  Phased rows, which blocks move element by element, always where they are long,
// and from 100 rows on (32 x 5121 4.5 / 3.5, 300 x 5121 13.4 / 5.2; a ring's setup shows with
// short rows, 100 x 517 1.9 / 3.7).
constexpr int64_t RING_MIN_ROWS = 608, RING_MIN_ROWS_PHASED = 100, RING_LONG_D = 1024;
constexpr int RING_BUDGET = 225 * 1024;  // dynamic shared memory; RingSync takes 2 KB more
constexpr uint64_t RING_SETTLE_NS = 100000;  // after an abort: let copies in flight land

// Shared-memory layout of a ring kernel, computed on the host.
struct RingPlan {
    int group_threads, groups, slots;
    uint32_t row_bytes;                // one input row
    int w_shared;                          // weights copied to shared memory (else read where they are)
    uint32_t w_off, slot_off, slot_bytes;  // weights; slots ([group][slot][input][row])
    uint32_t bytes;                    // dynamic shared memory
};

struct RingSync {
    float2 sums[2][MAX_WARPS];
    int failed[2][MAX_WARPS];
    int wide;                      // the block had a row for wide_rows
    uint32_t wide_max[MAX_WARPS];  // (its sh)
    alignas(8) unsigned long long full[RING_MAX_GROUPS * RING_MAX_SLOTS];
};

// Bounded wait for a slot; on a timeout the code goes to the device error word.
__device__ __forceinline__ bool ring_wait(uint32_t bar, uint32_t parity, const WaitLimit &lim)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (global_timer_ns() - t0 > lim.timeout_ns) {
            atomicCAS(lim.err, 0, 0x102);
            return false;
        }
    }
    return true;
}

// block_reduce over one group.  `ok` (false in a thread whose wait gave up) is
// combined as well, so that the whole group leaves its loop together.
template <bool MAXB>
__device__ __forceinline__ float2 group_reduce(float a, uint32_t b, bool &ok, RingSync &sy, int buf, int first_warp,
                                               int warps, int id)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        const uint32_t c = __shfl_xor_sync(0xffffffffu, b, o);
        b = MAXB ? max(b, c) : __float_as_uint(__uint_as_float(b) + __uint_as_float(c));
    }
    ok = __all_sync(0xffffffffu, ok);
    if (warps == 1) {
        __syncwarp();  // orders the warp's reads of the slot before its refill
        return make_float2(a, __uint_as_float(b));
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) {
        sy.sums[buf][warp] = make_float2(a, __uint_as_float(b));
        sy.failed[buf][warp] = ok ? 0 : 1;
    }
    group_barrier(id, warps * 32);
    a = 0.f;
    b = 0u;
    int failed = 0;
    if (lane < warps) {
        const float2 t = sy.sums[buf][first_warp + lane];
        a = t.x;
        b = __float_as_uint(t.y);
        failed = sy.failed[buf][first_warp + lane];
    }
    ok = !__any_sync(0xffffffffu, failed);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        const uint32_t c = __shfl_xor_sync(0xffffffffu, b, o);
        b = MAXB ? max(b, c) : __float_as_uint(__uint_as_float(b) + __uint_as_float(c));
    }
    return make_float2(a, __uint_as_float(b));
}

// Where a block's rows lie in their granules.
template <class T, bool PH>
struct RowSpan {
    static constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    int phase, packs;
    const int64_t &M, &D;  // the kernel's parameters, which need no registers
    __device__ RowSpan(const int64_t &m, const int64_t &d)
        : phase(PH ? static_cast<int>((blockIdx.x % VEC) * (d % VEC) % VEC) : 0),
          packs(static_cast<int>((phase + d + VEC - 1) / VEC)), M(m), D(d)
    {
    }
    __device__ bool ragged(int c) const { return PH && (c == 0 || c == packs - 1); }
    __device__ bool inside(int c, int i) const
    {
        const int k = c * VEC + i - phase;
        return k >= 0 && k < D;
    }
    // Element 0 of the row's first granule, relative to the row's base address.
    __device__ int64_t first(int64_t row) const { return row * D - phase; }
    // Zero the granule's elements that belong to other rows.
    __device__ void mask(Pack<T, VEC> &v, int c) const
    {
        if (ragged(c)) {
            float f[VEC];
            v.get(f);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                f[i] = inside(c, i) ? f[i] : 0.f;
            v.set(f);
        }
    }
    __device__ void store(T *rows, int64_t row, int c, const Pack<T, VEC> &v) const
    {
        T *o = rows + first(row) + static_cast<int64_t>(c) * VEC;
        if (!ragged(c)) {
            v.store(o);
            return;
        }
        float f[VEC];
        v.get(f);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (inside(c, i))
                o[i] = from_f<T>(f[i]);
    }
    __device__ void store_codes(uint8_t *rows, int64_t row, int c, const float (&f)[VEC]) const
    {
        uint8_t *o = rows + first(row) + static_cast<int64_t>(c) * VEC;
        if (!ragged(c)) {
            store_e4m3<VEC>(o, f);
            return;
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (inside(c, i))
                o[i] = static_cast<uint8_t>(e4m3_pair(f[i], 0.f) & 0xffu);
    }
    // Fill a ring slot's input `k` from `rows` (the bytes are counted by the
    // caller).  Granules that reach past the last row's end are not read there:
    // their elements are copied one by one, before the slot's barrier is armed.
    __device__ uint32_t bytes(int64_t row) const
    {
        const int64_t avail = M * D - first(row);
        return 16u * static_cast<uint32_t>(PH && static_cast<int64_t>(packs) * VEC > avail ? packs - 1 : packs);
    }
    __device__ void copy_tail(T *slot, const T *rows, int64_t row) const
    {
        if (PH)
            for (int64_t e = first(row) + bytes(row) / sizeof(T); e < M * D && e < first(row) + packs * VEC; ++e)
                slot[e - first(row)] = rows[e];
    }
};

// One group's ring: `inputs` rows (bulk copies) per slot.
struct Ring {
    uint32_t slots_s, full_s;  // shared addresses: the group's slots, its barriers
    const uint8_t *slots;
    int n, slot = 0;
    uint32_t phase = 0;
    uint32_t row_bytes, slot_bytes;
    __device__ Ring(const RingPlan &r, uint8_t *smem, RingSync &sy, int group)
        : n(r.slots), row_bytes(r.row_bytes), slot_bytes(r.slot_bytes)
    {
        slots = smem + r.slot_off + static_cast<size_t>(group) * r.slots * r.slot_bytes;
        slots_s = smem_u32(slots);
        full_s = smem_u32(&sy.full[group * RING_MAX_SLOTS]);
    }
    // One thread of the group, before its first fill.
    __device__ void init() const
    {
        for (int s = 0; s < n; ++s)
            mbar_init(full_s + 8u * s, 1);
        fence_mbar_init();
    }
    // One thread: arm slot s and start the copies of row `row` (with a PH span,
    // pitches are D).
    template <class T, bool PH>
    __device__ void fill(const RowSpan<T, PH> &span, int s, int64_t row, const T *a, int64_t lda, const T *b,
                         int64_t ldb, const T *c, int64_t ldc) const
    {
        const uint32_t bar = full_s + 8u * s, dst = slots_s + s * slot_bytes, n = span.bytes(row);
        if (PH) {
            T *slot_p = reinterpret_cast<T *>(const_cast<uint8_t *>(slots) + s * slot_bytes);
            const int gap = static_cast<int>(row_bytes / sizeof(T));
            span.copy_tail(slot_p, a, row);
            if (b)
                span.copy_tail(slot_p + gap, b, row);
            if (c)
                span.copy_tail(slot_p + 2 * gap, c, row);
        }
        mbar_arrive_expect_tx(bar, n * (1u + (b ? 1u : 0u) + (c ? 1u : 0u)));
        if (n == 0)
            return;
        bulk_load_g2s(dst, a + (PH ? span.first(row) : row * lda), n, bar);
        if (b)
            bulk_load_g2s(dst + row_bytes, b + (PH ? span.first(row) : row * ldb), n, bar);
        if (c)
            bulk_load_g2s(dst + 2 * row_bytes, c + (PH ? span.first(row) : row * ldc), n, bar);
    }
    __device__ const uint8_t *input(int i) const { return slots + slot * slot_bytes + i * row_bytes; }
    __device__ void advance()
    {
        if (++slot == n) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// Copies the weights to shared memory, shifted by the block's phase (zeros
// around them); after it every thread sees them and the groups' barriers.
template <class W, bool PH, class Span>
__device__ __forceinline__ const W *ring_weights(uint8_t *smem, const RingPlan &r, const W *w, const Span &span)
{
    W *ws = reinterpret_cast<W *>(smem + r.w_off);
    if (!PH && !r.w_shared) {
        __syncthreads();
        return w;
    }
    if (PH) {
        // 16 bytes a load, several in flight, each element to its shifted place
        constexpr int VW = 16 / static_cast<int>(sizeof(W));
        const int d = static_cast<int>(span.D), whole = d / VW, end = span.phase + d;
#pragma unroll 4
        for (int c = threadIdx.x; c < whole; c += blockDim.x) {
            const uint4 v = reinterpret_cast<const uint4 *>(w)[c];
            const W *e = reinterpret_cast<const W *>(&v);
#pragma unroll
            for (int i = 0; i < VW; ++i)
                ws[span.phase + c * VW + i] = e[i];
        }
        if (threadIdx.x < VW && whole * VW + static_cast<int>(threadIdx.x) < d)
            ws[span.phase + whole * VW + threadIdx.x] = w[whole * VW + threadIdx.x];
        if (static_cast<int>(threadIdx.x) < span.phase)
            ws[threadIdx.x] = from_f<W>(0.f);
        if (end + static_cast<int>(threadIdx.x) < span.packs * Span::VEC)
            ws[end + threadIdx.x] = from_f<W>(0.f);
    } else {
        for (int i = threadIdx.x; i < static_cast<int>(span.D * sizeof(W) / 16); i += blockDim.x)
            reinterpret_cast<uint4 *>(ws)[i] = reinterpret_cast<const uint4 *>(w)[i];
    }
    __syncthreads();
    return ws;
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

// A ring of `inputs` rows of D elements per slot, or false where a row is too
// long for two slots.  At least two slots per group, then as many groups as the
// threads and the shared memory allow, then more slots.
bool plan_ring(RingPlan *r, bool phased, int64_t D, int elem, int welem, int inputs, int max_threads)
{
    const int64_t vec = 16 / elem;
    const int64_t packs = phased ? (D + 2 * vec - 2) / vec : D / vec;  // at most
    const int64_t row_bytes = packs * 16, slot = row_bytes * inputs;
    int64_t wbytes = (packs * vec * welem + 127) / 128 * 128;
    r->w_shared = 1;
    if (!phased && wbytes + 2 * slot > RING_BUDGET && 2 * slot <= RING_BUDGET) {
        wbytes = 0;
        r->w_shared = 0;
    }
    const int64_t gt = (packs + 32 * RING_NV - 1) / (32 * RING_NV) * 32;
    if (gt > max_threads || wbytes + 2 * slot > RING_BUDGET)
        return false;
    int64_t groups = max_threads / gt;
    groups = groups < RING_MAX_GROUPS ? groups : RING_MAX_GROUPS;
    const int64_t fit = (RING_BUDGET - wbytes) / (2 * slot);
    groups = groups < fit ? groups : fit;
    int64_t slots = (RING_BUDGET - wbytes) / (slot * groups);
    slots = slots < RING_MAX_SLOTS ? slots : RING_MAX_SLOTS;
    r->group_threads = static_cast<int>(gt);
    r->groups = static_cast<int>(groups);
    r->slots = static_cast<int>(slots);
    r->row_bytes = static_cast<uint32_t>(row_bytes);
    r->w_off = 0;
    r->slot_off = static_cast<uint32_t>(wbytes);
    r->slot_bytes = static_cast<uint32_t>(slot);
    r->bytes = static_cast<uint32_t>(wbytes + groups * slots * slot);
    return true;
}

template <class K>
cudaError_t ring_opt_in(K kernel, std::atomic<unsigned long long> &done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (done.load() & (1ull << (dev & 63))))
        return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, RING_BUDGET);
    if (e == cudaSuccess)
        done.fetch_or(1ull << (dev & 63));
    return e;
}

// How a call's rows may be moved: 16-byte packs that start with every row; 16-byte
// granules of contiguous rows of any length; or element by element.
enum Rows { ROWS_VEC, ROWS_PHASED, ROWS_ANY };
bool use_ring(Rows rows, int64_t M, int64_t D)
{
    if (rows == ROWS_PHASED)
        return D >= RING_LONG_D || M >= RING_MIN_ROWS_PHASED;
    return rows == ROWS_VEC && M >= RING_MIN_ROWS;
}
// Blocks of a ring kernel: a multiple of eight (RowSpan), at most one per SM.
int ring_blocks(int64_t M, int num_sms)
{
    const int64_t most = num_sms / 8 * 8, want = (M + 7) / 8 * 8;
    return static_cast<int>(want < most ? want : most);
}
constexpr int64_t PHASED_MIN_D = 32;  // a row covers whole granules besides its two ragged ones

// Threads per block for a row of `packs` packs, NV per thread.
int threads_for(int64_t packs, int nv)
{
    const int64_t t = ((packs + nv - 1) / nv + 31) / 32 * 32;
    return t <= 1024 ? static_cast<int>(t) : 0;
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

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

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
