// rms_norm.cu -- the residual addition with its root-mean-square norm, the
// 8-bit form of its output, and the gradient of both.
//
// Forward, one row (token) of D channels:
//   h = rn(x + residual)                      the stream, kept in its own type
//   r = 1 / sqrt(mean_d h^2 + eps),  f = h r weight
//   y = rn(f),  or  scale = max_d |f| / 448 (1 if that is 0),  y = e4m3(f / scale)
// Backward, with g = dy weight and the same r (recomputed from the h that the
// forward pass kept, so nothing but h has to be saved):
//   dx = r g - h r^3 mean_d(g h) + dh         the gradient of x and of residual
//   dweight = sum over rows of dy h r
//
// Both passes are bound by memory: every element of the row is read once and
// held in registers between the reduction and the output (rows too long for
// that take the *_long kernels, which read the row again from L2).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <type_traits>

#include "lf_internal.h"

namespace lf {
namespace {

constexpr float E4M3_MAX = 448.f;
constexpr int MAX_WARPS = 32;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v)
{
    return v;
}
template <>
__device__ __forceinline__ __half from_f<__half>(float v)
{
    return __float2half_rn(v);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v)
{
    return __float2bfloat16_rn(v);
}

// VEC consecutive elements, moved 16 bytes (VEC * sizeof(T) if that is less) at
// a time; VEC = 1 has no alignment beyond the element's.
template <class T, int VEC>
struct Pack {
    static constexpr int BYTES = VEC * static_cast<int>(sizeof(T));
    static constexpr int ALIGN = BYTES >= 16 ? 16 : BYTES;
    alignas(ALIGN) T v[VEC];
};

template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T *p)
{
    Pack<T, VEC> r;
    if constexpr (Pack<T, VEC>::BYTES >= 16) {
#pragma unroll
        for (int i = 0; i < Pack<T, VEC>::BYTES / 16; ++i)
            reinterpret_cast<uint4 *>(r.v)[i] = reinterpret_cast<const uint4 *>(p)[i];
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            r.v[i] = p[i];
    }
    return r;
}

template <class T, int VEC>
__device__ __forceinline__ void store_pack(T *p, const Pack<T, VEC> &r)
{
    if constexpr (Pack<T, VEC>::BYTES >= 16) {
#pragma unroll
        for (int i = 0; i < Pack<T, VEC>::BYTES / 16; ++i)
            reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(r.v)[i];
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            p[i] = r.v[i];
    }
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

// The e4m3 scale of a row whose largest |f| is amax, and how to divide by it:
// a product with the reciprocal, or a division where the reciprocal of a tiny
// scale could overflow.
struct RowScale {
    float scale, inv;
    bool divide;
    __device__ __forceinline__ explicit RowScale(float amax)
    {
        scale = amax == 0.f ? 1.f : amax / E4M3_MAX;
        divide = scale < 0x1p-100f;
        inv = 1.f / scale;
    }
    __device__ __forceinline__ float operator()(float f) const { return divide ? f / scale : f * inv; }
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

// One row per block and step; thread t holds the row's packs t, t + threads, ...
// (NV of them at most).
template <class T, class W, int VEC, int NV, bool FP8>
__global__ void __launch_bounds__(NV <= 2 ? 512 : 1024) k_rms_norm(const NormParams p)
{
    __shared__ float2 sh[2][MAX_WARPS];
    const int packs = static_cast<int>(p.D / VEC);
    const T *x = static_cast<const T *>(p.x);
    const T *res = static_cast<const T *>(p.residual);
    const W *w = static_cast<const W *>(p.weight);
    int buf = 0;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, buf ^= 1) {
        Pack<T, VEC> h[NV];
        float ss = 0.f;
        uint32_t mx = 0u;
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
                    const Pack<T, VEC> r = load_pack<T, VEC>(res + row * p.ldr + static_cast<int64_t>(c) * VEC);
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        h[j].v[i] = from_f<T>(to_f(h[j].v[i]) + to_f(r.v[i]));
                    store_pack<T, VEC>(static_cast<T *>(p.h) + row * p.D + static_cast<int64_t>(c) * VEC, h[j]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c < packs) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float v = to_f(h[j].v[i]);
                    ss = fmaf(v, v, ss);
                }
                if (FP8) {
                    const Pack<W, VEC> wv = load_pack<W, VEC>(w + static_cast<int64_t>(c) * VEC);
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        mx = max(mx, mag_bits(to_f(h[j].v[i]) * to_f(wv.v[i])));
                }
            }
        }
        const float2 sums = block_reduce<true>(ss, mx, sh[buf]);
        const float r = rsqrtf(sums.x / static_cast<float>(p.D) + p.eps);
        const RowScale rs(sums.y * r);
        if (FP8 && threadIdx.x == 0)
            p.scale[row] = rs.scale;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c < packs) {
                const Pack<W, VEC> wv = load_pack<W, VEC>(w + static_cast<int64_t>(c) * VEC);
                const int64_t o = row * p.D + static_cast<int64_t>(c) * VEC;
                float f[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    f[i] = to_f(h[j].v[i]) * r * to_f(wv.v[i]);
                if (FP8) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        f[i] = rs(f[i]);
                    store_e4m3<VEC>(static_cast<uint8_t *>(p.y) + o, f);
                } else {
                    Pack<T, VEC> yv;
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        yv.v[i] = from_f<T>(f[i]);
                    store_pack<T, VEC>(static_cast<T *>(p.y) + o, yv);
                }
            }
        }
    }
}

// Rows that do not fit the registers of a block: the row is read a second time
// (h, which each thread wrote itself, or x where nothing is added).
template <class T, class W, bool FP8>
__global__ void __launch_bounds__(1024) k_rms_norm_long(const NormParams p)
{
    __shared__ float2 sh[2][MAX_WARPS];
    const T *res = static_cast<const T *>(p.residual);
    const W *w = static_cast<const W *>(p.weight);
    int buf = 0;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, buf ^= 1) {
        const T *x = static_cast<const T *>(p.x) + row * p.ldx;
        T *h = res ? static_cast<T *>(p.h) + row * p.D : nullptr;
        float ss = 0.f;
        uint32_t mx = 0u;
        for (int64_t c = threadIdx.x; c < p.D; c += blockDim.x) {
            T t = x[c];
            if (res) {
                t = from_f<T>(to_f(t) + to_f(res[row * p.ldr + c]));
                h[c] = t;
            }
            const float v = to_f(t);
            ss = fmaf(v, v, ss);
            if (FP8)
                mx = max(mx, mag_bits(v * to_f(w[c])));
        }
        const float2 sums = block_reduce<true>(ss, mx, sh[buf]);
        const float r = rsqrtf(sums.x / static_cast<float>(p.D) + p.eps);
        const RowScale rs(sums.y * r);
        if (FP8 && threadIdx.x == 0)
            p.scale[row] = rs.scale;
        for (int64_t c = threadIdx.x; c < p.D; c += blockDim.x) {
            const float f[1] = {to_f(res ? h[c] : x[c]) * r * to_f(w[c])};
            if (FP8) {
                const float q[1] = {rs(f[0])};
                store_e4m3<1>(static_cast<uint8_t *>(p.y) + row * p.D + c, q);
            } else {
                static_cast<T *>(p.y)[row * p.D + c] = from_f<T>(f[0]);
            }
        }
    }
}

// Backward: block b takes rows b, b + blocks, ...; thread t keeps the weight
// gradient of its own columns (packs t, t + threads, ...) in fp32 registers
// over all of them and writes it to row b of `partial` at the end; the sum over
// blocks is k_rms_norm_dweight's, in block order: no atomics, one result.
template <class T, class W, int VEC, int NV>
__global__ void __launch_bounds__(VEC * NV <= 8 ? 512 : 1024) k_rms_norm_bwd(const NormBwdParams p)
{
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
                const Pack<W, VEC> wv = load_pack<W, VEC>(w + static_cast<int64_t>(c) * VEC);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float v = to_f(h[j].v[i]);
                    ss = fmaf(v, v, ss);
                    gh = fmaf(to_f(dy[j].v[i]) * to_f(wv.v[i]), v, gh);
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
                const Pack<W, VEC> wv = load_pack<W, VEC>(w + static_cast<int64_t>(c) * VEC);
                Pack<T, VEC> dh, dx;
                if (p.dh)
                    dh = load_pack<T, VEC>(static_cast<const T *>(p.dh) + oc);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float v = to_f(h[j].v[i]), d = to_f(dy[j].v[i]);
                    acc[j][i] = fmaf(d, v * r, acc[j][i]);
                    const float g = r * (d * to_f(wv.v[i]) - v * k);
                    dx.v[i] = from_f<T>(p.dh ? g + to_f(dh.v[i]) : g);
                }
                store_pack<T, VEC>(static_cast<T *>(p.dx) + oc, dx);
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
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    a.v[i] = acc[j][i];
                store_pack<float, VEC>(out + static_cast<int64_t>(c) * VEC, a);
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

// dweight[c] = sum over blocks of partial[b][c]: 32 columns per block, 16 rows of
// threads that each sum every 16th block's row; the 16 sums are added in order.
constexpr int DW_ROWS = 16;
template <class W>
__global__ void __launch_bounds__(32 * DW_ROWS)
    k_rms_norm_dweight(const float *partial, W *dweight, int64_t D, int blocks)
{
    __shared__ float sh[DW_ROWS][32];
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    float s = 0.f;
    if (c < D)
        for (int b = threadIdx.y; b < blocks; b += DW_ROWS)
            s += partial[b * D + c];
    sh[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < D) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < DW_ROWS; ++i)
            s += sh[i][threadIdx.x];
        dweight[c] = from_f<W>(s);
    }
}

// Threads per block for a row of `packs` packs, NV per thread.
int threads_for(int64_t packs, int nv)
{
    const int64_t t = ((packs + nv - 1) / nv + 31) / 32 * 32;
    return t <= 1024 ? static_cast<int>(t) : 0;
}

template <class T, class W, int VEC, bool FP8>
bool launch_norm_regs(const NormParams &p, int num_sms, cudaStream_t s)
{
    const int64_t packs = p.D / VEC;
    (void)num_sms;
    const unsigned grid = static_cast<unsigned>(p.M < 0x7fffffff ? p.M : 0x7fffffff);
    int t;
    if ((t = threads_for(packs, 1)) && t <= 512)
        k_rms_norm<T, W, VEC, 1, FP8><<<grid, t, 0, s>>>(p);
    else if ((t = threads_for(packs, 2)) && t <= 512)
        k_rms_norm<T, W, VEC, 2, FP8><<<grid, t, 0, s>>>(p);
    else if ((t = threads_for(packs, 4)))
        k_rms_norm<T, W, VEC, 4, FP8><<<grid, t, 0, s>>>(p);
    else if ((t = threads_for(packs, 8)))
        k_rms_norm<T, W, VEC, 8, FP8><<<grid, t, 0, s>>>(p);
    else
        return false;
    return true;
}

template <class T, class W, bool FP8>
cudaError_t launch_norm_t(const NormParams &p, bool vec, int num_sms, cudaStream_t s)
{
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    const bool done = vec ? launch_norm_regs<T, W, V, FP8>(p, num_sms, s) : launch_norm_regs<T, W, 1, FP8>(p, num_sms, s);
    if (!done)
        k_rms_norm_long<T, W, FP8><<<static_cast<unsigned>(p.M < 0x7fffffff ? p.M : 0x7fffffff), 1024, 0, s>>>(p);
    return cudaGetLastError();
}

template <class T, class W>
cudaError_t launch_norm_tw(const NormParams &p, bool vec, bool fp8, int num_sms, cudaStream_t s)
{
    return fp8 ? launch_norm_t<T, W, true>(p, vec, num_sms, s) : launch_norm_t<T, W, false>(p, vec, num_sms, s);
}

template <class T, class W, int VEC>
bool launch_bwd_regs(const NormBwdParams &p, int grid, cudaStream_t s)
{
    constexpr int PER = 16 / VEC;  // at most 16 columns per thread
    const int64_t packs = p.D / VEC;
    int t;
    if constexpr (PER >= 2)
        if ((t = threads_for(packs, PER / 2)) && t <= 512) {
            k_rms_norm_bwd<T, W, VEC, PER / 2><<<grid, t, 0, s>>>(p);
            return true;
        }
    if ((t = threads_for(packs, PER))) {
        k_rms_norm_bwd<T, W, VEC, PER><<<grid, t, 0, s>>>(p);
        return true;
    }
    return false;
}

template <class T, class W>
cudaError_t launch_bwd_tw(const NormBwdParams &p, bool vec, void *dweight, int blocks, cudaStream_t s)
{
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    if (!(vec ? launch_bwd_regs<T, W, V>(p, blocks, s) : launch_bwd_regs<T, W, 1>(p, blocks, s)))
        k_rms_norm_bwd_long<T, W><<<blocks, 1024, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !dweight)
        return e;
    k_rms_norm_dweight<W><<<static_cast<unsigned>((p.D + 31) / 32), dim3(32, DW_ROWS), 0, s>>>(
        p.partial, static_cast<W *>(dweight), p.D, blocks);
    return cudaGetLastError();
}

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

// dtype / wdtype: 0 bf16, 1 fp16, 2 fp32; wdtype is dtype or 2.
cudaError_t launch_rms_norm(const NormParams &p, int dtype, int wdtype, bool fp8, int num_sms, cudaStream_t s)
{
    const int64_t v = dtype == 2 ? 4 : 8;
    const bool vec = p.D % v == 0 && p.ldx % v == 0 && al16(p.x) && al16(p.y) && al16(p.weight) &&
                     (!p.residual || (p.ldr % v == 0 && al16(p.residual) && al16(p.h)));
    if (dtype == 0)
        return wdtype == 0 ? launch_norm_tw<__nv_bfloat16, __nv_bfloat16>(p, vec, fp8, num_sms, s)
                           : launch_norm_tw<__nv_bfloat16, float>(p, vec, fp8, num_sms, s);
    if (dtype == 1)
        return wdtype == 1 ? launch_norm_tw<__half, __half>(p, vec, fp8, num_sms, s)
                           : launch_norm_tw<__half, float>(p, vec, fp8, num_sms, s);
    return launch_norm_tw<float, float>(p, vec, fp8, num_sms, s);
}

int rms_norm_bwd_blocks(int64_t M) { return static_cast<int>(M < RMS_BWD_BLOCKS ? M : RMS_BWD_BLOCKS); }

cudaError_t launch_rms_norm_bwd(const NormBwdParams &p, void *dweight, int dtype, int wdtype, cudaStream_t s)
{
    const int64_t v = dtype == 2 ? 4 : 8;
    const bool vec = p.D % v == 0 && al16(p.dy) && al16(p.h) && al16(p.weight) && al16(p.dx) &&
                     (!p.dh || al16(p.dh)) && (!p.partial || al16(p.partial));
    const int blocks = rms_norm_bwd_blocks(p.M);
    if (dtype == 0)
        return wdtype == 0 ? launch_bwd_tw<__nv_bfloat16, __nv_bfloat16>(p, vec, dweight, blocks, s)
                           : launch_bwd_tw<__nv_bfloat16, float>(p, vec, dweight, blocks, s);
    if (dtype == 1)
        return wdtype == 1 ? launch_bwd_tw<__half, __half>(p, vec, dweight, blocks, s)
                           : launch_bwd_tw<__half, float>(p, vec, dweight, blocks, s);
    return launch_bwd_tw<float, float>(p, vec, dweight, blocks, s);
}

}  // namespace lf
