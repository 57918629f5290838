// block_norm_common.cuh -- what block_norm and its gradient share.
#pragma once
#include "rms_norm_common.cuh"

namespace lf {
namespace {

// N columns in fp32 as pairs; one column is the first half of a pair of which the
// second counts for nothing.
template <int VEC>
constexpr int PAIRS = VEC == 1 ? 1 : VEC / 2;
template <class T, int VEC>
__device__ __forceinline__ void pairs_of(const Pack<T, VEC> &p, float2 (&f)[PAIRS<VEC>])
{
    float v[VEC];
    p.get(v);
    if constexpr (VEC == 1) {
        f[0] = make_float2(v[0], 0.f);
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i)
            f[i] = make_float2(v[2 * i], v[2 * i + 1]);
    }
}
template <class T, int VEC>
__device__ __forceinline__ void from_pairs(Pack<T, VEC> &p, const float2 (&f)[PAIRS<VEC>])
{
    if constexpr (VEC == 1) {
        const float v[1] = {f[0].x};
        p.set(v);
    } else {
        set2<T, VEC>(p, f);
    }
}

// The gate from element i on, VEC columns, 16 bytes or one element a load.
template <class T, int VEC>
__device__ __forceinline__ void gate_at(const void *gate, bool f32, int64_t i, float2 (&u)[PAIRS<VEC>])
{
    if (f32)
        pairs_of<float, VEC>(load_pack<float, VEC>(static_cast<const float *>(gate) + i), u);
    else
        pairs_of<T, VEC>(load_pack<T, VEC>(static_cast<const T *>(gate) + i), u);
}
template <class T>
__device__ __forceinline__ float gate_one(const void *gate, bool f32, int64_t i)
{
    return f32 ? static_cast<const float *>(gate)[i] : to_f(static_cast<const T *>(gate)[i]);
}

// What a column of the block's output is multiplied by besides its row's factor: post
// times the gate (1 where the call has neither), an fp32 product, from memory.  P: the
// parameters of either pass.
template <class T, class W, int VEC, class P>
__device__ __forceinline__ void column_factors(const P &p, int64_t gate_row, int64_t at, float2 (&cf)[PAIRS<VEC>])
{
    if (p.post) {
        pairs_of<W, VEC>(load_pack<W, VEC>(static_cast<const W *>(p.post) + at), cf);
    } else {
#pragma unroll
        for (int i = 0; i < PAIRS<VEC>; ++i)
            cf[i] = both(1.f);
    }
    if (p.gate) {
        float2 u[PAIRS<VEC>];
        gate_at<T, VEC>(p.gate, p.gate_f32, gate_row + at, u);
#pragma unroll
        for (int i = 0; i < PAIRS<VEC>; ++i)
            cf[i] = mul2(cf[i], u[i]);
    }
}

// VEC elements at a shared-memory address, 16 bytes a load.
template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> lds_pack(uint32_t at)
{
    Pack<T, VEC> p;
#pragma unroll
    for (int i = 0; i < Pack<T, VEC>::WORDS; i += 4)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(p.u[i]), "=r"(p.u[i + 1]), "=r"(p.u[i + 2]), "=r"(p.u[i + 3])
                     : "r"(at + 4u * i));
    return p;
}

}  // namespace
}  // namespace lf
