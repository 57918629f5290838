// block_norm_common.cuh -- what block_norm and its gradient share: the gate, and the
// parameters of the ring kernels in shared memory.
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

// The parameters of a ring kernel: pre in its type, then post times a gate of one row in
// fp32 (one load and one product less for a column than the two of them apart), both in
// shared memory where they fit, shifted by the block's phase.  A gate of several rows is
// read where it is: the tokens of a row of it follow one another.
template <class T, class W, bool PH, class P>
struct RingParams {
    using Span = RowSpan<T, PH>;
    static constexpr int VEC = Span::VEC;
    const W *pre;
    const float *factor;  // null: none, or not in shared memory
    bool gate_apart;
    __device__ __forceinline__ RingParams(uint8_t *smem, const RingPlan &r, const Span &span, const P &p)
        : pre(static_cast<const W *>(p.pre)), factor(nullptr), gate_apart(p.gate && p.gate_tokens != p.M)
    {
        RingPlan at = r;
        if (pre) {
            pre = ring_weights<W, PH>(smem, at, pre, span);
            at.w_off += r.row_bytes / static_cast<uint32_t>(sizeof(T)) * static_cast<uint32_t>(sizeof(W));
        }
        const bool one_gate = p.gate && !gate_apart;
        if ((p.post || one_gate) && (PH || r.w_shared)) {
            float *f = reinterpret_cast<float *>(smem + at.w_off);
            for (int i = threadIdx.x; i < span.packs * VEC; i += blockDim.x) {
                const int k = i - span.phase;
                const bool in = k >= 0 && k < span.D;
                float v = in ? 1.f : 0.f;
                if (in && p.post)
                    v = to_f(static_cast<const W *>(p.post)[k]);
                if (in && one_gate)
                    v *= gate_one<T>(p.gate, p.gate_f32, k);
                f[i] = v;
            }
            factor = f;
        }
        __syncthreads();
    }
    // the factors of pack c of row `row`
    __device__ __forceinline__ void factors(const P &p, const Span &span, int64_t row, int c, float2 (&cf)[VEC / 2]) const
    {
        const int64_t gate_row = gate_apart ? row / p.gate_tokens * p.D : 0;
        if (!PH && !factor) {
            column_factors<T, W, VEC>(p, gate_row, c * VEC, cf);
            return;
        }
        if (factor) {
            get2<float, VEC>(load_pack<float, VEC>(factor + c * VEC), cf);
        } else {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i)
                cf[i] = both(1.f);
        }
        if (!gate_apart)
            return;
        float2 u[VEC / 2];
        if constexpr (PH) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float v = span.inside(c, i) ? gate_one<T>(p.gate, p.gate_f32, gate_row + c * VEC + i - span.phase) : 0.f;
                (i % 2 ? u[i / 2].y : u[i / 2].x) = v;
            }
        } else {
            gate_at<T, VEC>(p.gate, p.gate_f32, gate_row + c * VEC, u);
        }
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i)
            cf[i] = mul2(cf[i], u[i]);
    }
};
// Bytes of them for each column.
template <class W, class P>
int param_bytes(const P &p)
{
    return static_cast<int>((p.pre ? sizeof(W) : 0) + (p.post || (p.gate && p.gate_tokens == p.M) ? sizeof(float) : 0));
}

}  // namespace
}  // namespace lf
