// block_norm_grads.cu -- the gradient of block_norm.  With x, h, the gate row u and
// g = dy pre, r1 and r2 recomputed from the x and h that were kept:
//   H  = r2 (g - h r2^2 mean(g h)) + dh                       the gradient at h
//   dresidual = alpha H,   dx = r1 (c' - x r1^2 mean(c' x)),  c' = beta H (post u)
//                          (dx = c' without post)
// mean(c' x) needs no second reduction: with c = x (post u),
//   sum c' x = beta (r2 (sum g c - r2^2 mean(g h) sum h c) + sum dh c),
// so one reduction of six sums serves the row.  The parameters' gradients are
//   dpre = sum over rows of dy h r2,   S = sum over a gate row's tokens of H x r1,
//   dpost = beta sum over gate rows of u S,   dgate = beta post S
// (S of H x, and dgate = beta S, without post), so a thread keeps two sums for each of
// its columns, not three.  Bound by memory: every element is read once.
#include "block_norm_common.cuh"

namespace lf {
namespace {

// A row's six sums over its columns (what a term has none of is 0).
struct RowSums {
    float v[6];  // h^2, g h, x^2, g c, h c, dh c
    __device__ __forceinline__ explicit RowSums(const float2 (&s)[6])
    {
#pragma unroll
        for (int i = 0; i < 6; ++i)
            v[i] = s[i].x + s[i].y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < 6; ++i)
                v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
    __device__ __forceinline__ void put(float *sh) const
    {
        *reinterpret_cast<float4 *>(sh) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float2 *>(sh + 4) = make_float2(v[4], v[5]);
    }
    // sh: [CTA of the cluster][warp][8]
    template <int WARPS>
    __device__ __forceinline__ void add_all(const float (*sh)[WARPS][8], int ctas, int first_warp, int warps)
    {
#pragma unroll
        for (int i = 0; i < 6; ++i)
            v[i] = 0.f;
        for (int c = 0; c < ctas; ++c)
            for (int w = first_warp; w < first_warp + warps; ++w) {
                const float4 a = *reinterpret_cast<const float4 *>(sh[c][w]);
                const float2 b = *reinterpret_cast<const float2 *>(sh[c][w] + 4);
                v[0] += a.x;
                v[1] += a.y;
                v[2] += a.z;
                v[3] += a.w;
                v[4] += b.x;
                v[5] += b.y;
            }
    }
};

// A row's factors: H = r2 dy pre - h m + dh, dx = r1 H cf - x k, where cf has beta in it
// (and so have the sums of c).
struct RowFactors {
    float r1, r2, m, k;
    __device__ __forceinline__ RowFactors(const BlockNormBwdParams &p, const RowSums &s)
    {
        const float inv_d = 1.f / static_cast<float>(p.D);
        r2 = p.pre ? rsqrtf(s.v[0] * inv_d + p.eps) : 0.f;
        const float m2 = p.pre ? (s.v[1] * inv_d) * r2 * r2 : 0.f;
        m = m2 * r2;
        r1 = p.post ? rsqrtf(s.v[2] * inv_d + p.eps) : 1.f;
        k = p.post ? (fmaf(r2, fmaf(-m2, s.v[4], s.v[3]), s.v[5]) * inv_d) * r1 * r1 * r1 : 0.f;
    }
};

// VEC columns of a row.  What the call has none of is 0 (pre too, where it multiplies a
// dy that is 0), the factors are beta.
template <class T, class W, int VEC>
struct Columns {
    static constexpr int N = PAIRS<VEC>;
    float2 dy[N], h[N], x[N], dh[N], pre[N], cf[N];
    // at(k): the columns in input k (h, dy, x, dh)
    template <class At>
    __device__ __forceinline__ void load(const At &at, const Pack<W, VEC> &w)
    {
        pairs_of<T, VEC>(at(0), h);
        pairs_of<T, VEC>(at(1), dy);
        pairs_of<T, VEC>(at(2), x);
        pairs_of<T, VEC>(at(3), dh);
        pairs_of<W, VEC>(w, pre);
    }
    __device__ __forceinline__ void add_to(const BlockNormBwdParams &p, float2 (&s)[6]) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float2 g = mul2(dy[i], pre[i]);
            s[0] = fma2(h[i], h[i], s[0]);
            s[1] = fma2(g, h[i], s[1]);
            const float2 c = mul2(x[i], cf[i]);  // (not used without post)
            s[2] = fma2(x[i], x[i], s[2]);
            s[3] = fma2(g, c, s[3]);
            s[4] = fma2(h[i], c, s[4]);
            s[5] = fma2(dh[i], c, s[5]);
        }
    }
    // dresidual, dx, and the two sums of the parameters' gradients
    __device__ __forceinline__ void finish(const BlockNormBwdParams &p, const RowFactors &f, Pack<T, VEC> &dres,
                                           Pack<T, VEC> &dx, float2 (&a_pre)[N], float2 (&a_sum)[N]) const
    {
        float2 o[N], q[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float2 dyr = mul2(dy[i], both(f.r2));
            const float2 at_h = fma2(h[i], both(-f.m), fma2(dyr, pre[i], dh[i]));
            const float2 at_x = mul2(at_h, both(f.r1));
            o[i] = mul2(at_h, both(p.residual_scale));
            q[i] = mul2(at_x, cf[i]);
            if (p.post)
                q[i] = fma2(x[i], both(-f.k), q[i]);
            a_pre[i] = fma2(dyr, h[i], a_pre[i]);
            a_sum[i] = fma2(at_x, x[i], a_sum[i]);
        }
        from_pairs<T, VEC>(dres, o);
        from_pairs<T, VEC>(dx, q);
    }
};

// A pack, or zeros where there is nothing to read.
template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> pack_or_zeros(const T *p, int64_t at)
{
    if (p)
        return load_pack<T, VEC>(p + at);
    Pack<T, VEC> z;
    float f[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        f[i] = 0.f;
    z.set(f);
    return z;
}

// The columns' factors times beta.
template <class T, class W, int VEC>
__device__ __forceinline__ void scaled_factors(const BlockNormBwdParams &p, int64_t gate_row, int64_t at,
                                               float2 (&cf)[PAIRS<VEC>])
{
    column_factors<T, W, VEC>(p, gate_row, at, cf);
#pragma unroll
    for (int i = 0; i < PAIRS<VEC>; ++i)
        cf[i] = mul2(cf[i], both(p.branch_scale));
}

template <int N>
__device__ __forceinline__ void clear(float2 (&f)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        f[i] = both(0.f);
}

// Rows of a lane (a block, or a group of warps in the ring kernel).  With one gate row or
// none they are strided.  With several, lane l of `lanes` takes the rows M l / lanes ..
// M (l + 1) / lanes - 1, so that it meets the gate rows one after another, and leaves S of
// lane l and gate row g in row l + g of part_sum: a lane and a gate row that meet are on a
// path on which one or both of them grow, so no two of them share a row.  (Phased rows: the
// lane's rows are shared out over `residues` units, each with those of one phase, and row
// (l + g) residues + r is unit r's, which has no such row where none of its phase is there.)
struct LaneRows {
    int64_t first, end, step;
    __device__ LaneRows(const BlockNormBwdParams &p, int64_t lane, int residue, int64_t strided_first, int64_t strided_step)
    {
        const bool several = p.gate_rows > 1;
        first = several ? p.M * lane / p.lanes : strided_first;
        end = several ? p.M * (lane + 1) / p.lanes : p.M;
        step = several ? p.residues : strided_step;
        if (several && p.residues > 1)
            first += (residue - first % p.residues + p.residues) % p.residues;
    }
};
// After `row`: S of its gate row is complete for this lane.
__device__ __forceinline__ bool gate_row_ends(const BlockNormBwdParams &p, const LaneRows &rows, int64_t row)
{
    return p.gate_rows > 1 &&
           (row + rows.step >= rows.end || (row + rows.step) / p.gate_tokens != row / p.gate_tokens);
}
// The last kernel of a call counts its blocks in words that the first one clears.
__device__ __forceinline__ void clear_counters(const BlockNormBwdParams &p)
{
    if (p.counters && blockIdx.x == 0)
        for (int64_t i = threadIdx.x; i < (p.D + 31) / 32; i += blockDim.x)
            p.counters[i] = 0u;
}

// One row per block and step, its sums of the parameters' gradients in registers.
template <class T, class W, int VEC, int NV>
__global__ void __launch_bounds__(512) k_block_norm_bwd(const __grid_constant__ BlockNormBwdParams p)
{
    wait_previous_kernel();
    let_next_kernel_start();
    constexpr int N = PAIRS<VEC>;
    __shared__ __align__(16) float sh[2][1][MAX_WARPS][8];
    const int packs = static_cast<int>(p.D / VEC);
    const T *const in[4] = {static_cast<const T *>(p.h), static_cast<const T *>(p.dy), static_cast<const T *>(p.x),
                            static_cast<const T *>(p.dh)};
    float2 a_pre[NV][N], a_sum[NV][N];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        clear(a_pre[j]);
        clear(a_sum[j]);
    }
    int buf = 0;
    const LaneRows rows(p, blockIdx.x, 0, blockIdx.x, gridDim.x);
    clear_counters(p);
    for (int64_t row = rows.first; row < rows.end; row += rows.step, buf ^= 1) {
        const int64_t o = row * p.D, gate_row = p.gate ? row / p.gate_tokens * p.D : 0;
        Pack<T, VEC> q[NV][4];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c < packs)
                    q[j][k] = pack_or_zeros<T, VEC>(in[k], o + static_cast<int64_t>(c) * VEC);
        }
        const auto columns = [&](int j, int64_t at) {
            Columns<T, W, VEC> v;
            v.load([&](int k) { return q[j][k]; }, pack_or_zeros<W, VEC>(static_cast<const W *>(p.pre), at));
            scaled_factors<T, W, VEC>(p, gate_row, at, v.cf);
            return v;
        };
        float2 s2[6];
        clear(s2);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c < packs)
                columns(j, static_cast<int64_t>(c) * VEC).add_to(p, s2);
        }
        RowSums s(s2);
        if ((threadIdx.x & 31) == 0)
            s.put(sh[buf][0][threadIdx.x >> 5]);
        __syncthreads();
        s.add_all(sh[buf], 1, 0, blockDim.x >> 5);
        const RowFactors f(p, s);
        const bool ends = p.part_sum && gate_row_ends(p, rows, row);
        float *seg = ends ? p.part_sum + (blockIdx.x + row / p.gate_tokens) * p.D : nullptr;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c < packs) {
                const int64_t at = static_cast<int64_t>(c) * VEC;
                Pack<T, VEC> dres, dx;
                columns(j, at).finish(p, f, dres, dx, a_pre[j], a_sum[j]);
                dres.store(static_cast<T *>(p.dres) + o + at);
                dx.store(static_cast<T *>(p.dx) + o + at);
                if (ends) {
                    Pack<float, VEC> a;
                    from_pairs<float, VEC>(a, a_sum[j]);
                    a.store(seg + at);
                    clear(a_sum[j]);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = threadIdx.x + j * blockDim.x;
        if (c < packs) {
            const int64_t at = static_cast<int64_t>(blockIdx.x) * p.D + static_cast<int64_t>(c) * VEC;
            Pack<float, VEC> a;
            from_pairs<float, VEC>(a, a_pre[j]);
            if (p.part_pre)
                a.store(p.part_pre + at);
            from_pairs<float, VEC>(a, a_sum[j]);
            if (p.part_sum && p.gate_rows <= 1)
                a.store(p.part_sum + at);
        }
    }
}

// Rows too long for the registers: the row is read twice, and the sums are kept in
// their rows of part_pre and part_sum (each thread updates its own columns only).
template <class T, class W>
__global__ void __launch_bounds__(1024) k_block_norm_bwd_long(const __grid_constant__ BlockNormBwdParams p)
{
    wait_previous_kernel();
    let_next_kernel_start();
    __shared__ __align__(16) float sh[2][1][MAX_WARPS][8];
    const T *const in[4] = {static_cast<const T *>(p.h), static_cast<const T *>(p.dy), static_cast<const T *>(p.x),
                            static_cast<const T *>(p.dh)};
    int buf = 0;
    const LaneRows rows(p, blockIdx.x, 0, blockIdx.x, gridDim.x);
    clear_counters(p);
    const auto columns = [&](int64_t row, int64_t c) {
        Columns<T, W, 1> v;
        v.load([&](int k) { return pack_or_zeros<T, 1>(in[k], row * p.D + c); },
               pack_or_zeros<W, 1>(static_cast<const W *>(p.pre), c));
        scaled_factors<T, W, 1>(p, p.gate ? row / p.gate_tokens * p.D : 0, c, v.cf);
        return v;
    };
    const bool several = p.gate_rows > 1;
    for (int64_t row = rows.first; row < rows.end; row += rows.step, buf ^= 1) {
        float2 s2[6];
        clear(s2);
#pragma unroll 4
        for (int64_t c = threadIdx.x; c < p.D; c += blockDim.x)
            columns(row, c).add_to(p, s2);
        RowSums s(s2);
        if ((threadIdx.x & 31) == 0)
            s.put(sh[buf][0][threadIdx.x >> 5]);
        __syncthreads();
        s.add_all(sh[buf], 1, 0, blockDim.x >> 5);
        const RowFactors f(p, s);
        float *pre_sum = p.part_pre ? p.part_pre + static_cast<int64_t>(blockIdx.x) * p.D : nullptr;
        float *sum = p.part_sum ? p.part_sum + (blockIdx.x + (several ? row / p.gate_tokens : 0)) * p.D : nullptr;
        const bool first = row == rows.first, first_of_gate = first || (several && row % p.gate_tokens == 0);
        for (int64_t c = threadIdx.x; c < p.D; c += blockDim.x) {
            float2 a[1] = {both(pre_sum && !first ? pre_sum[c] : 0.f)};
            float2 b[1] = {both(sum && !first_of_gate ? sum[c] : 0.f)};
            Pack<T, 1> dres, dx;
            columns(row, c).finish(p, f, dres, dx, a, b);
            dres.store(static_cast<T *>(p.dres) + row * p.D + c);
            dx.store(static_cast<T *>(p.dx) + row * p.D + c);
            if (pre_sum)
                pre_sum[c] = a[0].x;
            if (sum)
                sum[c] = b[0].x;
        }
    }
}

// ---------------------------------------------------------------- many rows
// Rings of bulk copies as in rms_norm_common.cuh, with three differences.
//
// A row stays in its slot until it is done: with two sums for each column there are no
// registers to keep it in, so it is read from shared memory twice.  Its warps count
// themselves off on an mbarrier when they have, and the slot is filled again.
//
// A row may be shared by the two or four CTAs of a cluster, each with a part of its columns,
// so that longer rows fit.  Every warp stores its six sums in all CTAs, in a place of its
// own, and arrives on an mbarrier of the group there; all are added in the same order
// everywhere.
//
// What the call has none of is read as 16 bytes of zeros (factors of beta), so that a pack's
// loads stand in one straight line.
constexpr int BWD_THREADS = 384;  // 168 registers a thread, 64 of them sums
constexpr int BWD_WARPS = BWD_THREADS / 32;
constexpr int BWD_CLUSTER = 4;
constexpr int BWD_BUDGET = 221 * 1024;  // dynamic shared memory; BwdSync and the ragged granules take 5.5 KB more

struct BwdPlan {
    int cluster, group_threads, groups, slots, packs;  // packs of a CTA's share of a row
    uint32_t factor_off, factor_bytes;                 // factors: of the block, or of each group
    uint32_t row_bytes, slot_off, slot_bytes, bytes;
};

struct BwdSync {
    alignas(16) float sums[2][BWD_CLUSTER][BWD_WARPS][8];
    alignas(16) float constants[2][8];  // zeros, beta
    alignas(8) unsigned long long full[BWD_WARPS][RING_MAX_SLOTS], empty[BWD_WARPS][RING_MAX_SLOTS], landed[BWD_WARPS][2];
};

// ring_wait for what another CTA of the cluster wrote.
__device__ __forceinline__ bool sums_wait(uint32_t bar, uint32_t parity, const WaitLimit &lim)
{
    const auto there = [&] {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        return ok != 0;
    };
    if (there())
        return true;
    const uint64_t t0 = global_timer_ns();
    while (!there()) {
        if (global_timer_ns() - t0 > lim.timeout_ns) {
            atomicCAS(lim.err, 0, 0x108);
            return false;
        }
    }
    return true;
}
// Four floats into any CTA's shared memory (a shared::cluster address).
__device__ __forceinline__ void st_cluster_f32x4(uint32_t addr, float4 v)
{
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

template <class T, class W, bool PH>
__global__ void __launch_bounds__(BWD_THREADS)
    k_block_norm_bwd_ring(const __grid_constant__ BlockNormBwdParams p, const BwdPlan r)
{
    constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ BwdSync sy;
    // The two ragged granules of each group's row, dresidual's and dx's: stored element by element
    // after the others, by one loop.  (Unrolled into every pack's code the kernel does not fit the
    // instruction cache: 8192 x 4081 116 us, so 101, 16384 x 1015 68 and 53.)
    __shared__ uint4 edges[PH ? BWD_WARPS : 1][2][2];
    const int group = threadIdx.x / r.group_threads, t = threadIdx.x % r.group_threads;
    const int warps = r.group_threads >> 5, first_warp = group * warps, warp = threadIdx.x >> 5, lane_id = threadIdx.x & 31;
    const uint32_t clusters = r.cluster, rank = blockIdx.x % clusters;
    const int unit = static_cast<int>(blockIdx.x / clusters), units = static_cast<int>(gridDim.x / clusters);
    const RowSpan<T, PH> span(p.M, p.D, unit);
    const int pack0 = static_cast<int>(rank) * r.packs, packs = min(r.packs, span.packs - pack0);
    const int64_t col0 = static_cast<int64_t>(pack0) * VEC - span.phase;  // of the share's first granule
    const int residues = PH && p.gate_rows > 1 ? VEC : 1, residue = unit % residues;
    const int64_t lane = static_cast<int64_t>(unit / residues) * r.groups + group;
    // neighbouring rows go to neighbouring SMs
    const LaneRows rows(p, lane, residue, static_cast<int64_t>(group) * units + unit, static_cast<int64_t>(units) * r.groups);
    const T *in[4] = {static_cast<const T *>(p.h), static_cast<const T *>(p.dy), static_cast<const T *>(p.x),
                      static_cast<const T *>(p.dh)};
    const uint32_t slots = smem_u32(smem + r.slot_off) + static_cast<uint32_t>(group) * r.slots * r.slot_bytes;
    const uint32_t full = smem_u32(sy.full[group]), empty = smem_u32(sy.empty[group]), landed = smem_u32(sy.landed[group]);
    const auto fill = [&](int slot, int64_t row) {
        const uint32_t bar = full + 8u * slot;
        uint32_t n = 16u * packs, inputs = 0;
        const int64_t at = row * p.D + col0;
        if (PH && at + static_cast<int64_t>(packs) * VEC > p.M * p.D) {
            // the granule that reaches past the last row's end: its elements one by one
            n -= 16u;
            T *s = reinterpret_cast<T *>(smem + r.slot_off + (static_cast<size_t>(group) * r.slots + slot) * r.slot_bytes);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (in[k]) {
                    for (int64_t e = at + (packs - 1) * VEC; e < p.M * p.D; ++e)
                        s[inputs * (r.row_bytes / sizeof(T)) + (e - at)] = in[k][e];
                    ++inputs;
                }
            inputs = 0;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            inputs += in[k] ? 1u : 0u;
        mbar_arrive_expect_tx(bar, n * inputs);
        uint32_t dst = slots + slot * r.slot_bytes;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (in[k]) {
                if (n)
                    bulk_load_g2s(dst, in[k] + at, n, bar);
                dst += r.row_bytes;
            }
    };
    if (t == 0) {
        for (int i = 0; i < r.slots; ++i) {
            mbar_init(full + 8u * i, 1);
            mbar_init(empty + 8u * i, warps);
        }
        mbar_init(landed, warps * clusters);
        mbar_init(landed + 8u, warps * clusters);
        fence_mbar_init();
    }
    if (threadIdx.x < 16)
        sy.constants[threadIdx.x >> 3][threadIdx.x & 7] = threadIdx.x >> 3 ? p.branch_scale : 0.f;
    wait_previous_kernel();
    let_next_kernel_start();
    clear_counters(p);
    if (t == 0) {
        // (test hook: the first block's first group never loads its first row)
        for (int i = p.limit.inject && blockIdx.x == 0 && group == 0 ? 1 : 0;
             i < r.slots && rows.first + i * rows.step < rows.end; ++i)
            fill(i, rows.first + i * rows.step);
    }
    // pre, and post times a gate of one row (a gate of several rows: post times the group's)
    const bool several = p.gate_rows > 1;
    const T *const gate_t = several || !p.gate ? nullptr : static_cast<const T *>(p.gate);
    {
        W *const s_pre = reinterpret_cast<W *>(smem);
        float *const s_f = reinterpret_cast<float *>(smem + r.factor_off);
        const W *pre = static_cast<const W *>(p.pre), *post = static_cast<const W *>(p.post);
        const bool factors = !several && (post || gate_t);
#pragma unroll 4
        for (int i = threadIdx.x; i < packs * VEC; i += blockDim.x) {
            const int64_t k = i + col0;
            const bool inside = !PH || (k >= 0 && k < p.D);
            if (pre)
                s_pre[i] = inside ? pre[k] : from_f<W>(0.f);
            if (factors) {
                float f = inside && post ? to_f(post[k]) : 1.f;
                if (inside && gate_t)
                    f *= gate_one<T>(p.gate, p.gate_f32, k);
                s_f[i] = inside ? f * p.branch_scale : 0.f;
            }
        }
    }
    const uint32_t zeros = smem_u32(sy.constants[0]), betas = smem_u32(sy.constants[1]);
    const uint32_t pre = p.pre ? smem_u32(smem) : zeros, pre_apart = p.pre ? VEC * sizeof(W) : 0u;
    const bool has_factor = p.post || p.gate;
    float *const group_factor =
        reinterpret_cast<float *>(smem + r.factor_off + (several ? static_cast<uint32_t>(group) * r.factor_bytes : 0u));
    const uint32_t factor = has_factor ? smem_u32(group_factor) : betas, factor_apart = has_factor ? VEC * sizeof(float) : 0u;
    if (clusters > 1)
        cluster_sync();  // both CTAs' barriers exist before any sum is sent
    else
        __syncthreads();
    float2 a_pre[RING_NV][VEC / 2], a_sum[RING_NV][VEC / 2];
#pragma unroll
    for (int j = 0; j < RING_NV; ++j) {
        clear(a_pre[j]);
        clear(a_sum[j]);
    }
    // What belongs to the row of its two ragged granules, where they are this thread's (chosen
    // without a branch in the loop, which would keep the packs' loads apart: 8192 x 4081 117.5
    // us with one, 115.7 without)
    uint4 head = make_uint4(~0u, ~0u, ~0u, ~0u), tail = head;
    int j_tail = -1;
    if constexpr (PH) {
        if (t == 0 && pack0 == 0)
            head = span.words(0);
        const int c = span.packs - 1 - pack0;
        if (c >= 0 && c < packs && c % r.group_threads == t) {
            tail = span.words(span.packs - 1);
            j_tail = c / r.group_threads;
        }
    }
    bool ok = true;
    int slot = 0;
    uint32_t phase = 0, count = 0;
    int64_t gate_row = -1;
    for (int64_t row = rows.first; row < rows.end; row += rows.step, ++count) {
        if (several && row / p.gate_tokens != gate_row) {
            // the factors of the next gate row; every thread reads its own columns' only
            gate_row = row / p.gate_tokens;
#pragma unroll(PH ? 1 : RING_NV)
            for (int j = 0; j < RING_NV; ++j) {
                const int c = t + j * r.group_threads;
                if (c >= packs)
                    continue;
                if constexpr (PH) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const int64_t k = col0 + c * VEC + i;
                        float2 f[1] = {both(0.f)};
                        if (k >= 0 && k < p.D)
                            scaled_factors<T, W, 1>(p, gate_row * p.D, k, f);
                        group_factor[c * VEC + i] = f[0].x;
                    }
                } else {
                    float2 f[VEC / 2];
                    scaled_factors<T, W, VEC>(p, gate_row * p.D, col0 + c * VEC, f);
                    Pack<float, VEC> v;
                    set2<float, VEC>(v, f);
                    v.store(group_factor + c * VEC);
                }
            }
        }
        ok = ok && ring_wait(full + 8u * slot, phase, p.limit);
        if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
        }
        // an input's bytes in the slot, and how far apart its packs are
        uint32_t base[4], apart[4], inputs = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            base[k] = in[k] ? slots + slot * r.slot_bytes + inputs * r.row_bytes : zeros;
            apart[k] = in[k] ? 16u : 0u;
            inputs += in[k] ? 1u : 0u;
        }
        // (what lies beside a phased row is cut off for the sums; its results go nowhere)
        const auto columns = [&](int j, int c, bool cut) {
            Columns<T, W, VEC> v;
            uint4 keep = make_uint4(~0u, ~0u, ~0u, ~0u);
            if (PH && cut) {
                if (j == 0)
                    keep = head;
                if (j == j_tail)
                    keep = make_uint4(keep.x & tail.x, keep.y & tail.y, keep.z & tail.z, keep.w & tail.w);
            }
            const auto at = [&](int k) {
                Pack<T, VEC> q = lds_pack<T, VEC>(base[k] + c * apart[k]);
                if (PH && cut)
                    q.keep(keep);
                return q;
            };
            v.load(at, lds_pack<W, VEC>(pre + c * pre_apart));
            get2<float, VEC>(lds_pack<float, VEC>(factor + c * factor_apart), v.cf);
            return v;
        };
        float2 s2[6];
        clear(s2);
#pragma unroll
        for (int j = 0; j < RING_NV; ++j) {
            const int c = t + j * r.group_threads;
            if (c < packs)
                columns(j, c, true).add_to(p, s2);
        }
        RowSums s(s2);
        const uint32_t buf = count & 1u, bar = landed + 8u * buf;
        if (clusters * warps > 1) {
            if (clusters == 1) {
                if (lane_id == 0) {
                    s.put(sy.sums[buf][0][warp]);
                    mbar_arrive(bar);
                }
            } else if (static_cast<uint32_t>(lane_id) < clusters) {
                const uint32_t to = mapa_shared(smem_u32(sy.sums[buf][rank][warp]), lane_id);
                st_cluster_f32x4(to, make_float4(s.v[0], s.v[1], s.v[2], s.v[3]));
                st_cluster_f32x4(to + 16u, make_float4(s.v[4], s.v[5], 0.f, 0.f));
                mbar_arrive_cluster(mapa_shared(bar, lane_id));
            }
            ok = sums_wait(bar, (count >> 1) & 1u, p.limit);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            s.add_all(sy.sums[buf], clusters, first_warp, warps);
        }
        const RowFactors f(p, s);
        const bool ends = p.part_sum && gate_row_ends(p, rows, row);
        float *seg = ends ? p.part_sum + ((lane + row / p.gate_tokens) * residues + residue) * p.D + col0 : nullptr;
#pragma unroll
        for (int j = 0; j < RING_NV; ++j) {
            const int c = t + j * r.group_threads;
            if (c < packs) {
                Pack<T, VEC> dres, dx;
                columns(j, c, false).finish(p, f, dres, dx, a_pre[j], a_sum[j]);
                const int64_t at = row * p.D + col0 + c * VEC;
                if (!span.ragged(pack0 + c)) {
                    dres.store(static_cast<T *>(p.dres) + at);
                    dx.store(static_cast<T *>(p.dx) + at);
                } else {
                    uint4 *e = edges[group][pack0 + c > 0];
                    dres.store(reinterpret_cast<T *>(e));
                    dx.store(reinterpret_cast<T *>(e + 1));
                }
                if (ends) {
                    if constexpr (PH) {
#pragma unroll
                        for (int i = 0; i < VEC; ++i)
                            if (span.inside(pack0 + c, i))
                                seg[c * VEC + i] = i % 2 ? a_sum[j][i / 2].y : a_sum[j][i / 2].x;
                    } else {
                        Pack<float, VEC> a;
                        set2<float, VEC>(a, a_sum[j]);
                        a.store(seg + c * VEC);
                    }
                    clear(a_sum[j]);
                }
            }
        }
        if constexpr (PH) {
            const auto finish_edge = [&](int edge, int c) {
                const T *e = reinterpret_cast<const T *>(edges[group][edge]);
                const int64_t at = row * p.D + static_cast<int64_t>(c) * VEC - span.phase;
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (span.inside(c, i)) {
                        static_cast<T *>(p.dres)[at + i] = e[i];
                        static_cast<T *>(p.dx)[at + i] = e[VEC + i];
                    }
            };
            // (one copy of the code: a thread with both goes round twice)
            const bool first = t == 0 && pack0 == 0, last = j_tail >= 0 && span.packs > 1;
#pragma unroll 1
            for (int e = first ? 0 : 1; e < (last ? 2 : 1); ++e)
                finish_edge(e, e ? span.packs - 1 : 0);
        }
        __syncwarp();
        if (lane_id == 0)
            mbar_arrive(empty + 8u * slot);
        if (t == 0 && row + r.slots * rows.step < rows.end) {
            ok = ring_wait(empty + 8u * slot, phase, p.limit, 0x101);
            if (ok)
                fill(slot, row + r.slots * rows.step);
        }
        if (++slot == r.slots) {
            slot = 0;
            phase ^= 1u;
        }
    }
    if (!ok) {  // copies of this group may still be in flight: give them time to land
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < RING_SETTLE_NS) {
        }
    }
    // the rings are idle: the groups' sums go there, are added in order and written as the unit's row
    float *sums = reinterpret_cast<float *>(smem + r.slot_off);
    const auto merge = [&](const float2 (&acc)[RING_NV][VEC / 2], float *out) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < RING_NV; ++j) {
            const int c = t + j * r.group_threads;
            if (c < packs) {
                Pack<float, VEC> a;
                set2<float, VEC>(a, acc[j]);
                a.store(sums + (static_cast<size_t>(group) * r.packs + c) * VEC);
            }
        }
        __syncthreads();
        const int64_t to = static_cast<int64_t>(unit) * p.D + col0;
        for (int c = threadIdx.x; c < packs * VEC; c += blockDim.x)
            if (!PH || (c + col0 >= 0 && c + col0 < p.D)) {
                float s = sums[c];
                for (int g = 1; g < r.groups; ++g)
                    s += sums[static_cast<size_t>(g) * r.packs * VEC + c];
                out[to + c] = s;
            }
    };
    if (p.part_pre)
        merge(a_pre, p.part_pre);
    if (p.part_sum && p.gate_rows <= 1)
        merge(a_sum, p.part_sum);
    if (clusters > 1)
        cluster_sync();  // no CTA leaves while sums may still be sent to it
}

// The parameters' gradients from their sums.  A block has 32 columns and SUM_ROWS rows of
// threads, whose sums the first warp adds up; what it does goes by blockIdx.y: 0 dpre; 1
// dpost and dgate of one gate row (or none), whose sums, like dpre's, have a row for each of
// `blocks` blocks.  With several gate rows S lies as LaneRows says and the blocks from 1 on
// share the gate rows: each adds up its rows' S, writes their dgate and leaves its part of
// dpost (the sum of u S) in the first row of S that only it reads; the last of a column's
// blocks to do so adds those up, in their order.
constexpr int SUM_ROWS = 16;
// S of many lanes to a gate row is added by all threads of a block, else a gate row each.
__host__ __device__ constexpr bool many_lanes(int64_t lanes, int64_t gate_rows) { return lanes >= SUM_ROWS / 2 * gate_rows; }

// RESIDUES: of phased rows with several gate rows, else 1 (a kernel of its own: its searches
// would cost the other one half of its blocks on an SM, 64 x 5120 9.0 -> 10.7 us).
template <class T, class W, int RESIDUES>
__global__ void __launch_bounds__(32 * SUM_ROWS)
    k_block_norm_sums(const __grid_constant__ BlockNormBwdParams p, int blocks, W *dpost, W *dpre, void *dgate)
{
    wait_previous_kernel();
    __shared__ float sh[SUM_ROWS][32];
    __shared__ bool last;
    const int ty = threadIdx.y;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    const bool in = c < p.D, writes = in && ty == 0;
    const float post = p.post && in ? to_f(static_cast<const W *>(p.post)[c]) : 1.f;
    const auto put_gate = [&](int64_t i, float v) {
        if (p.gate_f32)
            static_cast<float *>(dgate)[i] = v;
        else
            static_cast<T *>(dgate)[i] = from_f<T>(v);
    };
    // the sum over the rows of threads, in their order, in the first of them
    const auto over_rows = [&](float s) {
        __syncthreads();
        sh[ty][threadIdx.x] = s;
        __syncthreads();
        if (ty == 0) {
            s = sh[0][threadIdx.x];
#pragma unroll
            for (int r = 1; r < SUM_ROWS; ++r)
                s += sh[r][threadIdx.x];
        }
        return s;
    };
    if (blockIdx.y == 0 || p.gate_rows <= 1) {
        const float *part = blockIdx.y == 0 ? p.part_pre : p.part_sum;
        if (blockIdx.y == 0 ? !dpre : !dpost && !dgate)
            return;
        float s = 0.f;
#pragma unroll 8
        for (int b = ty; b < blocks; b += SUM_ROWS)
            s += in ? part[static_cast<int64_t>(b) * p.D + c] : 0.f;
        s = over_rows(s);
        if (!writes)
            return;
        if (blockIdx.y == 0) {
            dpre[c] = from_f<W>(s);
            return;
        }
        const float u = p.gate ? gate_one<T>(p.gate, p.gate_f32, c) : 1.f;
        if (dpost)
            dpost[c] = from_f<W>(p.branch_scale * u * s);
        if (dgate)
            put_gate(c, p.branch_scale * post * s);
        return;
    }
    if (!dpost && !dgate)
        return;
    const int sets = gridDim.y - 1, set = blockIdx.y - 1;
    const bool many = many_lanes(p.lanes * RESIDUES, p.gate_rows);
    const auto first_lane = [&](int64_t g) { return ((g * p.gate_tokens + 1) * p.lanes - 1) / p.M; };
    const auto last_lane = [&](int64_t g) { return ((g + 1) * p.gate_tokens * p.lanes - 1) / p.M; };
    // the row of part_sum where a set of blocks leaves its part of dpost
    const auto place = [&](int64_t set_of) {
        const int64_t g = set_of * (many ? 1 : SUM_ROWS);
        return (first_lane(g) + g) * RESIDUES;
    };
    // whether unit r of lane l has rows of gate row g
    const auto there = [&](int64_t l, int64_t g, int r) {
        const int64_t a = max(p.M * l / p.lanes, g * p.gate_tokens);
        const int64_t b = min(p.M * (l + 1) / p.lanes, (g + 1) * p.gate_tokens);
        return b - a >= RESIDUES || a + (r - a % RESIDUES + RESIDUES) % RESIDUES < b;
    };
    // this thread's share (i0, i0 + step, ..) of gate row g's S
    const auto share = [&](int64_t g, int64_t i0, int64_t step) {
        const int64_t l0 = first_lane(g), last = last_lane(g) - l0, n = (last + 1) * RESIDUES;
        const float *part = p.part_sum + (l0 + g) * RESIDUES * p.D + c;
        float s = 0.f;
        if (RESIDUES == 1) {
#pragma unroll 8
            for (int64_t i = i0; i < n; i += step)
                s += in ? part[i * p.D] : 0.f;
        } else {
            // (a lane has `residues` rows or more, so only those at the gate row's ends can lack one)
            constexpr int bits = RESIDUES == 4 ? 2 : 3;
#pragma unroll 4
            for (int64_t i = i0; i < n; i += step) {
                const int64_t l = i >> bits;
                const bool inner = l > 0 && l < last;
                s += in && (inner || there(l0 + l, g, static_cast<int>(i - (l << bits)))) ? part[i * p.D] : 0.f;
            }
        }
        return s;
    };
    float acc = 0.f;  // of dpost
    const int64_t g0 = many ? set : static_cast<int64_t>(set) * SUM_ROWS + ty;
    for (int64_t g = g0; g < p.gate_rows; g += static_cast<int64_t>(sets) * (many ? 1 : SUM_ROWS)) {
        float s = share(g, many ? ty : 0, many ? SUM_ROWS : 1);
        if (many)
            s = over_rows(s);
        if (in && (ty == 0 || !many)) {
            if (dgate)
                put_gate(g * p.D + c, p.branch_scale * post * s);
            if (dpost)
                acc = fmaf(gate_one<T>(p.gate, p.gate_f32, g * p.D + c), s, acc);
        }
    }
    if (!dpost)
        return;
    if (!many)
        acc = over_rows(acc);
    if (sets > 1) {
        // (the rows that the set's first thread row writes over have been read by all of them)
        if (ty == 0) {
            if (in)
                p.part_sum[place(set) * p.D + c] = acc;
            __threadfence();
            __syncwarp();
            if (threadIdx.x == 0)
                last = atomicAdd(p.counters + blockIdx.x, 1u) == static_cast<unsigned>(sets) - 1u;
        }
        __syncthreads();
        if (!last)
            return;
        __threadfence();
        acc = 0.f;
#pragma unroll 4
        for (int i = ty; i < sets; i += SUM_ROWS)
            acc += in ? __ldcg(p.part_sum + place(i) * p.D + c) : 0.f;
        acc = over_rows(acc);
    }
    if (writes)
        dpost[c] = from_f<W>(p.branch_scale * acc);
}

// ---------------------------------------------------------------- launches
template <class T, class W, int VEC>
bool launch_block_bwd_regs(const BlockNormBwdParams &p, int grid, cudaStream_t s, cudaError_t *e)
{
    const int64_t packs = p.D / VEC;
    int t;
    if ((t = threads_for(packs, 8 / VEC)) && t <= 512) {  // eight columns per thread
        *e = launch_overlapped(k_block_norm_bwd<T, W, VEC, 8 / VEC>, dim3(grid), dim3(t), 0, 1, s, p);
        return true;
    }
    if ((t = threads_for(packs, 16 / VEC)) && t <= 512) {
        *e = launch_overlapped(k_block_norm_bwd<T, W, VEC, 16 / VEC>, dim3(grid), dim3(t), 0, 1, s, p);
        return true;
    }
    return false;
}

template <class T, class W, bool PH>
cudaError_t launch_block_bwd_ring(const BlockNormBwdParams &p, const BwdPlan &r, int units, cudaStream_t s)
{
    static std::atomic<unsigned long long> opted{0};
    const cudaError_t e = ring_opt_in(k_block_norm_bwd_ring<T, W, PH>, opted, BWD_BUDGET);
    if (e != cudaSuccess)
        return e;
    return launch_overlapped(k_block_norm_bwd_ring<T, W, PH>, dim3(units * r.cluster), dim3(r.groups * r.group_threads),
                             r.bytes, r.cluster, s, p, r);
}

// Threads of a group for rows of D elements shared by `cluster` CTAs.
int64_t bwd_group_threads(int64_t D, int elem, bool phased, int cluster, int64_t *packs)
{
    const int64_t vec = 16 / elem, all = phased ? (D + 2 * vec - 2) / vec : D / vec;
    *packs = all < cluster ? 1 : (all + cluster - 1) / cluster;
    return (*packs + 32 * RING_NV - 1) / (32 * RING_NV) * 32;
}
// A plan with at most max_groups groups and two slots for each, or false where the rows are
// too long for it.  groups_apart: each group has factors of its own.
bool plan_bwd(BwdPlan *r, bool phased, int64_t D, int elem, int wbytes, bool factors, bool groups_apart, int inputs,
              int cluster, int64_t max_groups)
{
    int64_t packs;
    const int64_t gt = bwd_group_threads(D, elem, phased, cluster, &packs), vec = 16 / elem;
    if (gt > BWD_THREADS || packs * (cluster - 1) * vec >= D)
        return false;
    const int64_t pre = (packs * vec * wbytes + 127) / 128 * 128, f = factors ? packs * vec * 4 : 0;
    const int64_t slot = packs * 16 * inputs;
    int64_t groups = BWD_THREADS / gt;
    groups = groups < max_groups ? groups : max_groups;
    for (; groups > 0; --groups) {
        const int64_t fixed = (pre + f * (groups_apart ? groups : 1) + 127) / 128 * 128;
        int64_t n = (BWD_BUDGET - fixed) / (slot * groups);
        n = n < RING_MAX_SLOTS ? n : RING_MAX_SLOTS;
        if (n < 2)
            continue;
        r->cluster = cluster;
        r->group_threads = static_cast<int>(gt);
        r->groups = static_cast<int>(groups);
        r->slots = static_cast<int>(n);
        r->packs = static_cast<int>(packs);
        r->factor_off = static_cast<uint32_t>(pre);
        r->factor_bytes = static_cast<uint32_t>(f);
        r->row_bytes = static_cast<uint32_t>(packs * 16);
        r->slot_off = static_cast<uint32_t>(fixed);
        r->slot_bytes = static_cast<uint32_t>(slot);
        r->bytes = static_cast<uint32_t>(fixed + groups * n * slot);
        return true;
    }
    return false;
}

// CTAs to a row: two from 8192 elements of 16 bits (4916 of 32) on (us with one / two: 4096 x
// 8192 bf16 102 / 97, 8192 x 5120 109 / 121, 8192 x 4096 79 / 94, in fp32 130 / 147), four where
// half a row does not fit (2048 x 16384 bf16 element by element 483, on two CTAs 124; 1024 x
// 16384 fp32 217, on four 195).  One CTA has room for slots of four inputs and the parameters
// of one group of warps only from 5960 elements of 16 bits on (5664 with fp32 parameters), and
// two would be faster from there: 4096 x 5632 63 / 74, but 4096 x 6144 94 / 77, 4096 x 7168 95 / 90,
// 1133 x 6373 69 / 52, 4096 x 8184 97 / 97 (with fp32 parameters 101 / 114).
int bwd_cluster(int64_t D, int elem)
{
    if (D * (8 * elem + 8) < 24 * 8192)
        return 1;
    const int64_t half = (D / 2 / (16 / elem) + 2) * (16 / elem);
    return half * (8 * elem + 8) <= BWD_BUDGET - 256 && half <= BWD_THREADS * RING_NV * (16 / elem) ? 2 : 4;
}
// Clusters, a multiple of eight where the rows of each have one phase.
int64_t bwd_units(int64_t M, int num_sms, int cluster, bool phased)
{
    const int sms = num_sms < BLOCK_NORM_BWD_BLOCKS ? num_sms : BLOCK_NORM_BWD_BLOCKS;
    if (cluster == 1 || phased)
        return ring_blocks(M, sms / cluster);
    return M < sms / cluster ? M : sms / cluster;
}
// Phased rows with several gate rows take the ring where each phase meets each gate row
// once at least (else their parts would be most of the traffic) and a block has more than
// one row, or a row is too long for its registers (us by blocks, element by element, / in
// rings, four gates of bf16: 100 x 1027 12.9 / 13.3, 100 x 4097 38 / 41, 2048 x 65 30 / 24, 1020 x 4097
// 195 / 62, 256 x 16383 120 / 87).
bool bwd_phased_gates(int64_t M, int64_t D, int elem, int64_t gate_rows)
{
    const int64_t vec = 16 / elem;
    return gate_rows > 1 && D % vec != 0 && D >= PHASED_MIN_D && M / gate_rows >= vec && (M > RMS_BWD_BLOCKS || D > 8192);
}
// Groups of a block at most.
int64_t bwd_groups(int64_t D, int elem, int cluster)
{
    int64_t packs;
    const int64_t gt = bwd_group_threads(D, elem, false, cluster, &packs);
    return gt > BWD_THREADS ? 1 : BWD_THREADS / gt;
}

template <class T, class W>
cudaError_t launch_block_bwd_tw(BlockNormBwdParams p, Rows rows, void *dpost, void *dpre, void *dgate, int num_sms,
                                cudaStream_t s)
{
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    const int inputs = (p.pre ? 2 : 0) + (p.x ? 1 : 0) + (p.dh ? 1 : 0);
    const bool several = p.gate_rows > 1;
    int blocks = static_cast<int>(p.M < RMS_BWD_BLOCKS ? p.M : RMS_BWD_BLOCKS);
    cudaError_t e = cudaSuccess;
    BwdPlan r;
    p.residues = 1;
    if (several && rows == ROWS_PHASED && !bwd_phased_gates(p.M, p.D, sizeof(T), p.gate_rows))
        rows = ROWS_ANY;
    const bool phased = rows == ROWS_PHASED;
    const int cluster = bwd_cluster(p.D, sizeof(T));
    const int64_t units = num_sms >= 64 ? bwd_units(p.M, num_sms, cluster, phased) : 0;
    // (rows of more than 16 columns for each of 512 threads: always)
    const bool ring = units > 0 && (use_ring(rows, p.M, p.D) || (rows != ROWS_ANY && p.D > 8192));
    if (ring && plan_bwd(&r, phased, p.D, sizeof(T), p.pre ? sizeof(W) : 0, p.post || p.gate, several, inputs, cluster,
                         several ? p.M / units : BWD_WARPS)) {  // (with several gate rows every lane has a row)
        p.residues = several && phased ? V : 1;
        blocks = static_cast<int>(units);
        p.lanes = units / p.residues * r.groups;
        e = phased ? launch_block_bwd_ring<T, W, true>(p, r, blocks, s)
                   : launch_block_bwd_ring<T, W, false>(p, r, blocks, s);
    } else {
        p.lanes = blocks;
        if (!(rows == ROWS_VEC ? launch_block_bwd_regs<T, W, V>(p, blocks, s, &e)
                               : launch_block_bwd_regs<T, W, 1>(p, blocks, s, &e)))
            e = launch_overlapped(k_block_norm_bwd_long<T, W>, dim3(blocks), dim3(1024), 0, 1, s, p);
    }
    if (e != cudaSuccess || (!dpost && !dpre && !dgate))
        return e;
    int64_t jobs = 2;
    if (several) {
        const int64_t sets = many_lanes(p.lanes * p.residues, p.gate_rows) ? p.gate_rows : (p.gate_rows + SUM_ROWS - 1) / SUM_ROWS;
        jobs = 1 + (sets < 65534 ? sets : 65534);
    }
    const auto sums = p.residues > 1 ? k_block_norm_sums<T, W, V> : k_block_norm_sums<T, W, 1>;
    return launch_overlapped(sums, dim3(static_cast<unsigned>((p.D + 31) / 32), static_cast<unsigned>(jobs)),
                             dim3(32, SUM_ROWS), 0, 1, s, p, blocks, static_cast<W *>(dpost), static_cast<W *>(dpre), dgate);
}

}  // namespace

BlockNormScratch block_norm_bwd_scratch(int64_t M, int64_t D, int dtype, int64_t gate_rows)
{
    // a row for as many lanes as the ring kernel can have, or for every block
    const int elem = dtype == 2 ? 4 : 2, cluster = bwd_cluster(D, elem);
    const int64_t most = bwd_units(M, BLOCK_NORM_BWD_BLOCKS, cluster, false) * bwd_groups(D, elem, cluster);
    const int64_t ring = M < most ? M : most;
    const int64_t blocks = M < RMS_BWD_BLOCKS ? (M + 7) / 8 * 8 : RMS_BWD_BLOCKS;  // (304 is a multiple of eight)
    const int64_t lanes = ring > blocks ? ring : blocks;
    const int64_t residues = bwd_phased_gates(M, D, elem, gate_rows) ? 16 / elem : 1;
    const auto floats = [](int64_t n) { return (n + 3) / 4 * 4; };
    return {floats(lanes * D), floats((lanes + gate_rows * residues) * D), (D + 31) / 32};
}

cudaError_t launch_block_norm_bwd(const BlockNormBwdParams &p, void *dpost, void *dpre, void *dgate, int dtype, int wdtype,
                                  int num_sms, cudaStream_t s)
{
    const int64_t v = dtype == 2 ? 4 : 8;
    const bool based = al16(p.dy) && al16(p.x) && al16(p.h) && al16(p.post) && al16(p.pre) && al16(p.gate) && al16(p.dh) &&
                       al16(p.dx) && al16(p.dres) && al16(p.part_pre) && al16(p.part_sum);
    const Rows rows = !based ? ROWS_ANY : p.D % v == 0 ? ROWS_VEC : p.D >= PHASED_MIN_D ? ROWS_PHASED : ROWS_ANY;
    if (dtype == 0)
        return wdtype == 0 ? launch_block_bwd_tw<__nv_bfloat16, __nv_bfloat16>(p, rows, dpost, dpre, dgate, num_sms, s)
                           : launch_block_bwd_tw<__nv_bfloat16, float>(p, rows, dpost, dpre, dgate, num_sms, s);
    if (dtype == 1)
        return wdtype == 1 ? launch_block_bwd_tw<__half, __half>(p, rows, dpost, dpre, dgate, num_sms, s)
                           : launch_block_bwd_tw<__half, float>(p, rows, dpost, dpre, dgate, num_sms, s);
    return launch_block_bwd_tw<float, float>(p, rows, dpost, dpre, dgate, num_sms, s);
}

}  // namespace lf
