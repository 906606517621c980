// Group norm with an activation, channels last: the groups are the heads, and the
// statistics run over one head's channels of one token,
//
//     xh = (x - mean) rstd,  n = xh w + b,   y = n act(gate)   (act(n) without a gate)
//
// with mean = 0 in the RMS form.  Backward, with f = act:
//
//     dn = dy f(gate)  (dy f'(n) without),  dgate = dy n f'(gate),  dxh = dn w,
//     dx = rstd (dxh - xh mean(dxh xh) - mean(dxh)),  dw = sum dn xh,  db = sum dn
//
// (the last mean only when centred).  x, gate, dy are read once and the row stays in
// registers between the statistics and the result; the mean is subtracted before the
// squares are summed, so a large offset loses no digits.
//
// A group of LPG lanes (a "slot") holds one row, NV vectors of VEC elements a lane.  Slot s of
// the grid keeps head s % G and takes tokens s / G, s / G + R, ..: its weights stay in
// registers, and so do its sums for the weight gradients, which each CTA (or each slot, when
// there are more heads than slots in a CTA) leaves in the workspace for a second kernel to add
// in a fixed order: the gradients are the same on every run.  Bound by memory: forward 65536 x 32 x 128
// bf16, 1.61 GB, 267 us (6.0 TB/s); backward 20011 x 16 x 128 fp32, 0.82 GB, 150 us (5.5 TB/s, 4 of them
// the second kernel), 65536 x 32 x 128 bf16, 2.68 GB, 527 us (5.1 TB/s: the same arithmetic for half the bytes).
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {

constexpr int kNormThreads = 256;
constexpr int kNormMaxD = 512;      // at most 16 elements a lane

// VEC consecutive elements: one access, as they are stored (Raw) and as fp32.
template <typename T, int VEC> struct Row;
template <> struct Row<float, 4> {
    using Raw = float4;
    static __device__ __forceinline__ Raw load(const float* p) { return __ldcs(reinterpret_cast<const float4*>(p)); }
    static __device__ __forceinline__ void unpack(const Raw& x, float* v) {
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    }
    static __device__ __forceinline__ void store(float* p, const float* v) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    }
};
struct RowBf16 {
    static __device__ __forceinline__ void two(uint32_t u, float* v) {
        v[0] = __uint_as_float(u << 16);
        v[1] = __uint_as_float(u & 0xffff0000u);
    }
    static __device__ __forceinline__ uint32_t pack(const float* v) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[0], v[1]);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
template <> struct Row<__nv_bfloat16, 8> : RowBf16 {
    using Raw = uint4;
    static __device__ __forceinline__ Raw load(const __nv_bfloat16* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }
    static __device__ __forceinline__ void unpack(const Raw& u, float* v) {
        two(u.x, v); two(u.y, v + 2); two(u.z, v + 4); two(u.w, v + 6);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) {
        __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack(v), pack(v + 2), pack(v + 4), pack(v + 6)));
    }
};
template <> struct Row<__nv_bfloat16, 4> : RowBf16 {
    using Raw = uint2;
    static __device__ __forceinline__ Raw load(const __nv_bfloat16* p) { return __ldcs(reinterpret_cast<const uint2*>(p)); }
    static __device__ __forceinline__ void unpack(const Raw& u, float* v) { two(u.x, v); two(u.y, v + 2); }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) {
        __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack(v), pack(v + 2)));
    }
};
template <typename T> struct Row<T, 1> {
    using Raw = T;
    static __device__ __forceinline__ Raw load(const T* p) { return *p; }
    static __device__ __forceinline__ void unpack(const Raw& x, float* v) { v[0] = IO<T>::load(&x, 0); }
    static __device__ __forceinline__ void store(T* p, const float* v) { IO<T>::store(p, 0, v[0]); }
};

// The lane's vectors of one row of a tensor; what lies past the row's end, or in no row, is zero.
template <typename T, int VEC, int NV, int LPG>
__device__ __forceinline__ void load_row(const T* row, bool on, int lane, int d, typename Row<T, VEC>::Raw (&r)[NV])
{
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * LPG + lane) * VEC;
        if (on && c < d) r[v] = Row<T, VEC>::load(row + c);
        else r[v] = typename Row<T, VEC>::Raw{};
    }
}

// Sum over the LPG lanes of a slot; every lane gets it.
template <int LPG>
__device__ __forceinline__ float slot_sum(float v)
{
#pragma unroll
    for (int o = LPG / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The reciprocal is the hardware's (2 half steps of 2^-24) in place of a division of ten instructions.
// fp32 I/O: with expf, within 6 half steps.  bf16 I/O: the exponential's argument is rounded once more,
// |z| + 4 half steps, far below the output's own 2^-8; 4 instructions for about 20, which is what bounded
// the forward (65536 x 32 x 128: 411 -> 267 us).  A sigmoid below 2^-126 is 0.
__device__ __forceinline__ float reciprocal(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
template <typename T> __device__ __forceinline__ float exponential(float z);
template <> __device__ __forceinline__ float exponential<float>(float z) { return expf(z); }
template <> __device__ __forceinline__ float exponential<__nv_bfloat16>(float z)
{
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * 1.4426950408889634f));
    return e;
}
template <typename T> __device__ __forceinline__ float sigmoid(float z) { return reciprocal(1.f + exponential<T>(-z)); }
// The sigmoid s and 1 - s, which the slopes need, each to its own last digits: with e = exp(-|z|), which
// cannot overflow, they are 1 / (1 + e) and e / (1 + e).  (1 - s from a rounded s is 17 % off at z = 15.)
template <typename T> __device__ __forceinline__ void sigmoids(float z, float& s, float& rest)
{
    const float e = exponential<T>(-fabsf(z)), large = reciprocal(1.f + e), small = e * large;
    s = z >= 0.f ? large : small;
    rest = z >= 0.f ? small : large;
}

// Which rows a slot takes.
struct SlotPlan {
    int64_t M, G;
    int64_t stride;       // tokens between a slot's rows
    int64_t slots;        // slots in use over the whole grid, a multiple of G
    int per_cta;          // slots in use of a CTA
    int d;
};

template <typename T, int VEC, int NV, int LPG>
__global__ void __launch_bounds__(kNormThreads)
group_norm_fwd_kernel(const T* __restrict__ x, const T* __restrict__ gate,
                      const float* __restrict__ weight, const float* __restrict__ bias,
                      T* __restrict__ out, SlotPlan p, int per_group, int center, float eps, int act)
{
    const int in_cta = threadIdx.x / LPG, lane = threadIdx.x % LPG;
    const int64_t slot = (int64_t)blockIdx.x * p.per_cta + in_cta;
    const bool used = in_cta < p.per_cta && slot < p.slots;
    const int64_t g = used ? slot % p.G : 0;
    const float inv_d = 1.f / (float)p.d;
    float w[NV][VEC], b[NV][VEC];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int c = (v * LPG + lane) * VEC + e;
            const bool in = c < p.d;
            w[v][e] = in && weight ? weight[(per_group ? g * p.d : 0) + c] : 1.f;
            b[v][e] = in && bias ? bias[(per_group ? g * p.d : 0) + c] : 0.f;
        }
    // every lane of a warp makes the same number of rounds (the shuffles need all of them); the next
    // row is on its way while this one is worked on
    typename Row<T, VEC>::Raw next_x[NV], next_z[NV] = {};
    int64_t m = used ? slot / p.G : p.M, at = (m * p.G + g) * p.d;
    const int64_t pitch = p.stride * p.G * p.d;
    load_row<T, VEC, NV, LPG>(x + at, m < p.M, lane, p.d, next_x);
    if (gate) load_row<T, VEC, NV, LPG>(gate + at, m < p.M, lane, p.d, next_z);
    for (; __any_sync(0xffffffffu, m < p.M); m += p.stride, at += pitch) {
        const bool on = m < p.M;
        float r[NV][VEC], z[NV][VEC];
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            Row<T, VEC>::unpack(next_x[v], r[v]);
            Row<T, VEC>::unpack(next_z[v], z[v]);
        }
        load_row<T, VEC, NV, LPG>(x + at + pitch, m + p.stride < p.M, lane, p.d, next_x);
        if (gate) load_row<T, VEC, NV, LPG>(gate + at + pitch, m + p.stride < p.M, lane, p.d, next_z);
        if (center) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < VEC; ++e) sum += r[v][e];
            const float mean = slot_sum<LPG>(sum) * inv_d;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < VEC; ++e) r[v][e] = (v * LPG + lane) * VEC + e < p.d ? r[v][e] - mean : 0.f;
        }
        float sq = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < VEC; ++e) sq += r[v][e] * r[v][e];
        const float rstd = rsqrtf(slot_sum<LPG>(sq) * inv_d + eps);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * LPG + lane) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) r[v][e] = r[v][e] * rstd * w[v][e] + b[v][e];
            if (act != KDA_ACT_NONE)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float t = gate ? z[v][e] : r[v][e], s = sigmoid<T>(t);
                    z[v][e] = act == KDA_ACT_SILU ? t * s : s;
                }
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                r[v][e] = gate ? r[v][e] * z[v][e] : act != KDA_ACT_NONE ? z[v][e] : r[v][e];
            if (on && c < p.d) Row<T, VEC>::store(out + at + c, r[v]);
        }
    }
}

template <typename T, int VEC, int NV, int LPG>
__global__ void __launch_bounds__(kNormThreads)
group_norm_bwd_kernel(const T* __restrict__ x, const T* __restrict__ gate,
                      const float* __restrict__ weight, const float* __restrict__ bias,
                      const T* __restrict__ dout, T* __restrict__ dx, T* __restrict__ dgate,
                      float* __restrict__ wpart, float* __restrict__ bpart, SlotPlan p, int per_group,
                      int center, float eps, int act)
{
    __shared__ float red[kNormThreads * NV * VEC];
    const int in_cta = threadIdx.x / LPG, lane = threadIdx.x % LPG;
    const int64_t slot = (int64_t)blockIdx.x * p.per_cta + in_cta;
    const bool used = in_cta < p.per_cta && slot < p.slots;
    const int64_t g = used ? slot % p.G : 0;
    const float inv_d = 1.f / (float)p.d;
    float w[NV][VEC], b[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int c = (v * LPG + lane) * VEC + e;
            const bool in = c < p.d;
            w[v][e] = in && weight ? weight[(per_group ? g * p.d : 0) + c] : 1.f;
            b[v][e] = in && bias ? bias[(per_group ? g * p.d : 0) + c] : 0.f;
            dw[v][e] = 0.f;
            db[v][e] = 0.f;
        }
    typename Row<T, VEC>::Raw next_x[NV], next_z[NV] = {}, next_y[NV];
    int64_t m = used ? slot / p.G : p.M, at = (m * p.G + g) * p.d;
    const int64_t pitch = p.stride * p.G * p.d;
    const auto fetch = [&](int64_t from, bool on) {
        load_row<T, VEC, NV, LPG>(x + from, on, lane, p.d, next_x);
        if (gate) load_row<T, VEC, NV, LPG>(gate + from, on, lane, p.d, next_z);
        load_row<T, VEC, NV, LPG>(dout + from, on, lane, p.d, next_y);
    };
    fetch(at, m < p.M);
    for (; __any_sync(0xffffffffu, m < p.M); m += p.stride, at += pitch) {
        const bool on = m < p.M;
        float r[NV][VEC], z[NV][VEC], y[NV][VEC];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            Row<T, VEC>::unpack(next_x[v], r[v]);
            Row<T, VEC>::unpack(next_z[v], z[v]);
            Row<T, VEC>::unpack(next_y[v], y[v]);
        }
        fetch(at + pitch, m + p.stride < p.M);
        if (center) {
            float sum = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < VEC; ++e) sum += r[v][e];
            const float mean = slot_sum<LPG>(sum) * inv_d;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < VEC; ++e) r[v][e] = (v * LPG + lane) * VEC + e < p.d ? r[v][e] - mean : 0.f;
        }
        float sq = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < VEC; ++e) sq += r[v][e] * r[v][e];
        const float rstd = rsqrtf(slot_sum<LPG>(sq) * inv_d + eps);
        float s1 = 0.f, s2 = 0.f;                // sums of dxh xh and dxh
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float xh = r[v][e] * rstd, n = xh * w[v][e] + b[v][e];
                const float t = gate ? z[v][e] : n;
                float f = t, df = 1.f;
                if (act != KDA_ACT_NONE) {
                    float s, rest;
                    sigmoids<T>(t, s, rest);
                    f = act == KDA_ACT_SILU ? t * s : s;
                    df = act == KDA_ACT_SILU ? s + f * rest : s * rest;
                }
                const float dn = y[v][e] * (gate ? f : df);
                z[v][e] = y[v][e] * n * df;      // dgate
                dw[v][e] += dn * xh;
                db[v][e] += dn;
                const float dxh = dn * w[v][e];
                r[v][e] = xh;
                y[v][e] = dxh;
                s1 += dxh * xh;
                s2 += dxh;
            }
        s1 = slot_sum<LPG>(s1) * inv_d;
        s2 = center ? slot_sum<LPG>(s2) * inv_d : 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * LPG + lane) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) r[v][e] = rstd * (y[v][e] - r[v][e] * s1 - s2);
            if (on && c < p.d) {
                Row<T, VEC>::store(dx + at + c, r[v]);
                if (gate) Row<T, VEC>::store(dgate + at + c, z[v]);
            }
        }
    }
    // Partial sums.  Heads of weights (per_group) that fit a CTA, and shared weights: the CTA's
    // slots are added first; otherwise every slot leaves its own row.
    const int64_t heads = per_group ? p.G : 1;
    const bool in_cta_sum = heads <= p.per_cta;
    for (int pass = 0; pass < 2; ++pass) {
        float* part = pass == 0 ? wpart : bpart;
        if (part == nullptr) continue;
        float(&acc)[NV][VEC] = pass == 0 ? dw : db;
        if (!in_cta_sum) {
            if (used)
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const int c = (v * LPG + lane) * VEC + e;
                        if (c < p.d) part[slot * p.d + c] = acc[v][e];
                    }
            continue;
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                red[(in_cta * NV * LPG + v * LPG + lane) * VEC + e] = used ? acc[v][e] : 0.f;
        __syncthreads();
        constexpr int kRow = NV * LPG * VEC;     // channels a slot has room for
        for (int i = threadIdx.x; i < heads * p.d; i += kNormThreads) {
            const int h = i / p.d, c = i - h * p.d;
            float s = 0.f;
            for (int k = h; k < p.per_cta; k += (int)heads) s += red[k * kRow + c];
            part[(int64_t)blockIdx.x * heads * p.d + i] = s;
        }
    }
}

// dst[c] = sum over rows r of part[r][c]: 32 columns a CTA, 32 row groups, added in a fixed order.
__global__ void __launch_bounds__(1024)
group_norm_wgrad_kernel(const float* __restrict__ wpart, const float* __restrict__ bpart,
                        float* __restrict__ dweight, float* __restrict__ dbias, int64_t rows, int64_t cols)
{
    __shared__ float red[32][33];
    const float* part = blockIdx.y == 0 ? wpart : bpart;
    float* dst = blockIdx.y == 0 ? dweight : dbias;
    if (dst == nullptr) return;
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * 32 + tx;
    float s = 0.f;
    if (c < cols)
#pragma unroll 8
        for (int64_t r = ty; r < rows; r += 32) s += part[r * cols + c];
    red[ty][tx] = s;
    __syncthreads();
    // warp ty adds up column ty
    s = red[tx][ty];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (tx == 0 && (int64_t)blockIdx.x * 32 + ty < cols) dst[(int64_t)blockIdx.x * 32 + ty] = s;
}

namespace {

// CTAs of the kernel that an SM holds at once: the grid is one wave of them, so that all slots work from
// the first row to the last.
template <typename Kernel> int64_t resident(Kernel kernel)
{
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kNormThreads, 0) != cudaSuccess || n < 1) n = 1;
    return n * device_sm_count();
}

SlotPlan plan_slots(const GroupNormArgs& a, int lpg, int64_t ctas_most, int& grid)
{
    const int64_t room = kNormThreads / lpg;
    SlotPlan p;
    p.M = a.M; p.G = a.G; p.d = (int)a.d;
    p.per_cta = (int)(a.G <= room ? room / a.G * a.G : room);
    const int64_t rows = a.M * a.G;
    int64_t n = (rows + p.per_cta - 1) / p.per_cta;
    if (n > ctas_most) n = ctas_most;
    const int64_t need = (a.G + p.per_cta - 1) / p.per_cta;    // at least one slot for every head
    if (n < need) n = need;
    grid = (int)n;
    p.slots = n * p.per_cta / a.G * a.G;
    p.stride = p.slots / a.G;
    return p;
}

template <typename T, int VEC, int NV, int LPG>
cudaError_t norm_fwd(const GroupNormArgs& a, cudaStream_t st)
{
    int grid;
    static const int64_t most = resident(group_norm_fwd_kernel<T, VEC, NV, LPG>);
    const SlotPlan p = plan_slots(a, LPG, most, grid);
    LaunchScope scope(st, K_GNORM_FWD);
    group_norm_fwd_kernel<T, VEC, NV, LPG><<<grid, kNormThreads, 0, st>>>(
        (const T*)a.x, (const T*)a.gate, a.weight, a.bias, (T*)a.out, p, a.per_group, a.center, a.eps, a.act);
    return cudaGetLastError();
}

template <typename T, int VEC, int NV, int LPG>
cudaError_t norm_bwd(const GroupNormArgs& a, cudaStream_t st)
{
    int grid;
    static const int64_t most = resident(group_norm_bwd_kernel<T, VEC, NV, LPG>);
    const SlotPlan p = plan_slots(a, LPG, most, grid);
    const int64_t heads = a.per_group ? a.G : 1;
    const int64_t rows = heads <= p.per_cta ? grid : p.slots / a.G, cols = heads * a.d;
    StreamBuffer buf;
    const int64_t one = a.dweight || a.dbias ? rows * cols : 0;
    if (one > 0) {
        const cudaError_t e = buf.alloc((size_t)(2 * one * 4), st);
        if (e != cudaSuccess) return e;
    }
    float* wpart = a.dweight ? (float*)buf.ptr : nullptr;
    float* bpart = a.dbias ? (float*)buf.ptr + one : nullptr;
    {
        LaunchScope scope(st, K_GNORM_BWD);
        group_norm_bwd_kernel<T, VEC, NV, LPG><<<grid, kNormThreads, 0, st>>>(
            (const T*)a.x, (const T*)a.gate, a.weight, a.bias, (const T*)a.dout, (T*)a.dx, (T*)a.dgate, wpart,
            bpart, p, a.per_group, a.center, a.eps, a.act);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (one == 0) return cudaSuccess;
    LaunchScope scope(st, K_GNORM_WGRAD);
    group_norm_wgrad_kernel<<<dim3((unsigned)((cols + 31) / 32), 2), 1024, 0, st>>>(wpart, bpart, a.dweight, a.dbias,
                                                                                  rows, cols);
    return cudaGetLastError();
}

// F(NV, LPG) for rows of `vecs` vectors of VEC elements, at least LEAST vectors a lane.  The forward takes two
// where a vector is 8 bytes (20000 x 13 x 100 bf16: 50 -> 45 us); the backward has enough in work
// with one (30000 x 10 x 100 bf16: 108 us, 114 with two).
#define KDA_NORM_BY_VECS(F, T, VEC, LEAST)                                      \
    do {                                                                       \
        constexpr int NV = VEC * sizeof(T) == 16 ? 1 : LEAST;                   \
        if (vecs <= 8 * NV) return F<T, VEC, NV, 8>(a, st);                     \
        if (vecs <= 16 * NV) return F<T, VEC, NV, 16>(a, st);                   \
        if (vecs <= 32 * NV) return F<T, VEC, NV, 32>(a, st);                   \
        if (VEC == 8 || vecs <= 64) return F<T, VEC, 2, 32>(a, st);             \
        return F<T, VEC, VEC == 8 ? 2 : 4, 32>(a, st);                          \
    } while (0)
// ceil(d / 32) elements a lane, for widths that no vector divides
#define KDA_NORM_SCALAR(F, T)                                                   \
    do {                                                                       \
        if (a.d <= 128) return F<T, 1, 4, 32>(a, st);                           \
        return F<T, 1, 16, 32>(a, st);                                         \
    } while (0)

}  // namespace

// Widest access that the width allows: every row then starts on its boundary.
cudaError_t launch_group_norm_fwd(const GroupNormArgs& a, cudaStream_t st)
{
    if (a.io == KDA_IO_F32) {
        const int64_t vecs = a.d / 4;
        if (a.d % 4 == 0) KDA_NORM_BY_VECS(norm_fwd, float, 4, 2);
        KDA_NORM_SCALAR(norm_fwd, float);
    }
    if (a.d % 8 == 0) {
        const int64_t vecs = a.d / 8;
        KDA_NORM_BY_VECS(norm_fwd, __nv_bfloat16, 8, 2);
    }
    const int64_t vecs = a.d / 4;
    if (a.d % 4 == 0) KDA_NORM_BY_VECS(norm_fwd, __nv_bfloat16, 4, 2);
    KDA_NORM_SCALAR(norm_fwd, __nv_bfloat16);
}

cudaError_t launch_group_norm_bwd(const GroupNormArgs& a, cudaStream_t st)
{
    if (a.M == 0) {
        const size_t n = (size_t)((a.per_group ? a.G : 1) * a.d) * 4;
        cudaError_t e = a.dweight ? cudaMemsetAsync(a.dweight, 0, n, st) : cudaSuccess;
        if (e == cudaSuccess && a.dbias) e = cudaMemsetAsync(a.dbias, 0, n, st);
        return e;
    }
    if (a.io == KDA_IO_F32) {
        const int64_t vecs = a.d / 4;
        if (a.d % 4 == 0) KDA_NORM_BY_VECS(norm_bwd, float, 4, 1);
        KDA_NORM_SCALAR(norm_bwd, float);
    }
    if (a.d % 8 == 0) {
        const int64_t vecs = a.d / 8;
        KDA_NORM_BY_VECS(norm_bwd, __nv_bfloat16, 8, 1);
    }
    const int64_t vecs = a.d / 4;
    if (a.d % 4 == 0) KDA_NORM_BY_VECS(norm_bwd, __nv_bfloat16, 4, 1);
    KDA_NORM_SCALAR(norm_bwd, __nv_bfloat16);
}

}  // namespace kda

using namespace kda;

namespace {

kda_status_t norm_check(int64_t M, int64_t G, int64_t d, float eps, kda_activation_t act, kda_io_dtype_t io)
{
    if (M < 0 || G < 0 || d < 1) return KDA_ERR_INVALID_ARG;
    if (!(eps > 0.f) || !(eps < 1e30f)) return KDA_ERR_INVALID_ARG;
    if (act != KDA_ACT_NONE && act != KDA_ACT_SIGMOID && act != KDA_ACT_SILU) return KDA_ERR_INVALID_ARG;
    if (io != KDA_IO_F32 && io != KDA_IO_BF16) return KDA_ERR_UNSUPPORTED;
    if (d > kNormMaxD || G > 65535 || M > (int64_t(1) << 40)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status_t kda_group_norm_fwd(const void* x, const void* gate, const float* weight,
                                const float* bias, void* out, int64_t M, int64_t G, int64_t d,
                                int per_group, int center, float eps, kda_activation_t act,
                                kda_io_dtype_t io_dtype, cudaStream_t stream)
{
    const kda_status_t s = norm_check(M, G, d, eps, act, io_dtype);
    if (s != KDA_OK) return s;
    if (M == 0 || G == 0) return KDA_OK;
    const int64_t n = M * G * d * (io_dtype == KDA_IO_F32 ? 4 : 2), nw = (per_group ? G : 1) * d * 4;
    if (!tensor_ok(x) || !tensor_ok(out) || !optional_ok(gate)) return KDA_ERR_INVALID_ARG;
    if (!optional_ok(weight) || !optional_ok(bias)) return KDA_ERR_INVALID_ARG;
    if (overlap(out, n, x, n) || overlap(out, n, gate, n) || overlap(out, n, weight, nw) ||
        overlap(out, n, bias, nw))
        return KDA_ERR_INVALID_ARG;
    GroupNormArgs a = {};
    a.x = x; a.gate = gate; a.weight = weight; a.bias = bias; a.out = out;
    a.M = M; a.G = G; a.d = d; a.per_group = per_group != 0; a.center = center != 0;
    a.eps = eps; a.act = act; a.io = io_dtype;
    return finish_call(launch_group_norm_fwd(a, stream), stream);
}

kda_status_t kda_group_norm_bwd(const void* x, const void* gate, const float* weight,
                                const float* bias, const void* dout, void* dx, void* dgate,
                                float* dweight, float* dbias, int64_t M, int64_t G, int64_t d,
                                int per_group, int center, float eps, kda_activation_t act,
                                kda_io_dtype_t io_dtype, cudaStream_t stream)
{
    const kda_status_t s = norm_check(M, G, d, eps, act, io_dtype);
    if (s != KDA_OK) return s;
    if ((gate == nullptr) != (dgate == nullptr) && M > 0 && G > 0) return KDA_ERR_INVALID_ARG;
    if (!optional_ok(weight) || !optional_ok(bias) || !optional_ok(dweight) || !optional_ok(dbias))
        return KDA_ERR_INVALID_ARG;
    if (G == 0) return KDA_OK;
    const int64_t n = M * G * d * (io_dtype == KDA_IO_F32 ? 4 : 2), nw = (per_group ? G : 1) * d * 4;
    if (M > 0 && (!tensor_ok(x) || !tensor_ok(dout) || !tensor_ok(dx) || !optional_ok(gate) || !optional_ok(dgate)))
        return KDA_ERR_INVALID_ARG;
    const struct { const void* p; int64_t n; } in[] = {{x, n}, {gate, n}, {dout, n}, {weight, nw}, {bias, nw}},
                                               res[] = {{dx, n}, {dgate, n}, {dweight, nw}, {dbias, nw}};
    for (int i = 0; i < 4; ++i) {
        for (const auto& q : in)
            if (overlap(res[i].p, res[i].n, q.p, q.n)) return KDA_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(res[i].p, res[i].n, res[j].p, res[j].n)) return KDA_ERR_INVALID_ARG;
    }
    GroupNormArgs a = {};
    a.x = x; a.gate = gate; a.weight = weight; a.bias = bias; a.dout = dout; a.dx = dx; a.dgate = dgate;
    a.dweight = dweight; a.dbias = dbias; a.M = M; a.G = G; a.d = d;
    a.per_group = per_group != 0; a.center = center != 0; a.eps = eps; a.act = act; a.io = io_dtype;
    return finish_call(launch_group_norm_bwd(a, stream), stream);
}

}  // extern "C"
