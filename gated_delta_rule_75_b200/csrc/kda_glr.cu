// Gated linear recurrence, h_t = exp(log_a_t) h_{t-1} + x_t per channel: the
// elementwise sibling of the delta rule (a vector state, the same per-channel
// decay), its gradients and its decode step.
//
// Scan.  A run of tokens maps the state it enters with affinely, h -> A h + B, and
// runs compose: the token axis is cut into tiles of kTile tokens, a tile into eight
// runs of kSteps tokens, one per warp, each lane owning V channels of its run in
// registers.  One pass over memory:
//   1. every warp loads its run and folds it into (A, B); the tile's (A, B) is
//      published in the workspace;
//   2. the state entering the tile is put together from what earlier tiles
//      published, in an order that does not depend on timing: the state entering its
//      group of kGroup tiles, then the (A, B) of the group's earlier tiles one by
//      one (the last tile of a group publishes the next group's entry state);
//   3. every warp walks its run again from its entry state and writes the outputs.
// So a value is the same on every run, and the chain of waits is one hop per
// kGroup * kTile tokens.  Tiles are taken by a ticket, tokens first: whatever a
// tile waits for was taken earlier and never waits for it, so every wait ends (and
// is bounded all the same).  Sequences: a token that begins one replaces the state
// by h0 (A = 0, B = h0), whatever came before it.
//
// Backward.  With c_t = exp(log_a_t) g_t, g_t = dout_t + c_{t+1}: the same scan over
// tiles from the last to the first, replaced by dhT at a sequence's last token.
// dlog_a_t = c_t h_{t-1} needs the forward states too; they are walked again inside
// the tile from its kept entry state (starts), so the pass reads x, log_a, dout and
// writes dx, dlog_a once.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {

constexpr int kTile = KDA_GLR_TILE;     // tokens of a tile
constexpr int kWarps = 8;
constexpr int kSteps = kTile / kWarps;  // tokens of a warp
constexpr int kGroup = 16;              // tiles between published entry states
constexpr int kPolls = 1 << 21;         // about two seconds of polling
static_assert(kGroup <= 32, "one polling lane per tile of a group");

// V channels of one token as they are stored, and as fp32.
template <typename T, int V> struct Raw;
template <int V> struct Raw<float, V> {
    float v[V];
    __device__ __forceinline__ void load(const float* p) {
        if constexpr (V == 4) {
            const float4 x = __ldcs(reinterpret_cast<const float4*>(p));
            v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        } else if constexpr (V == 2) {
            const float2 x = __ldcs(reinterpret_cast<const float2*>(p));
            v[0] = x.x; v[1] = x.y;
        } else {
            v[0] = __ldcs(p);
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = 0.f;
    }
    __device__ __forceinline__ float get(int e) const { return v[e]; }
    static __device__ __forceinline__ void store(float* p, const float* v) {
        if constexpr (V == 4) __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
        else if constexpr (V == 2) __stcs(reinterpret_cast<float2*>(p), make_float2(v[0], v[1]));
        else __stcs(p, v[0]);
    }
};
template <int V> struct Raw<__nv_bfloat16, V> {
    uint32_t u[(V + 1) / 2];
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        if constexpr (V == 4) {
            const uint2 x = __ldcs(reinterpret_cast<const uint2*>(p));
            u[0] = x.x; u[1] = x.y;
        } else if constexpr (V == 2) {
            u[0] = __ldcs(reinterpret_cast<const unsigned int*>(p));
        } else {
            u[0] = __ldcs(reinterpret_cast<const unsigned short*>(p));
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int e = 0; e < (V + 1) / 2; ++e) u[e] = 0;
    }
    __device__ __forceinline__ float get(int e) const {
        return __uint_as_float(e & 1 ? u[e / 2] & 0xffff0000u : u[e / 2] << 16);
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) {
        if constexpr (V == 4)
            __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack(v[0], v[1]), pack(v[2], v[3])));
        else if constexpr (V == 2)
            __stcs(reinterpret_cast<unsigned int*>(p), pack(v[0], v[1]));
        else
            *p = __float2bfloat16_rn(v[0]);
    }
};

// Workspace of a call with more than one tile: a ticket, a flag per (tile, column) and the
// groups' entry states, all zeroed first, then the published (A, B).
// A column is one block of 32 V channels of one row of the token axis; tiles and
// groups are numbered in the order of the scan (from the end in the backward).
struct ScanWork {
    int* ticket;
    int* tile_flag;    // [tiles][cols]
    unsigned long long* entry;   // [groups][cols][32 V]: value, and 1 in the high word once it is there
    float* tile_ab;    // [tiles][cols][2][32 V]
    int64_t cols, tiles;
};

__device__ __forceinline__ int load_acquire(const int* p)
{
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void store_release(int* p, int v)
{
    asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

__device__ __forceinline__ unsigned long long load_relaxed(const unsigned long long* p)
{
    unsigned long long v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void store_relaxed(unsigned long long* p, unsigned long long v)
{
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
template <int V> __device__ __forceinline__ void load_cg(const float* p, float (&v)[V])
{
    if constexpr (V == 4) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(p));
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = __ldcg(p + e);
    }
}

// The state behind a run (A, B) entered with h.  A negative A (-0 too): the run holds the
// border of a sequence and nothing crosses it.
__device__ __forceinline__ float leave(float A, float B, float h)
{
    return __float_as_int(A) < 0 ? B : A * h + B;
}
// A of a run followed by a run with A = a.
__device__ __forceinline__ float chain(float A, float a) { return __float_as_int(a) < 0 ? a : A * a; }

// Which sequence begins, and which ends, at each token of a tile (-1: none).
struct Marks {
    int first[kTile], last[kTile];
};

// Row of h0 / hT / the pool that holds sequence n's state; -1: none.
__device__ __forceinline__ int64_t glr_row(const GlrArgs& a, int64_t n, bool report)
{
    if (a.slots == nullptr) return n;
    const int64_t s = a.slots[n];
    if (s >= a.P && report && a.err) atomicOr(a.err, kErrSeqlens);
    return s >= 0 && s < a.P ? s : -1;
}

// Marks of tokens [t0, t0 + kTile) of row b.  All threads call it; the marks are
// there after the next __syncthreads.  Offsets are found by a search of the whole
// warp; an array that is not sorted gives some offsets, never an index outside
// the tile or the arrays.
__device__ __forceinline__ void find_marks(const GlrArgs& a, int64_t b, int64_t t0, Marks& m)
{
    const int tid = threadIdx.x;
    if (a.cu == nullptr) {
        if (tid < kTile) {
            m.first[tid] = t0 + tid == 0 ? (int)b : -1;
            m.last[tid] = t0 + tid == a.T - 1 ? (int)b : -1;
        }
        return;
    }
    if (tid < kTile) m.first[tid] = m.last[tid] = -1;
    __syncthreads();
    if (tid >= 32) return;
    int64_t lo = 0, hi = a.N + 1;                // first index with cu[index] >= t0 lies in [lo, hi]
    while (hi - lo > 32) {
        const int64_t step = (hi - lo + 31) / 32, i = lo + tid * step;
        const int c = __popc(__ballot_sync(0xffffffffu, i < hi && a.cu[i] < t0));
        if (c == 0) {
            hi = lo;
        } else {
            lo += (c - 1) * step + 1;
            hi = lo + step - 1 < hi ? lo + step - 1 : hi;
        }
    }
    lo += __popc(__ballot_sync(0xffffffffu, lo + tid < hi && a.cu[lo + tid] < t0));
    for (int64_t base = lo; base <= a.N; base += 32) {
        const int64_t i = base + tid;
        const int64_t o = i <= a.N ? a.cu[i] - t0 : kTile + 1;
        if (o >= 0 && o < kTile && i < a.N && a.cu[i + 1] > a.cu[i]) m.first[o] = (int)i;
        if (o > 0 && o <= kTile && i > 0 && a.cu[i - 1] < a.cu[i]) m.last[o - 1] = (int)(i - 1);
        if (__any_sync(0xffffffffu, o > kTile)) break;
    }
}

// Offsets that are not sorted from 0 to T; each tile looks at its share.
__device__ __forceinline__ void check_offsets(const GlrArgs& a, int64_t tile, int64_t tiles)
{
    for (int64_t n = tile * blockDim.x + threadIdx.x; n < a.N; n += tiles * blockDim.x)
        if (a.cu[n + 1] < a.cu[n] || (n == 0 && (a.cu[0] != 0 || a.cu[a.N] != a.T))) atomicOr(a.err, kErrSeqlens);
}

// The state entering tile i of column col: every lane its V channels, in `carry`.  One warp.
// ab: the tile's own (A, B), published for the tiles behind it.
template <int V>
__device__ __forceinline__ void tile_carry(const ScanWork& w, int64_t i, int64_t col, const float (&A)[V],
                                           const float (&B)[V], float (&carry)[V], int* err)
{
    constexpr int CB = 32 * V;
    const int lane = threadIdx.x % 32;
    const int64_t g = i / kGroup, first = g * kGroup;
    const int behind = (int)(i - first);         // earlier tiles of the group
    const bool last = behind == kGroup - 1, more = i + 1 < w.tiles;
    if (more && !last) {
        float* p = w.tile_ab + (i * w.cols + col) * 2 * CB + lane * V;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            __stcg(p + e, A[e]);
            __stcg(p + CB + e, B[e]);
        }
        __syncwarp();
        if (lane == 0) store_release(w.tile_flag + i * w.cols + col, 1);
    }
    // the group's earlier tiles as one run: nothing of it waits for the group's entry state
    float rA[V], rB[V];
#pragma unroll
    for (int e = 0; e < V; ++e) rA[e] = 1.f, rB[e] = 0.f, carry[e] = 0.f;
    if (lane < behind) {
        const int* flag = w.tile_flag + (first + lane) * w.cols + col;
        for (int k = 0; load_acquire(flag) == 0;)
            if (++k >= kPolls) {
                if (err) atomicOr(err, kErrScanWait);
                break;
            }
    }
    __syncwarp();
#pragma unroll 8
    for (int k = 0; k < behind; ++k) {
        const float* p = w.tile_ab + ((first + k) * w.cols + col) * 2 * CB + lane * V;
        float pa[V], pb[V];
        load_cg<V>(p, pa);
        load_cg<V>(p + CB, pb);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            rB[e] = leave(pa[e], pb[e], rB[e]);
            rA[e] = chain(rA[e], pa[e]);
        }
    }
    if (g > 0) {
        // a published entry state is a word of the value and a tag: it is read as soon as it is there
        const unsigned long long* p = w.entry + (g * w.cols + col) * CB + lane * V;
        int k = 0;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            unsigned long long v;
            while (((v = load_relaxed(p + e)) >> 32) == 0)
                if (++k >= kPolls) {
                    if (err) atomicOr(err, kErrScanWait);
                    break;
                }
            carry[e] = __uint_as_float((unsigned)v);
        }
    }
    if (more && last) {
        unsigned long long* p = w.entry + ((g + 1) * w.cols + col) * CB + lane * V;
#pragma unroll
        for (int e = 0; e < V; ++e)
            store_relaxed(p + e, (1ull << 32) | __float_as_uint(leave(A[e], B[e], leave(rA[e], rB[e], carry[e]))));
    }
#pragma unroll
    for (int e = 0; e < V; ++e) carry[e] = leave(rA[e], rB[e], carry[e]);
}

// (tile in scan order, column) of this CTA: by ticket when tiles wait on one another.
__device__ __forceinline__ int64_t take_tile(const ScanWork& w, int& slot)
{
    if (w.tiles == 1) return blockIdx.x;
    if (threadIdx.x == 0) slot = atomicAdd(w.ticket, 1);
    __syncthreads();
    return slot;
}

template <typename T, int V>
__global__ void __launch_bounds__(kWarps * 32, 3) glr_fwd_kernel(GlrArgs a, ScanWork w)
{
    constexpr int CB = 32 * V;
    __shared__ float sA[kWarps][CB], sB[kWarps][CB], sC[CB];
    __shared__ Marks marks;
    __shared__ int slot;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t id = take_tile(w, slot);
    const int64_t i = id / w.cols, col = id - i * w.cols;
    const int64_t blocks = (a.D + CB - 1) / CB, b = col / blocks;
    const int64_t c = (col - b * blocks) * CB + lane * V;
    const bool on = c < a.D;
    const int64_t t0 = i * kTile, tw = t0 + warp * kSteps;
    const int64_t at = (b * a.T + tw) * a.D + c;

    Raw<T, V> x[kSteps];
    Raw<float, V> al[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        if (on && tw + s < a.T) {
            al[s].load(a.log_a + at + s * a.D);
            x[s].load((const T*)a.x + at + s * a.D);
        } else {                                  // past the end: h stays as it is
            al[s].clear();
            x[s].clear();
        }
    }
    find_marks(a, b, t0, marks);
    __syncthreads();
    if (a.cu && col == 0) check_offsets(a, i, w.tiles);

    float A[V], B[V];
#pragma unroll
    for (int e = 0; e < V; ++e) A[e] = 1.f, B[e] = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
#pragma unroll
        for (int e = 0; e < V; ++e) al[s].v[e] = expf(al[s].v[e]);
        const int n = marks.first[warp * kSteps + s];
        if (n >= 0) {
            // from here on this token's register holds exp(log_a) h0: hT may be written over h0
            // before the second walk
            const int64_t row = glr_row(a, n, lane == 0 && c == 0);
            const bool has = a.h0 && row >= 0 && on;
            float h0[V];
#pragma unroll
            for (int e = 0; e < V; ++e) h0[e] = has ? a.h0[row * a.D + c + e] : 0.f;
            if (a.starts && warp == 0 && s == 0 && on)
                Raw<float, V>::store(a.starts + (b * w.tiles + i) * a.D + c, h0);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                al[s].v[e] *= h0[e];
                A[e] = -1.f;
                B[e] = al[s].v[e] + x[s].get(e);
            }
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                A[e] *= al[s].v[e];
                B[e] = al[s].v[e] * B[e] + x[s].get(e);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) sA[warp][lane * V + e] = A[e], sB[warp][lane * V + e] = B[e];
    __syncthreads();
    if (warp == 0) {
        float carry[V];
#pragma unroll
        for (int k = 1; k < kWarps; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float ak = sA[k][lane * V + e];
                B[e] = leave(ak, sB[k][lane * V + e], B[e]);
                A[e] = chain(A[e], ak);
            }
        tile_carry<V>(w, i, col, A, B, carry, a.err);
#pragma unroll
        for (int e = 0; e < V; ++e) sC[lane * V + e] = carry[e];
    }
    __syncthreads();
    float h[V];
#pragma unroll
    for (int e = 0; e < V; ++e) h[e] = sC[lane * V + e];
    for (int k = 0; k < warp; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = leave(sA[k][lane * V + e], sB[k][lane * V + e], h[e]);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int64_t t = tw + s;
        if (t >= a.T) break;
        const bool begins = marks.first[warp * kSteps + s] >= 0;
        if (a.starts && warp == 0 && s == 0 && on && !begins)
            Raw<float, V>::store(a.starts + (b * w.tiles + i) * a.D + c, h);
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = (begins ? al[s].v[e] : al[s].v[e] * h[e]) + x[s].get(e);
        if (a.out && on) Raw<T, V>::store((T*)a.out + at + s * a.D, h);
        const int m = marks.last[warp * kSteps + s];
        if (m >= 0 && a.hT) {
            const int64_t row = glr_row(a, m, false);
            if (row >= 0 && on) Raw<float, V>::store(a.hT + row * a.D + c, h);
        }
    }
    // sequences without tokens: every tile takes its share, a warp a sequence
    if ((a.cu || a.T == 0) && a.hT)
        for (int64_t n = i * kWarps + warp; n < a.N; n += w.tiles * kWarps)
            if (!a.cu || a.cu[n + 1] <= a.cu[n]) {
                const int64_t row = glr_row(a, n, lane == 0 && c == 0);
                if (row >= 0 && on)
#pragma unroll
                    for (int e = 0; e < V; ++e) a.hT[row * a.D + c + e] = a.h0 ? a.h0[row * a.D + c + e] : 0.f;
            }
}

template <typename T, int V>
__global__ void __launch_bounds__(kWarps * 32, 2) glr_bwd_kernel(GlrArgs a, ScanWork w)
{
    constexpr int CB = 32 * V;
    __shared__ float sA[kWarps][CB], sB[kWarps][CB], sC[CB];     // backward runs
    __shared__ float fA[kWarps][CB], fB[kWarps][CB];             // forward runs
    __shared__ Marks marks;
    __shared__ int slot;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t id = take_tile(w, slot);
    const int64_t order = id / w.cols, col = id - order * w.cols;
    const int64_t i = w.tiles - 1 - order;       // the last tile first
    const int64_t blocks = (a.D + CB - 1) / CB, b = col / blocks;
    const int64_t c = (col - b * blocks) * CB + lane * V;
    const bool on = c < a.D;
    const int64_t t0 = i * kTile, tw = t0 + warp * kSteps;
    const int64_t at = (b * a.T + tw) * a.D + c;

    Raw<T, V> x[kSteps], y[kSteps];
    Raw<float, V> al[kSteps];
    Raw<float, V> enter;
    enter.clear();
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        if (on && tw + s < a.T) {
            al[s].load(a.log_a + at + s * a.D);
            x[s].load((const T*)a.x + at + s * a.D);
            y[s].load((const T*)a.dout + at + s * a.D);
        } else {
            al[s].clear();
            x[s].clear();
            y[s].clear();
        }
    }
    if (on && a.T > 0) enter.load(a.starts + (b * w.tiles + i) * a.D + c);
    find_marks(a, b, t0, marks);
    __syncthreads();
    if (a.cu && col == 0) check_offsets(a, i, w.tiles);

    float A[V], B[V];
#pragma unroll
    for (int e = 0; e < V; ++e) A[e] = 1.f, B[e] = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int n = marks.first[warp * kSteps + s];
        if (n >= 0)
#pragma unroll
            for (int e = 0; e < V; ++e) A[e] = -1.f, B[e] = a.h0 && on ? a.h0[n * a.D + c + e] : 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            al[s].v[e] = expf(al[s].v[e]);
            A[e] *= al[s].v[e];
            B[e] = al[s].v[e] * B[e] + x[s].get(e);
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) fA[warp][lane * V + e] = A[e], fB[warp][lane * V + e] = B[e];
#pragma unroll
    for (int e = 0; e < V; ++e) A[e] = 1.f, B[e] = 0.f;
#pragma unroll
    for (int s = kSteps - 1; s >= 0; --s) {
        const int n = marks.last[warp * kSteps + s];
        if (n >= 0)
#pragma unroll
            for (int e = 0; e < V; ++e) A[e] = -1.f, B[e] = a.dhT && on ? a.dhT[n * a.D + c + e] : 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            A[e] *= al[s].v[e];
            B[e] = al[s].v[e] * (B[e] + y[s].get(e));
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) sA[warp][lane * V + e] = A[e], sB[warp][lane * V + e] = B[e];
    __syncthreads();
    if (warp == kWarps - 1) {
        float carry[V];
#pragma unroll
        for (int k = kWarps - 2; k >= 0; --k)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float ak = sA[k][lane * V + e];
                B[e] = leave(ak, sB[k][lane * V + e], B[e]);
                A[e] = chain(A[e], ak);
            }
        tile_carry<V>(w, order, col, A, B, carry, a.err);
#pragma unroll
        for (int e = 0; e < V; ++e) sC[lane * V + e] = carry[e];
    }
    // states before every token of the run, while the carry is on its way
    float h[V];
#pragma unroll
    for (int e = 0; e < V; ++e) h[e] = enter.v[e];
    for (int k = 0; k < warp; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = leave(fA[k][lane * V + e], fB[k][lane * V + e], h[e]);
    float before[kSteps][V];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int n = marks.first[warp * kSteps + s];
        if (n >= 0)
#pragma unroll
            for (int e = 0; e < V; ++e) h[e] = a.h0 && on ? a.h0[n * a.D + c + e] : 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            before[s][e] = h[e];
            h[e] = al[s].v[e] * h[e] + x[s].get(e);
        }
    }
    __syncthreads();
    float g[V];                                   // c of the token behind
#pragma unroll
    for (int e = 0; e < V; ++e) g[e] = sC[lane * V + e];
    for (int k = kWarps - 1; k > warp; --k)
#pragma unroll
        for (int e = 0; e < V; ++e) g[e] = leave(sA[k][lane * V + e], sB[k][lane * V + e], g[e]);
#pragma unroll
    for (int s = kSteps - 1; s >= 0; --s) {
        const int64_t t = tw + s;
        if (t >= a.T) continue;
        const int n = marks.last[warp * kSteps + s];
        if (n >= 0)
#pragma unroll
            for (int e = 0; e < V; ++e) g[e] = a.dhT && on ? a.dhT[n * a.D + c + e] : 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) g[e] += y[s].get(e);
        if (on) Raw<T, V>::store((T*)a.dx + at + s * a.D, g);
        float dl[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            g[e] *= al[s].v[e];
            dl[e] = g[e] * before[s][e];
        }
        if (on) Raw<float, V>::store(a.dlog_a + at + s * a.D, dl);
        const int m = marks.first[warp * kSteps + s];
        if (m >= 0 && a.dh0 && on) Raw<float, V>::store(a.dh0 + (int64_t)m * a.D + c, g);
    }
    if ((a.cu || a.T == 0) && a.dh0)
        for (int64_t n = i * kWarps + warp; n < a.N; n += w.tiles * kWarps)
            if ((!a.cu || a.cu[n + 1] <= a.cu[n]) && on)
#pragma unroll
                for (int e = 0; e < V; ++e) a.dh0[n * a.D + c + e] = a.dhT ? a.dhT[n * a.D + c + e] : 0.f;
}

template <typename T>
__global__ void __launch_bounds__(128)
glr_step_kernel(const T* __restrict__ x, const float* __restrict__ log_a, float* __restrict__ state,
                const int32_t* __restrict__ slots, T* __restrict__ out, int64_t P, int64_t D,
                int* __restrict__ err)
{
    const int64_t n = blockIdx.x;
    const int64_t c = (int64_t)blockIdx.y * 128 + threadIdx.x;
    if (c >= D) return;
    int64_t row = n;
    if (slots) {
        row = slots[n];
        if (row >= P && c == 0 && err) atomicOr(err, kErrSeqlens);
        if (row < 0 || row >= P) {
            IO<T>::store(out, n * D + c, 0.f);
            return;
        }
    }
    const float h = expf(log_a[n * D + c]) * state[row * D + c] + IO<T>::load(x, n * D + c);
    state[row * D + c] = h;
    IO<T>::store(out, n * D + c, h);
}

namespace {

// V channels a lane: the widest access that D allows, halved while it would leave half of
// the lanes without channels.
int lane_channels(int64_t D)
{
    int v = D % 4 == 0 ? 4 : D % 2 == 0 ? 2 : 1;
    while (v > 1 && 16 * v >= D) v /= 2;
    return v;
}

template <typename T, int V>
cudaError_t launch_scan(const GlrArgs& a, bool backward, cudaStream_t st)
{
    constexpr int64_t CB = 32 * V;
    ScanWork w = {};
    w.cols = a.B * ((a.D + CB - 1) / CB);
    w.tiles = a.T > 0 ? (a.T + kTile - 1) / kTile : 1;
    if (w.tiles > 0x7fffffffLL / w.cols) return cudaErrorInvalidConfiguration;
    StreamBuffer buf;
    if (w.tiles > 1) {
        const int64_t groups = (w.tiles + kGroup - 1) / kGroup;
        const int64_t flags = (4 + w.tiles * w.cols + 3) / 4 * 4, entries = groups * w.cols * CB;
        const int64_t zeroed = flags * 4 + entries * 8;
        cudaError_t e = buf.alloc((size_t)(zeroed + 2 * w.tiles * w.cols * CB * 4), st);
        if (e == cudaSuccess) e = cudaMemsetAsync(buf.ptr, 0, (size_t)zeroed, st);
        if (e != cudaSuccess) return e;
        w.ticket = static_cast<int*>(buf.ptr);
        w.tile_flag = w.ticket + 4;
        w.entry = reinterpret_cast<unsigned long long*>(w.ticket + flags);
        w.tile_ab = reinterpret_cast<float*>(w.entry + entries);
    }
    LaunchScope scope(st, backward ? K_GLR_BWD : K_GLR_FWD);
    const unsigned grid = (unsigned)(w.tiles * w.cols);
    if (backward) glr_bwd_kernel<T, V><<<grid, kWarps * 32, 0, st>>>(a, w);
    else glr_fwd_kernel<T, V><<<grid, kWarps * 32, 0, st>>>(a, w);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_scan_t(const GlrArgs& a, bool backward, cudaStream_t st)
{
    switch (lane_channels(a.D)) {
    case 4: return launch_scan<T, 4>(a, backward, st);
    case 2: return launch_scan<T, 2>(a, backward, st);
    }
    return launch_scan<T, 1>(a, backward, st);
}

}  // namespace

cudaError_t launch_glr_fwd(const GlrArgs& a, cudaStream_t st)
{
    return a.io == KDA_IO_F32 ? launch_scan_t<float>(a, false, st) : launch_scan_t<__nv_bfloat16>(a, false, st);
}

cudaError_t launch_glr_bwd(const GlrArgs& a, cudaStream_t st)
{
    return a.io == KDA_IO_F32 ? launch_scan_t<float>(a, true, st) : launch_scan_t<__nv_bfloat16>(a, true, st);
}

cudaError_t launch_glr_step(const void* x, const float* log_a, float* state, const int32_t* slots,
                            void* out, int64_t N, int64_t P, int64_t D, kda_io_dtype_t io, int* err,
                            cudaStream_t st)
{
    LaunchScope scope(st, K_GLR_STEP);
    const dim3 grid((unsigned)N, (unsigned)((D + 127) / 128));
    if (io == KDA_IO_F32)
        glr_step_kernel<float><<<grid, 128, 0, st>>>((const float*)x, log_a, state, slots, (float*)out, P, D, err);
    else
        glr_step_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>((const __nv_bfloat16*)x, log_a, state, slots,
                                                            (__nv_bfloat16*)out, P, D, err);
    return cudaGetLastError();
}

}  // namespace kda

using namespace kda;

namespace {

// Channels of one call: grid.y and the 32-bit tile arithmetic of the kernels.
constexpr int64_t kMaxChannels = int64_t(1) << 20;
constexpr int64_t kMaxTokens = int64_t(1) << 40;

kda_status_t glr_check_sizes(int64_t B, int64_t T, int64_t D, kda_io_dtype_t io)
{
    if (B < 0 || T < 0 || D < 0) return KDA_ERR_INVALID_ARG;
    if (io != KDA_IO_F32 && io != KDA_IO_BF16) return KDA_ERR_UNSUPPORTED;
    if (D > kMaxChannels || B > 0x7fffffffLL || T > kMaxTokens) return KDA_ERR_UNSUPPORTED;
    if (B > 0 && T > kMaxTokens / B) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status_t glr_fwd_impl(const void* x, const float* log_a, const float* h0, void* out, float* hT,
                          float* starts, const int32_t* slots, int64_t P, const int32_t* cu,
                          int64_t B, int64_t T, int64_t D, kda_io_dtype_t io, cudaStream_t stream)
{
    const kda_status_t s = glr_check_sizes(B, T, D, io);
    if (s != KDA_OK) return s;
    if (cu && B < 1) return KDA_ERR_INVALID_ARG;
    if (B == 0 || D == 0) return KDA_OK;
    if ((cu && !is_aligned(cu, 4)) || (slots && !is_aligned(slots, 4))) return KDA_ERR_INVALID_ARG;
    if (!optional_ok(h0) || !optional_ok(hT) || !optional_ok(starts)) return KDA_ERR_INVALID_ARG;
    const int64_t rows = cu ? 1 : B, n = rows * T * D, e = io == KDA_IO_F32 ? 4 : 2;
    if (n > 0) {
        if (!tensor_ok(x) || !tensor_ok(log_a) || !tensor_ok(out)) return KDA_ERR_INVALID_ARG;
        const int64_t ns = rows * ((T + KDA_GLR_TILE - 1) / KDA_GLR_TILE) * D * 4;
        const int64_t nh = (slots ? P : B) * D * 4;
        if (overlap(out, n * e, x, n * e) || overlap(out, n * e, log_a, n * 4) ||
            overlap(out, n * e, h0, nh) || overlap(out, n * e, hT, nh) || overlap(out, n * e, starts, ns) ||
            overlap(hT, nh, x, n * e) || overlap(hT, nh, log_a, n * 4) || overlap(hT, nh, starts, ns) ||
            overlap(starts, ns, x, n * e) || overlap(starts, ns, log_a, n * 4) || overlap(starts, ns, h0, nh))
            return KDA_ERR_INVALID_ARG;
        if (hT != h0 && overlap(hT, nh, h0, nh)) return KDA_ERR_INVALID_ARG;
    }
    GlrArgs a = {};
    a.x = x; a.log_a = log_a; a.h0 = h0; a.hT = hT; a.out = out; a.starts = starts;
    a.slots = slots; a.P = P; a.cu = cu; a.N = B; a.B = rows; a.T = T; a.D = D; a.io = io;
    cudaError_t err = library_error_word(&a.err);
    if (err == cudaSuccess) err = launch_glr_fwd(a, stream);
    return finish_call(err, stream);
}

kda_status_t glr_step_impl(const void* x, const float* log_a, float* state, const int32_t* slots,
                           void* out, int64_t N, int64_t P, int64_t D, kda_io_dtype_t io,
                           cudaStream_t stream)
{
    if (N < 0 || P < 0 || D < 0) return KDA_ERR_INVALID_ARG;
    if (io != KDA_IO_F32 && io != KDA_IO_BF16) return KDA_ERR_UNSUPPORTED;
    if (D > kMaxChannels || N > 0x7fffffffLL || P > kMaxTokens) return KDA_ERR_UNSUPPORTED;
    if (N == 0 || D == 0) return KDA_OK;
    if (!tensor_ok(x) || !tensor_ok(log_a) || !tensor_ok(out)) return KDA_ERR_INVALID_ARG;
    if (!(P == 0 && slots) && !tensor_ok(state)) return KDA_ERR_INVALID_ARG;
    if (slots && !is_aligned(slots, 4)) return KDA_ERR_INVALID_ARG;
    const int64_t e = io == KDA_IO_F32 ? 4 : 2, n = N * D, ns = P * D * 4;
    if (overlap(out, n * e, x, n * e) || overlap(out, n * e, log_a, n * 4) || overlap(out, n * e, state, ns) ||
        overlap(state, ns, x, n * e) || overlap(state, ns, log_a, n * 4))
        return KDA_ERR_INVALID_ARG;
    int* word = nullptr;
    cudaError_t err = slots ? library_error_word(&word) : cudaSuccess;
    if (err == cudaSuccess) err = launch_glr_step(x, log_a, state, slots, out, N, P, D, io, word, stream);
    return finish_call(err, stream);
}

}  // namespace

extern "C" {

kda_status_t kda_glr_scan_fwd(const void* x, const float* log_a, const float* h0, void* out,
                              float* hT, float* starts, const int32_t* cu_seqlens, int64_t B,
                              int64_t T, int64_t D, kda_io_dtype_t io_dtype, cudaStream_t stream)
{
    return glr_fwd_impl(x, log_a, h0, out, hT, starts, nullptr, 0, cu_seqlens, B, T, D, io_dtype,
                        stream);
}

kda_status_t kda_glr_scan_fwd_slots(const void* x, const float* log_a, float* state_pool,
                                    const int32_t* slots, void* out, float* starts,
                                    const int32_t* cu_seqlens, int64_t B, int64_t T, int64_t P,
                                    int64_t D, kda_io_dtype_t io_dtype, cudaStream_t stream)
{
    if (slots == nullptr || P < 0 || (P > 0 && state_pool == nullptr)) return KDA_ERR_INVALID_ARG;
    if (P > kMaxTokens) return KDA_ERR_UNSUPPORTED;
    return glr_fwd_impl(x, log_a, state_pool, out, state_pool, starts, slots, P, cu_seqlens, B, T, D,
                        io_dtype, stream);
}

kda_status_t kda_glr_scan_bwd(const void* x, const float* log_a, const float* h0,
                              const float* starts, const void* dout, const float* dhT, void* dx,
                              float* dlog_a, float* dh0, const int32_t* cu_seqlens, int64_t B,
                              int64_t T, int64_t D, kda_io_dtype_t io_dtype, cudaStream_t stream)
{
    const kda_status_t s = glr_check_sizes(B, T, D, io_dtype);
    if (s != KDA_OK) return s;
    if (cu_seqlens && B < 1) return KDA_ERR_INVALID_ARG;
    if (B == 0 || D == 0) return KDA_OK;
    if (cu_seqlens && !is_aligned(cu_seqlens, 4)) return KDA_ERR_INVALID_ARG;
    if (!optional_ok(h0) || !optional_ok(starts) || !optional_ok(dhT) || !optional_ok(dh0))
        return KDA_ERR_INVALID_ARG;
    const int64_t rows = cu_seqlens ? 1 : B, n = rows * T * D, e = io_dtype == KDA_IO_F32 ? 4 : 2;
    const int64_t ns = rows * ((T + KDA_GLR_TILE - 1) / KDA_GLR_TILE) * D * 4, nh = B * D * 4;
    if (n > 0) {
        if (!tensor_ok(x) || !tensor_ok(log_a) || !tensor_ok(dout) || !tensor_ok(dx) || !tensor_ok(dlog_a))
            return KDA_ERR_INVALID_ARG;
        const struct { const void* p; int64_t n; } in[] = {{x, n * e}, {log_a, n * 4}, {dout, n * e},
                                                            {h0, nh}, {starts, ns}, {dhT, nh}},
                                                   res[] = {{dx, n * e}, {dlog_a, n * 4}, {dh0, nh}};
        for (int i = 0; i < 3; ++i) {
            for (const auto& q : in)
                if (overlap(res[i].p, res[i].n, q.p, q.n))
                    return KDA_ERR_INVALID_ARG;
            for (int j = 0; j < i; ++j)
                if (overlap(res[i].p, res[i].n, res[j].p, res[j].n)) return KDA_ERR_INVALID_ARG;
        }
    }
    GlrArgs a = {};
    a.x = x; a.log_a = log_a; a.h0 = h0; a.starts = const_cast<float*>(starts);
    a.dout = dout; a.dhT = dhT; a.dx = dx; a.dlog_a = dlog_a; a.dh0 = dh0;
    a.cu = cu_seqlens; a.N = B; a.B = rows; a.T = T; a.D = D; a.io = io_dtype;
    cudaError_t err = library_error_word(&a.err);
    StreamBuffer buf;
    if (err == cudaSuccess && starts == nullptr && n > 0) {
        // the caller kept no tile starts: one forward pass that writes nothing else
        err = buf.alloc((size_t)ns, stream);
        if (err == cudaSuccess) {
            a.starts = static_cast<float*>(buf.ptr);
            GlrArgs f = a;
            f.hT = nullptr; f.out = nullptr;
            err = launch_glr_fwd(f, stream);
        }
    }
    if (err == cudaSuccess) err = launch_glr_bwd(a, stream);
    return finish_call(err, stream);
}

kda_status_t kda_glr_step(const void* x, const float* log_a, float* state, void* out, int64_t N,
                          int64_t D, kda_io_dtype_t io_dtype, cudaStream_t stream)
{
    return glr_step_impl(x, log_a, state, nullptr, out, N, N, D, io_dtype, stream);
}

kda_status_t kda_glr_step_slots(const void* x, const float* log_a, float* state_pool,
                                const int32_t* slots, void* out, int64_t N, int64_t P, int64_t D,
                                kda_io_dtype_t io_dtype, cudaStream_t stream)
{
    if (slots == nullptr) return KDA_ERR_INVALID_ARG;
    return glr_step_impl(x, log_a, state_pool, slots, out, N, P, D, io_dtype, stream);
}

}  // extern "C"
