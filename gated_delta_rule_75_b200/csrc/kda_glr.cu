// Gated linear recurrence, h_t = exp(log_a_t) h_{t-1} + x_t per channel: the
// elementwise sibling of the delta rule (a vector state, the same per-channel
// decay), its gradients and its decode step.
//
// Scan.  A run of tokens maps the state it enters with affinely, h -> A h + B, and
// runs compose.  A tile is kTile tokens of kCh channels, cut into kRuns runs; the
// scan is one pass over memory, bound by it, with one persistent CTA per SM whose
// warps each do one part of the work for the tiles that pass through a ring of
// shared-memory stages:
//   loaders      take a tile and start its copies, a few tiles ahead: TMA boxes where
//                every row starts on 16 bytes, else four more warps copy the 16-byte
//                chunks that cover each row (cp.async);
//   aggregators  (two groups of kRuns warps, tiles in turn) fold each run of the
//                tile into (A, B);
//   carriers     (three warps, tiles in turn) fold the runs, publish the tile's (A, B)
//                and put the state that enters the tile together from what earlier
//                tiles published: the state entering its group of kGroup tiles, then
//                the (A, B) of the group's earlier tiles, in that order whatever
//                arrives first; the last tile of a group publishes the state that
//                enters the next one;
//   finishers    (two groups of kRuns warps) walk the runs again from their entry
//                states and write the outputs.
// So loads, arithmetic and the waits of different tiles overlap, a value is the same on
// every run, and the chain of waits is one hop per kGroup * kTile tokens.  Tiles are
// taken by a ticket, first tokens first, and every CTA works through its tiles in
// that order: whatever a tile waits for was taken earlier and waits for nothing
// later, so every wait ends (and is bounded all the same).
//
// Sequences: a token that begins one replaces the state by h0, whatever came before it
// (a NaN too): A = -1 there, and a run whose A is negative is h -> B.
//
// Backward.  With c_t = exp(log_a_t) g_t, g_t = dout_t + c_{t+1}: the same scan over
// tiles from the last to the first, replaced by dhT at a sequence's last token.
// dlog_a_t = c_t h_{t-1} needs the forward states too; they are walked again inside
// the tile from its kept entry state (starts), so the pass reads x, log_a, dout and
// writes dx, dlog_a once.
#include "kda_common.cuh"
#include "kda_internal.h"
#include "kda_tma.cuh"
#include "kda_umma.cuh"

namespace kda {

constexpr int kTile = KDA_GLR_TILE;     // tokens of a tile
constexpr int kCh = 64;                 // channels of a tile, two a lane
constexpr int kRuns = 4;                // runs of a tile, one a warp
constexpr int kSteps = kTile / kRuns;   // tokens of a run
constexpr int kGroup = 16;              // tiles between published entry states
constexpr int kPolls = 1 << 21;         // about two seconds of polling
constexpr int kScanBit = 7;             // kErrScanWait
constexpr int kAtOnce = 8;              // published tiles asked for together

// Warps by role: with TMA 20, five to a quarter of the SM.
constexpr int kAggWarps = 2 * kRuns, kFinWarps = 2 * kRuns, kCarryWarps = 3, kCopyWarps = 4;
constexpr int scan_threads(bool aligned) { return 32 * (kAggWarps + kFinWarps + kCarryWarps + 1 + (aligned ? 0 : kCopyWarps)); }

// Workspace: a ticket, the groups' entry states and the tiles' (A, B), all zeroed by the setup
// kernel; with cu_seqlens each tile's range of offsets.  A column is one block of kCh
// channels of one row of the token axis; tiles and groups are numbered in the order of the
// scan (from the end in the backward).
struct ScanWork {
    int* ticket;                   // null: one tile a column, nothing waits, no ticket needed
    unsigned long long* entry;     // [groups][cols][kCh]: words (1, state)
    unsigned long long* tile_ab;   // [tiles][cols][kCh]: words (A, B)
    int2* range;                   // [tiles]: offsets cu[x .. y - 1] lie in [first token, first + kTile]
    int64_t cols, tiles, total;    // total = tiles * cols
    int64_t zeroed;                // 16-byte words from ticket on
};

// Published words, two channels at once: A, its lowest bit set as the tag of a word that is there
// (half a step more on A), and B in the high half.  Each word is read and written whole, so a tag
// comes with its value and nothing else has to be ordered.
__device__ __forceinline__ void load_words(const unsigned long long* p, unsigned long long& a, unsigned long long& b)
{
    asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "l"(p) : "memory");
}
__device__ __forceinline__ void store_words(unsigned long long* p, const float (&A)[2], const float (&B)[2])
{
    const unsigned long long a = ((unsigned long long)__float_as_uint(B[0]) << 32) | __float_as_uint(A[0]) | 1u;
    const unsigned long long b = ((unsigned long long)__float_as_uint(B[1]) << 32) | __float_as_uint(A[1]) | 1u;
    asm volatile("st.relaxed.gpu.global.v2.u64 [%0], {%1, %2};" ::"l"(p), "l"(a), "l"(b) : "memory");
}

// 16 bytes global -> shared, the first n of them read and the rest zero.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int n)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// One arrival on `bar` once this thread's copies so far are complete.
__device__ __forceinline__ void arrive_when_copied(uint64_t* bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(umma::smem_u32(bar)) : "memory");
}

// Two channels at once: a register pair, and one instruction for both.
struct F2 {
    unsigned long long v;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ float x() const { return __uint_as_float((unsigned)v); }
    __device__ __forceinline__ float y() const { return __uint_as_float((unsigned)(v >> 32)); }
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    F2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}

// exp of two logarithms of decays: 2^t with t = x / ln 2 rounded, times 1 + r ln 2 for the part r of
// x / ln 2 that the rounding and the constant dropped, so that large logarithms lose nothing.
// -200 and below (-inf too) give 0, NaN stays.
__device__ __forceinline__ F2 decay2(F2 l)
{
    float a, b;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(l.x()), "f"(-200.f));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(b) : "f"(l.y()), "f"(-200.f));
    constexpr float hi = 1.4426950408889634f, lo = (float)(1.4426950408889634 - (double)hi), ln2 = 0.6931471805599453f;
    const F2 x(a, b), t = mul2(x, F2(hi, hi));
    const F2 minus(-t.x(), -t.y());
    const F2 r = fma2(x, F2(lo, lo), fma2(x, F2(hi, hi), minus));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(t.x()));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(t.y()));
    const F2 e(a, b);
    return fma2(mul2(e, F2(ln2, ln2)), r, e);
}

// The state behind a run (A, B) entered with h.  A negative A (-0 too): the run holds the
// border of a sequence and nothing crosses it.
__device__ __forceinline__ float leave(float A, float B, float h)
{
    return __float_as_int(A) < 0 ? B : A * h + B;
}
// A of a run followed by a run with A = a.
__device__ __forceinline__ float chain(float A, float a) { return __float_as_int(a) < 0 ? a : A * a; }

// Row of h0 / hT / the pool that holds sequence n's state; -1: none.
__device__ __forceinline__ int64_t glr_row(const GlrArgs& a, int64_t n, bool report)
{
    if (a.slots == nullptr) return n;
    const int64_t s = a.slots[n];
    if (s >= a.P && report && a.err) atomicOr(a.err, kErrSeqlens);
    return s >= 0 && s < a.P ? s : -1;
}

// Rows of a tile in shared memory.  Aligned: every row of the tensor starts on 16 bytes and
// holds whole 16-byte chunks, lane l owns channels 2 l, 2 l + 1.  Otherwise the chunks that
// cover a row are copied, one more than its bytes need, the row starts (row index * D) mod
// (16 bytes) elements into them, and lane l owns channels l, l + 32.
template <typename E, bool Aligned>
struct Rows {
    static constexpr int kBytes = kCh * (int)sizeof(E);
    static constexpr int kPitch = kBytes + (Aligned ? 0 : 16);
    static constexpr int kPer16 = 16 / (int)sizeof(E);

    // Copies of rows [r0, r1) of the tile, whose row 0 is row `first`; rows from `live` on read as
    // zeros; channels from c0.  Unaligned rows only.
    static __device__ __forceinline__ void copy(unsigned char* dst, const E* src, int64_t first, int r0, int r1,
                                                int live, int64_t D, int64_t c0, int64_t total)
    {
        constexpr int kChunks = kBytes / 16, kRowsAtOnce = 32 / kChunks;
        const int lane = threadIdx.x % 32;
        strip(umma::smem_u32(dst), src, first, r0 + lane / kChunks, r1, live, D, c0, total, kRowsAtOnce, lane % kChunks);
        strip(umma::smem_u32(dst), src, first, r0 + lane, r1, live, D, c0, total, 32, kChunks);
    }
    // One chunk of rows r0, r0 + step, ..
    static __device__ __forceinline__ void strip(uint32_t to, const E* src, int64_t first, int r0, int r1, int live,
                                                 int64_t D, int64_t c0, int64_t total, const int step, int chunk)
    {
        const unsigned char* at = reinterpret_cast<const unsigned char*>(src + (first + r0) * D + c0);
        const unsigned char* end = reinterpret_cast<const unsigned char*>(src + total);
        const int64_t pitch = step * D * (int64_t)sizeof(E);
        const int left = (int)((D - c0 < kCh ? D - c0 : kCh) * sizeof(E)) - chunk * 16;    // row bytes from the chunk on
        to += r0 * kPitch + chunk * 16;
#pragma unroll 4
        for (int r = r0; r < r1; r += step, at += pitch, to += step * kPitch) {
            const int into = (int)(reinterpret_cast<uintptr_t>(at) & 15);
            const unsigned char* p = at - into + chunk * 16;
            const bool in = r < live && left + into > 0;
            const int64_t rest = end - p;        // never past the tensor's end
            copy16(to, in ? p : reinterpret_cast<const unsigned char*>(src), in ? rest < 16 ? (int)rest : 16 : 0);
        }
    }
    // Elements into its chunks at which row `row` starts.
    static __device__ __forceinline__ int shift(int64_t row, int64_t D)
    {
        return Aligned ? 0 : (int)((row * D) % kPer16);
    }
    // The lane's two channels of row r of the tile.
    static __device__ __forceinline__ F2 get(const unsigned char* base, int r, int shift, int lane)
    {
        const E* p = reinterpret_cast<const E*>(base + r * kPitch);
        if constexpr (!Aligned) return F2(IO<E>::load(p, shift + lane), IO<E>::load(p, shift + lane + 32));
        if constexpr (sizeof(E) == 4) {
            F2 v;
            v.v = reinterpret_cast<const unsigned long long*>(p)[lane];
            return v;
        } else {
            const uint32_t u = reinterpret_cast<const uint32_t*>(p)[lane];
            return F2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
        }
    }
    static __device__ __forceinline__ void put(unsigned char* base, int r, int shift, int lane, F2 v)
    {
        static_assert(sizeof(E) == 4, "decays only");
        float* p = reinterpret_cast<float*>(base + r * kPitch);
        if constexpr (Aligned) {
            reinterpret_cast<unsigned long long*>(p)[lane] = v.v;
        } else {
            p[shift + lane] = v.x();
            p[shift + lane + 32] = v.y();
        }
    }
};

// The lane's two channels, from c0, of a row of a tensor in global memory; on0, on1: which of
// them exist (aligned: both or none).
template <typename E, bool Aligned>
__device__ __forceinline__ void store_pair(E* at, bool on0, bool on1, F2 v)
{
    if constexpr (Aligned) {
        if (!on0) return;
        if constexpr (sizeof(E) == 4) {
            __stcs(reinterpret_cast<float2*>(at), make_float2(v.x(), v.y()));
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v.x(), v.y());
            __stcs(reinterpret_cast<unsigned int*>(at), *reinterpret_cast<const unsigned int*>(&h));
        }
    } else {
        if (on0) IO<E>::store(at, 0, v.x());
        if (on1) IO<E>::store(at, 32, v.y());
    }
}
template <bool Aligned>
__device__ __forceinline__ F2 load_pair(const float* at, bool on0, bool on1)
{
    return F2(at && on0 ? at[0] : 0.f, at && on1 ? at[Aligned ? 1 : 32] : 0.f);
}

// One stage of the ring.
template <typename T, bool Aligned, bool Bwd>
struct Stage {
    using La = Rows<float, Aligned>;
    using X = Rows<T, Aligned>;
    alignas(128) unsigned char la[kTile * La::kPitch];           // log_a, then exp(log_a)
    alignas(128) unsigned char x[kTile * X::kPitch];
    alignas(128) unsigned char y[Bwd ? kTile * X::kPitch : 128]; // dout
    float A[kRuns][kCh], B[kRuns][kCh];                          // runs in the scan's direction
    float fA[Bwd ? kRuns : 1][kCh], fB[Bwd ? kRuns : 1][kCh];    // backward: the forward runs too
    float carry[kCh];
    int first[kTile], last[kTile];                               // sequences that begin / end there, or -1
    int64_t id;                                                  // tile * cols + column; -1: no more
    int marked;                                                  // whether first / last hold anything
    uint64_t taken, full, agg, carried, empty;
    static constexpr uint32_t kCopied = kTile * (La::kBytes + X::kBytes * (Bwd ? 2 : 1));
};
template <typename T, bool Aligned, bool Bwd> constexpr int ring_stages()
{
    constexpr int n = (int)((227 * 1024 - 64) / sizeof(Stage<T, Aligned, Bwd>));
    return n < 8 ? n : 8;
}

// Where a tile lies (tiles, columns and their product fit 31 bits).
struct TileAt {
    uint32_t order, col, i;                      // order: in the scan; i: on the token axis
    int64_t b, t0, row0, c0;                     // row0 = b * T + t0
    __device__ __forceinline__ TileAt(const GlrArgs& a, const ScanWork& w, int64_t id, bool bwd)
    {
        order = (uint32_t)id / (uint32_t)w.cols;
        col = (uint32_t)id - order * (uint32_t)w.cols;
        i = bwd ? (uint32_t)w.tiles - 1 - order : order;
        const uint32_t blocks = (uint32_t)((a.D + kCh - 1) / kCh), row = col / blocks;
        b = row;
        c0 = (int64_t)(col - row * blocks) * kCh;
        t0 = (int64_t)i * kTile;
        row0 = b * a.T + t0;
    }
};

// Before a scan: zeroes the ticket, flags and entry states, finds every tile's offsets, checks
// the offsets, and passes the states of sequences without tokens on.
__global__ void __launch_bounds__(256) glr_setup_kernel(GlrArgs a, ScanWork w, int bwd)
{
    griddep_wait();
    griddep_launch_dependents();
    const int64_t me = (int64_t)blockIdx.x * 256 + threadIdx.x, all = (int64_t)gridDim.x * 256;
    for (int64_t k = me; k < w.zeroed; k += all) reinterpret_cast<uint4*>(w.ticket)[k] = make_uint4(0, 0, 0, 0);
    if (a.cu) {
        for (int64_t i = me; i < w.tiles; i += all) {
            int at[2];
            for (int k = 0; k < 2; ++k) {
                const int64_t bound = i * kTile + (k ? kTile + 1 : 0);
                int64_t lo = 0, hi = a.N + 1;    // first index with cu[index] >= bound
                while (lo < hi) {
                    const int64_t mid = (lo + hi) >> 1;
                    if (a.cu[mid] < bound) lo = mid + 1; else hi = mid;
                }
                at[k] = (int)lo;
            }
            w.range[i] = make_int2(at[0], at[1]);
        }
        for (int64_t n = me; n < a.N; n += all)
            if (a.cu[n + 1] < a.cu[n] || (n == 0 && (a.cu[0] != 0 || a.cu[a.N] != a.T))) atomicOr(a.err, kErrSeqlens);
    }
    const float* from = bwd ? a.dhT : a.h0;
    float* to = bwd ? a.dh0 : a.hT;
    if ((!a.cu && a.T > 0) || to == nullptr) return;
    for (int64_t n = me / 32; n < a.N; n += all / 32) {
        if (a.cu && a.cu[n + 1] > a.cu[n]) continue;
        const int64_t row = bwd ? n : glr_row(a, n, me % 32 == 0);
        if (row < 0 || to == from) continue;
        for (int64_t c = me % 32; c < a.D; c += 32) to[row * a.D + c] = from ? from[row * a.D + c] : 0.f;
    }
}

// Tensor maps of log_a, x and dout (aligned rows).
struct ScanMaps {
    CUtensorMap la, x, y;
};

// The loader warp that takes the tiles, marks their sequences and, for aligned rows, starts the
// copies.
template <typename T, bool Aligned, bool Bwd, int NS>
__device__ __forceinline__ void scan_load(const GlrArgs& a, const ScanWork& w, const ScanMaps& maps,
                                          Stage<T, Aligned, Bwd>* ring)
{
    using S = Stage<T, Aligned, Bwd>;
    const int lane = threadIdx.x % 32;
    int64_t next = blockIdx.x;
    if (w.ticket) {
        int v = 0;
        if (lane == 0) v = atomicAdd(w.ticket, 1);
        next = __shfl_sync(0xffffffffu, v, 0);
    }
    int ends = 0;
    for (int64_t q = 0; ends < kCarryWarps; ++q) {
        S& s = ring[q % NS];
        const int64_t id = next < w.total ? next : -1;
        int v = 0;
        if (w.ticket && id >= 0 && lane == 0) v = atomicAdd(w.ticket, 1);   // the next tile's, on its way meanwhile
        const TileAt at(a, w, id < 0 ? 0 : id, Bwd);
        int2 range = make_int2(0, 0);
        if (a.cu && id >= 0) range = w.range[at.i];
        if (q >= NS && !umma::mbar_wait(&s.empty, (uint32_t)((q / NS - 1) & 1), a.err, kScanBit)) {
            // given up: the copies under way have to land before the CTA may end
            for (int64_t k = q - NS; k < q; ++k)
                umma::mbar_wait(&ring[k % NS].full, (uint32_t)((k / NS) & 1), a.err, kScanBit);
            return;
        }
        if (id < 0) ++ends;                      // one for every worker that takes tiles in turn
        if (lane == 0) {
            s.id = id;
            if constexpr (Aligned) {
                if (id >= 0) {
                    tma::expect_tx(&s.full, S::kCopied);
                    tma::load_3d(s.la, &maps.la, (int)at.c0, (int)at.t0, (int)at.b, &s.full);
                    tma::load_3d(s.x, &maps.x, (int)at.c0, (int)at.t0, (int)at.b, &s.full);
                    if constexpr (Bwd) tma::load_3d(s.y, &maps.y, (int)at.c0, (int)at.t0, (int)at.b, &s.full);
                } else {
                    umma::mbar_arrive(&s.full);
                }
            } else {
                umma::mbar_arrive(&s.taken);
            }
        }
        if (id >= 0) {
            // sequences that begin or end in the tile
            const bool begins = !a.cu && at.t0 == 0, ends_here = !a.cu && at.t0 + kTile >= a.T;
            const bool marked = a.cu ? range.y > range.x : begins || ends_here;
            if (lane == 0) s.marked = marked;
            if (marked) {
                for (int t = lane; t < kTile; t += 32) {
                    s.first[t] = begins && t == 0 ? (int)at.b : -1;
                    s.last[t] = ends_here && at.t0 + t == a.T - 1 ? (int)at.b : -1;
                }
                __syncwarp();
                for (int64_t k = range.x + lane; k < range.y; k += 32) {
                    const int64_t o = a.cu[k] - at.t0;
                    if (o >= 0 && o < kTile && k < a.N && a.cu[k + 1] > a.cu[k]) s.first[o] = (int)k;
                    if (o > 0 && o <= kTile && k > 0 && a.cu[k - 1] < a.cu[k]) s.last[o - 1] = (int)(k - 1);
                }
            }
        }
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(&s.full);
        if (w.ticket) next = __shfl_sync(0xffffffffu, v, 0);
        else next += gridDim.x;
        if (id < 0) next = w.total;
    }
}

// A copying warp (unaligned rows): its share of every tile's rows.
template <typename T, bool Bwd, int NS>
__device__ __forceinline__ void scan_copy(const GlrArgs& a, const ScanWork& w, Stage<T, false, Bwd>* ring, int share)
{
    using S = Stage<T, false, Bwd>;
    const int64_t total = a.B * a.T * a.D;
    const int r0 = share * (kTile / kCopyWarps), r1 = r0 + kTile / kCopyWarps;
    int ends = 0;
    for (int64_t q = 0; ends < kCarryWarps; ++q) {
        S& s = ring[q % NS];
        if (!umma::mbar_wait(&s.taken, (uint32_t)((q / NS) & 1), a.err, kScanBit)) break;
        if (s.id < 0) {
            ++ends;
        } else {
            const TileAt at(a, w, s.id, Bwd);
            const int live = (int)(a.T - at.t0 < kTile ? a.T - at.t0 : kTile);
            S::La::copy(s.la, a.log_a, at.row0, r0, r1, live, a.D, at.c0, total);
            S::X::copy(s.x, (const T*)a.x, at.row0, r0, r1, live, a.D, at.c0, total);
            if constexpr (Bwd) S::X::copy(s.y, (const T*)a.dout, at.row0, r0, r1, live, a.D, at.c0, total);
        }
        arrive_when_copied(&s.full);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// An aggregator warp: run `run` of every second tile, from tile `group` on.
template <typename T, bool Aligned, bool Bwd, int NS>
__device__ __forceinline__ void scan_aggregate(const GlrArgs& a, const ScanWork& w, Stage<T, Aligned, Bwd>* ring,
                                               int group, int run)
{
    using S = Stage<T, Aligned, Bwd>;
    const int lane = threadIdx.x % 32, r0 = run * kSteps;
    const int dl = (int)(a.D % S::La::kPer16), dx = (int)(a.D % S::X::kPer16);   // shifts from row to row
    for (int64_t q = group;; q += 2) {
        S& s = ring[q % NS];
        if (!umma::mbar_wait(&s.full, (uint32_t)((q / NS) & 1), a.err, kScanBit) || s.id < 0) return;
        const TileAt at(a, w, s.id, Bwd);
        int sl = S::La::shift(at.row0 + r0, a.D), sx = S::X::shift(at.row0 + r0, a.D);
        F2 A(1.f, 1.f), B(0.f, 0.f);
        if (!s.marked) {
#pragma unroll 4
            for (int k = 0; k < kSteps; ++k) {
                const F2 l = decay2(S::La::get(s.la, r0 + k, sl, lane));
                A = mul2(A, l);
                B = fma2(l, B, S::X::get(s.x, r0 + k, sx, lane));
                S::La::put(s.la, r0 + k, sl, lane, l);   // the finishers take the decay from here
                sl = (sl + dl) % S::La::kPer16;
                sx = (sx + dx) % S::X::kPer16;
            }
            if constexpr (Bwd) {
                *reinterpret_cast<F2*>(&s.fA[run][2 * lane]) = A;
                *reinterpret_cast<F2*>(&s.fB[run][2 * lane]) = B;
                // the product of the decays is the same from either end but for its rounding
                B = F2(0.f, 0.f);
#pragma unroll 4
                for (int k = kSteps - 1; k >= 0; --k) {
                    sl = (sl + S::La::kPer16 - dl) % S::La::kPer16;
                    sx = (sx + S::X::kPer16 - dx) % S::X::kPer16;
                    B = mul2(S::La::get(s.la, r0 + k, sl, lane), add2(B, S::X::get(s.y, r0 + k, sx, lane)));
                }
            }
        } else {
            const int64_t c = at.c0 + (Aligned ? 2 * lane : lane);
            const bool on0 = c < a.D, on1 = c + (Aligned ? 1 : 32) < a.D;
            for (int k = 0; k < kSteps; ++k) {
                const int r = r0 + k;
                F2 l = decay2(S::La::get(s.la, r, sl, lane));
                const F2 x = S::X::get(s.x, r, sx, lane);
                const int n = s.first[r];
                if (n >= 0) {
                    const int64_t row = Bwd ? n : glr_row(a, n, lane == 0 && at.c0 == 0);
                    const F2 h0 = load_pair<Aligned>(a.h0 && row >= 0 ? a.h0 + row * a.D + c : nullptr, on0, on1);
                    A = F2(-1.f, -1.f);
                    B = add2(mul2(l, h0), x);
                    if constexpr (!Bwd) {
                        // the finishers find exp(log_a) h0 here: hT may be written over h0 before they come
                        l = mul2(l, h0);
                        if (a.starts && r == 0)
                            store_pair<float, Aligned>(a.starts + (at.b * w.tiles + at.i) * a.D + c, on0, on1, h0);
                    }
                } else {
                    A = mul2(A, l);
                    B = fma2(l, B, x);
                }
                S::La::put(s.la, r, sl, lane, l);
                sl = (sl + dl) % S::La::kPer16;
                sx = (sx + dx) % S::X::kPer16;
            }
            if constexpr (Bwd) {
                *reinterpret_cast<F2*>(&s.fA[run][2 * lane]) = A;
                *reinterpret_cast<F2*>(&s.fB[run][2 * lane]) = B;
                A = F2(1.f, 1.f);
                B = F2(0.f, 0.f);
                for (int k = kSteps - 1; k >= 0; --k) {
                    const int r = r0 + k;
                    sl = (sl + S::La::kPer16 - dl) % S::La::kPer16;
                    sx = (sx + S::X::kPer16 - dx) % S::X::kPer16;
                    const int n = s.last[r];
                    if (n >= 0) {
                        A = F2(-1.f, -1.f);
                        B = load_pair<Aligned>(a.dhT ? a.dhT + (int64_t)n * a.D + c : nullptr, on0, on1);
                    }
                    const F2 l = S::La::get(s.la, r, sl, lane);
                    A = mul2(A, l);
                    B = mul2(l, add2(B, S::X::get(s.y, r, sx, lane)));
                }
            }
        }
        *reinterpret_cast<F2*>(&s.A[run][2 * lane]) = A;
        *reinterpret_cast<F2*>(&s.B[run][2 * lane]) = B;
        // the decays written over log_a come before the TMA copy that fills the stage again
        if constexpr (Aligned) umma::fence_smem_to_async();
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(&s.agg);
    }
}

// A carrier warp: every third tile, from tile `first` on.
template <typename T, bool Aligned, bool Bwd, int NS>
__device__ __forceinline__ void scan_carry(const GlrArgs& a, const ScanWork& w, Stage<T, Aligned, Bwd>* ring, int from)
{
    using S = Stage<T, Aligned, Bwd>;
    const int lane = threadIdx.x % 32;
    for (int64_t q = from;; q += kCarryWarps) {
        S& s = ring[q % NS];
        // the end is announced by the loader alone
        if (!umma::mbar_wait(&s.full, (uint32_t)((q / NS) & 1), a.err, kScanBit) || s.id < 0) return;
        if (!umma::mbar_wait(&s.agg, (uint32_t)((q / NS) & 1), a.err, kScanBit)) return;
        const TileAt at(a, w, s.id, Bwd);
        const int64_t g = at.order / kGroup, first = g * kGroup;
        const int behind = (int)(at.order - first);      // earlier tiles of the group
        const bool last = behind == kGroup - 1, more = at.order + 1 < w.tiles;
        float A[2] = {1.f, 1.f}, B[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < kRuns; ++k) {
            const int run = Bwd ? kRuns - 1 - k : k;
            const float2 ra = *reinterpret_cast<const float2*>(&s.A[run][2 * lane]);
            const float2 rb = *reinterpret_cast<const float2*>(&s.B[run][2 * lane]);
            B[0] = leave(ra.x, rb.x, B[0]);
            B[1] = leave(ra.y, rb.y, B[1]);
            A[0] = chain(A[0], ra.x);
            A[1] = chain(A[1], ra.y);
        }
        if (more && !last) store_words(w.tile_ab + ((int64_t)at.order * w.cols + at.col) * kCh + 2 * lane, A, B);
        // an entry state is a word of the value and a tag: it is read as soon as it is there, and
        // asked for now
        const unsigned long long* entry = w.entry + (g * w.cols + at.col) * kCh + 2 * lane;
        unsigned long long e0 = 0, e1 = 0;
        if (g > 0) load_words(entry, e0, e1);
        // the group's earlier tiles as one run: nothing of it waits for the group's entry state
        float rA[2] = {1.f, 1.f}, rB[2] = {0.f, 0.f}, carry[2] = {0.f, 0.f};
        const unsigned long long* ab = w.tile_ab + (first * w.cols + at.col) * kCh + 2 * lane;
        int polls = 0;
        for (int k0 = 0; k0 < behind; k0 += kAtOnce) {
            unsigned long long v0[kAtOnce], v1[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
                if (k0 + k < behind) load_words(ab + (int64_t)(k0 + k) * w.cols * kCh, v0[k], v1[k]);
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
                if (k0 + k < behind) {
                    while (!(v0[k] & v1[k] & 1)) {
                        if (++polls >= kPolls) {
                            if (a.err) atomicOr(a.err, kErrScanWait);
                            break;
                        }
                        load_words(ab + (int64_t)(k0 + k) * w.cols * kCh, v0[k], v1[k]);
                    }
                    const float pa[2] = {__uint_as_float((unsigned)v0[k]), __uint_as_float((unsigned)v1[k])};
                    rB[0] = leave(pa[0], __uint_as_float((unsigned)(v0[k] >> 32)), rB[0]);
                    rB[1] = leave(pa[1], __uint_as_float((unsigned)(v1[k] >> 32)), rB[1]);
                    rA[0] = chain(rA[0], pa[0]);
                    rA[1] = chain(rA[1], pa[1]);
                }
        }
        if (g > 0) {
            while (!(e0 & e1 & 1)) {
                if (++polls >= kPolls) {
                    if (a.err) atomicOr(a.err, kErrScanWait);
                    break;
                }
                load_words(entry, e0, e1);
            }
            carry[0] = __uint_as_float((unsigned)(e0 >> 32));
            carry[1] = __uint_as_float((unsigned)(e1 >> 32));
        }
        carry[0] = leave(rA[0], rB[0], carry[0]);
        carry[1] = leave(rA[1], rB[1], carry[1]);
        if (more && last) {
            const float one[2] = {1.f, 1.f}, out[2] = {leave(A[0], B[0], carry[0]), leave(A[1], B[1], carry[1])};
            store_words(w.entry + ((g + 1) * w.cols + at.col) * kCh + 2 * lane, one, out);
        }
        *reinterpret_cast<float2*>(&s.carry[2 * lane]) = make_float2(carry[0], carry[1]);
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(&s.carried);
    }
}

// A finisher warp: run `run` of every second tile, from tile `group` on.
template <typename T, bool Aligned, bool Bwd, int NS>
__device__ __forceinline__ void scan_finish(const GlrArgs& a, const ScanWork& w, Stage<T, Aligned, Bwd>* ring,
                                            int group, int run)
{
    using S = Stage<T, Aligned, Bwd>;
    const int lane = threadIdx.x % 32, r0 = run * kSteps;
    const int dl = (int)(a.D % S::La::kPer16), dx = (int)(a.D % S::X::kPer16);
    for (int64_t q = group;; q += 2) {
        S& s = ring[q % NS];
        if (!umma::mbar_wait(&s.full, (uint32_t)((q / NS) & 1), a.err, kScanBit) || s.id < 0) return;
        const TileAt at(a, w, s.id, Bwd);
        const int live = (int)(a.T - at.t0 < kTile ? a.T - at.t0 : kTile) - r0;   // tokens of the run that exist
        const int64_t c = at.c0 + (Aligned ? 2 * lane : lane);
        const bool on0 = c < a.D, on1 = c + (Aligned ? 1 : 32) < a.D;
        F2 enter(0.f, 0.f);                      // backward: the kept entry state, asked for before the wait
        if constexpr (Bwd) enter = load_pair<Aligned>(a.starts + (at.b * w.tiles + at.i) * a.D + c, on0, on1);
        if (!umma::mbar_wait(&s.carried, (uint32_t)((q / NS) & 1), a.err, kScanBit)) return;
        const bool plain = !s.marked && live >= kSteps;
        int sl = S::La::shift(at.row0 + r0, a.D), sx = S::X::shift(at.row0 + r0, a.D);
        float h[2];
        if constexpr (!Bwd) {
            h[0] = s.carry[2 * lane];
            h[1] = s.carry[2 * lane + 1];
            for (int k = 0; k < run; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) h[e] = leave(s.A[k][2 * lane + e], s.B[k][2 * lane + e], h[e]);
            F2 H(h[0], h[1]);
            if (a.starts && run == 0 && live > 0 && !(s.marked && s.first[0] >= 0))
                store_pair<float, Aligned>(a.starts + (at.b * w.tiles + at.i) * a.D + c, on0, on1, H);
            T* out = (T*)a.out + (at.row0 + r0) * a.D + c;
            if (plain && a.out) {
#pragma unroll 4
                for (int k = 0; k < kSteps; ++k, out += a.D) {
                    H = fma2(S::La::get(s.la, r0 + k, sl, lane), H, S::X::get(s.x, r0 + k, sx, lane));
                    store_pair<T, Aligned>(out, on0, on1, H);
                    sl = (sl + dl) % S::La::kPer16;
                    sx = (sx + dx) % S::X::kPer16;
                }
            } else {
                for (int k = 0; k < live && k < kSteps; ++k, out += a.D) {
                    const int r = r0 + k;
                    const F2 l = S::La::get(s.la, r, sl, lane), x = S::X::get(s.x, r, sx, lane);
                    H = s.marked && s.first[r] >= 0 ? add2(l, x) : fma2(l, H, x);
                    if (a.out) store_pair<T, Aligned>(out, on0, on1, H);
                    const int n = s.marked && a.hT ? s.last[r] : -1;
                    if (n >= 0) {
                        const int64_t row = glr_row(a, n, false);
                        if (row >= 0) store_pair<float, Aligned>(a.hT + row * a.D + c, on0, on1, H);
                    }
                    sl = (sl + dl) % S::La::kPer16;
                    sx = (sx + dx) % S::X::kPer16;
                }
            }
        } else {
            // the state before every token of the run
            F2 before[kSteps];
            h[0] = enter.x();
            h[1] = enter.y();
            float g[2] = {s.carry[2 * lane], s.carry[2 * lane + 1]};     // c of the token behind
            for (int k = 0; k < run; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) h[e] = leave(s.fA[k][2 * lane + e], s.fB[k][2 * lane + e], h[e]);
            for (int k = kRuns - 1; k > run; --k)
#pragma unroll
                for (int e = 0; e < 2; ++e) g[e] = leave(s.A[k][2 * lane + e], s.B[k][2 * lane + e], g[e]);
            F2 H(h[0], h[1]), G(g[0], g[1]);
            if (plain) {
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    before[k] = H;
                    H = fma2(S::La::get(s.la, r0 + k, sl, lane), H, S::X::get(s.x, r0 + k, sx, lane));
                    sl = (sl + dl) % S::La::kPer16;
                    sx = (sx + dx) % S::X::kPer16;
                }
                T* to = (T*)a.dx + (at.row0 + r0 + kSteps - 1) * a.D + c;
                float* ta = a.dlog_a + (at.row0 + r0 + kSteps - 1) * a.D + c;
#pragma unroll
                for (int k = kSteps - 1; k >= 0; --k, to -= a.D, ta -= a.D) {
                    sl = (sl + S::La::kPer16 - dl) % S::La::kPer16;
                    sx = (sx + S::X::kPer16 - dx) % S::X::kPer16;
                    G = add2(G, S::X::get(s.y, r0 + k, sx, lane));
                    store_pair<T, Aligned>(to, on0, on1, G);
                    G = mul2(G, S::La::get(s.la, r0 + k, sl, lane));
                    store_pair<float, Aligned>(ta, on0, on1, mul2(G, before[k]));
                }
            } else {
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const int n = s.marked ? s.first[r0 + k] : -1;
                    if (n >= 0)
                        H = load_pair<Aligned>(a.h0 ? a.h0 + (int64_t)n * a.D + c : nullptr, on0, on1);
                    before[k] = H;
                    H = fma2(S::La::get(s.la, r0 + k, sl, lane), H, S::X::get(s.x, r0 + k, sx, lane));
                    sl = (sl + dl) % S::La::kPer16;
                    sx = (sx + dx) % S::X::kPer16;
                }
#pragma unroll
                for (int k = kSteps - 1; k >= 0; --k) {
                    sl = (sl + S::La::kPer16 - dl) % S::La::kPer16;
                    sx = (sx + S::X::kPer16 - dx) % S::X::kPer16;
                    if (k >= live) continue;
                    const int n = s.marked ? s.last[r0 + k] : -1;
                    if (n >= 0)
                        G = load_pair<Aligned>(a.dhT ? a.dhT + (int64_t)n * a.D + c : nullptr, on0, on1);
                    G = add2(G, S::X::get(s.y, r0 + k, sx, lane));
                    const int64_t to = (at.row0 + r0 + k) * a.D + c;
                    store_pair<T, Aligned>((T*)a.dx + to, on0, on1, G);
                    G = mul2(G, S::La::get(s.la, r0 + k, sl, lane));
                    store_pair<float, Aligned>(a.dlog_a + to, on0, on1, mul2(G, before[k]));
                    const int m = s.marked && a.dh0 ? s.first[r0 + k] : -1;
                    if (m >= 0) store_pair<float, Aligned>(a.dh0 + (int64_t)m * a.D + c, on0, on1, G);
                }
            }
        }
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(&s.empty);
    }
}

template <typename T, bool Aligned, bool Bwd>
__global__ void __launch_bounds__(scan_threads(Aligned), 1)
glr_scan_kernel(GlrArgs a, ScanWork w, const __grid_constant__ ScanMaps maps)
{
    griddep_wait();
    using S = Stage<T, Aligned, Bwd>;
    constexpr int NS = ring_stages<T, Aligned, Bwd>();
    static_assert(NS > kCarryWarps, "the ends take a stage each");
    extern __shared__ __align__(128) unsigned char smem[];
    S* ring = reinterpret_cast<S*>(smem);
    int warp = threadIdx.x / 32;
    if (threadIdx.x < NS) {
        S& s = ring[threadIdx.x];
        umma::mbar_init(&s.taken, 1);
        umma::mbar_init(&s.full, Aligned ? 2 : 1 + 32 * kCopyWarps);   // the marks, and the copies
        umma::mbar_init(&s.agg, kRuns);
        umma::mbar_init(&s.carried, 1);
        umma::mbar_init(&s.empty, kRuns);
        umma::fence_mbar_init();
    }
    __syncthreads();
    if (warp < kAggWarps) return scan_aggregate<T, Aligned, Bwd, NS>(a, w, ring, warp / kRuns, warp % kRuns);
    warp -= kAggWarps;
    if (warp < kFinWarps) return scan_finish<T, Aligned, Bwd, NS>(a, w, ring, warp / kRuns, warp % kRuns);
    warp -= kFinWarps;
    if (warp < kCarryWarps) return scan_carry<T, Aligned, Bwd, NS>(a, w, ring, warp);
    warp -= kCarryWarps;
    if (warp == 0) return scan_load<T, Aligned, Bwd, NS>(a, w, maps, ring);
    if constexpr (!Aligned) scan_copy<T, Bwd, NS>(a, w, ring, warp - 1);
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

template <typename T, bool Aligned, bool Bwd>
cudaError_t launch_scan(const GlrArgs& a, cudaStream_t st)
{
    ScanWork w = {};
    w.cols = a.B * ((a.D + kCh - 1) / kCh);
    w.tiles = (a.T + kTile - 1) / kTile;
    w.total = w.tiles * w.cols;
    StreamBuffer buf;
    // a single tile per column waits for nothing: no ticket, no setup, unless offsets or
    // sequences without tokens want looking at
    if (w.tiles > 1 || a.cu || a.T == 0) {
        const int64_t groups = (w.tiles + kGroup - 1) / kGroup;
        const int64_t words = (groups * w.cols + w.total) * kCh, ranges = (w.tiles + 1) / 2 * 2;
        const cudaError_t e = buf.alloc((size_t)(16 + (words + ranges) * 8), st);
        if (e != cudaSuccess) return e;
        w.ticket = static_cast<int*>(buf.ptr);
        w.entry = reinterpret_cast<unsigned long long*>(w.ticket + 4);
        w.tile_ab = w.entry + groups * w.cols * kCh;
        w.range = reinterpret_cast<int2*>(w.tile_ab + w.total * kCh);
        w.zeroed = 1 + words / 2;
        const int64_t work = w.zeroed / 8 + (a.cu ? w.tiles : 0) + (a.cu || a.T == 0 ? a.N * 32 : 0);
        const int64_t ctas = (work + 255) / 256;
        LaunchScope scope(st, K_GLR_SETUP);
        const cudaError_t s = launch_pdl(glr_setup_kernel, dim3((unsigned)(ctas < 296 ? ctas < 1 ? 1 : ctas : 296)),
                                         dim3(256), 0, st, a, w, Bwd ? 1 : 0);
        if (s != cudaSuccess) return s;
    }
    if (w.total == 0) return cudaSuccess;
    constexpr int smem = ring_stages<T, Aligned, Bwd>() * (int)sizeof(Stage<T, Aligned, Bwd>);
    const auto kernel = glr_scan_kernel<T, Aligned, Bwd>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ScanMaps maps = {};
    if (Aligned) {
        constexpr bool bf16 = sizeof(T) == 2;
        cudaError_t m = make_tensor_map_3d(&maps.la, a.log_a, false, a.D, a.T, a.B, kCh, kTile);
        if (m == cudaSuccess) m = make_tensor_map_3d(&maps.x, a.x, bf16, a.D, a.T, a.B, kCh, kTile);
        if (m == cudaSuccess && Bwd) m = make_tensor_map_3d(&maps.y, a.dout, bf16, a.D, a.T, a.B, kCh, kTile);
        if (m != cudaSuccess) return m;
    }
    LaunchScope scope(st, Bwd ? K_GLR_BWD : K_GLR_FWD);
    return launch_pdl(kernel, dim3((unsigned)(w.total < kSMs ? w.total : kSMs)), dim3(scan_threads(Aligned)), smem, st,
                      a, w, maps);
}

template <bool Bwd>
cudaError_t launch_scan_t(const GlrArgs& a, cudaStream_t st)
{
    if (a.io == KDA_IO_F32)
        return a.D % 4 == 0 ? launch_scan<float, true, Bwd>(a, st) : launch_scan<float, false, Bwd>(a, st);
    return a.D % 8 == 0 ? launch_scan<__nv_bfloat16, true, Bwd>(a, st) : launch_scan<__nv_bfloat16, false, Bwd>(a, st);
}

}  // namespace

cudaError_t launch_glr_fwd(const GlrArgs& a, cudaStream_t st) { return launch_scan_t<false>(a, st); }
cudaError_t launch_glr_bwd(const GlrArgs& a, cudaStream_t st) { return launch_scan_t<true>(a, st); }

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

// Rows, channels and tokens; `rows` = 1 with cu_seqlens.
kda_status_t glr_check_sizes(int64_t B, int64_t T, int64_t D, kda_io_dtype_t io, bool packed)
{
    if (B < 0 || T < 0 || D < 0) return KDA_ERR_INVALID_ARG;
    if (io != KDA_IO_F32 && io != KDA_IO_BF16) return KDA_ERR_UNSUPPORTED;
    if (D > kMaxChannels || B > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
    if (T > 0x7fffffffLL || (B > 0 && T > kMaxTokens / B)) return KDA_ERR_UNSUPPORTED;
    // tickets and offsets are 32-bit
    const int64_t cols = (packed ? 1 : B) * ((D + kCh - 1) / kCh);
    if (cols > 0 && (T + kTile - 1) / kTile > (0x7fffffffLL - 65536) / cols) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status_t glr_fwd_impl(const void* x, const float* log_a, const float* h0, void* out, float* hT,
                          float* starts, const int32_t* slots, int64_t P, const int32_t* cu,
                          int64_t B, int64_t T, int64_t D, kda_io_dtype_t io, cudaStream_t stream)
{
    const kda_status_t s = glr_check_sizes(B, T, D, io, cu != nullptr);
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
    const kda_status_t s = glr_check_sizes(B, T, D, io_dtype, cu_seqlens != nullptr);
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
