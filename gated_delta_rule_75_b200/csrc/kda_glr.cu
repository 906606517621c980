// Gated linear recurrence, h_t = exp(log_a_t) h_{t-1} + x_t per channel: the
// elementwise sibling of the delta rule (a vector state, the same per-channel
// decay), its gradients and its decode step.
//
// Scan.  A run of tokens maps the state it enters with affinely, h -> A h + B, and
// runs compose.  A tile is kTile tokens of kCh channels, cut into kRuns runs; the
// scan is one pass over memory, bound by it, with one persistent CTA per SM whose
// warps each do one part of the work for the tiles that pass through a ring of
// shared-memory stages:
//   loader       takes tiles and starts their TMA copies, a few tiles ahead;
//   aggregators  (groups of kRuns warps, tiles in turn) fold each run of the
//                tile into (A, B), and the runs into the tile's, and publish that;
//   carriers     (a warp per stage but one, tiles in turn) put the state that enters the
//                tile together, from when the tile is taken, of what earlier
//                tiles published: the state entering its group of kBlocks blocks of
//                kBlock tiles, then the (A, B) of the group's earlier blocks, then
//                those of the block's earlier tiles, in that order whatever arrives
//                first; the last tile of a block publishes the block's (A, B), or,
//                in the last block, the state that enters the next group;
//   finishers    (groups of kRuns warps) walk the runs again from their entry
//                states and write the outputs.
// So loads, arithmetic and the waits of different tiles overlap, a value is the same on
// every run, and the chain of waits is one hop per group.  CTA c takes tiles c, c + grid, ..
// (first tokens first; all CTAs are resident, by a cooperative launch) and works through
// them in that order: whatever a tile waits for comes before it in some CTA's order and
// waits for nothing later, so every wait ends (and is bounded all the same).  Handing tiles
// out by a counter instead lets a tile be taken long before it is loaded, and those
// behind it wait for it.
//
// Rows that do not start on 16 bytes.  TMA wants strides of 16 bytes: R = 2, 4 or 8 rows
// together have one, and the tensor is read as rows of R D elements.  A tile is then R
// boxes, one for each place of a token in such a row, that start on the 16-byte boundary
// before its channels and are 16 bytes wider.  The last tokens of the tensor, fewer than R,
// are read by the workers themselves.
//
// Sequences: a token that begins one replaces the state by h0, whatever came before it
// (a NaN too): A = -1 there, and a run whose A is negative is h -> B.
//
// Backward.  With c_t = exp(log_a_t) g_t, g_t = dout_t + c_{t+1}: the same scan over
// tiles from the last to the first, replaced by dhT at a sequence's last token.
// dlog_a_t = c_t h_{t-1} needs the forward states too; they are walked again inside
// the tile from its kept entry state (starts), so the pass reads x, log_a, dout and
// writes dx, dlog_a once.
//
// Measured (copies run at 6.46 TB/s): 8 x 8192 x 4096 bf16, 2.15 GB, 380 us when the SM clock is at
// its top and 440 under the power cap (1660 MHz); 131071 x 1024 fp32, 1.61 GB, 293 us (316); 8 x 8192 x
// 4096 in registers, a CTA a tile, 644.  Tiles of 64 x 64: their ring (8 stages of 28 KiB for bf16)
// keeps about 190 KiB of an SM on its way or in work for the 5 us from a tile's copy to its last store.
#include "kda_common.cuh"
#include "kda_f32x2.cuh"
#include "kda_internal.h"
#include "kda_tma.cuh"
#include "kda_umma.cuh"

namespace kda {

constexpr int kTile = KDA_GLR_TILE;     // tokens of a tile
constexpr int kCh = 64;                 // channels of a tile, two a lane
constexpr int kRuns = 4;                // runs of a tile, one a warp
constexpr int kSteps = kTile / kRuns;   // tokens of a run
constexpr int kBlock = 8;               // tiles of a block
constexpr int kBlocks = 8;              // blocks of a group
static_assert(kBlocks <= kBlock, "words of a group and of a block are held in the same registers");
constexpr int kPolls = 1 << 21;         // about two seconds of polling
constexpr int kScanBit = 7;             // kErrScanWait; its waits are a whole warp's, 4 us a poll, so 80 ms in all

// Warps by role.
constexpr int kFinGroups = 2, kFinWarps = kFinGroups * kRuns;
constexpr int agg_groups(bool bwd) { return bwd ? 2 : 3; }
constexpr int carry_warps(int stages) { return stages - 1; }
constexpr int scan_threads(int stages, bool bwd)
{
    return 32 * (agg_groups(bwd) * kRuns + kFinWarps + carry_warps(stages) + 1);
}

// n / d for 0 <= n < 2^31 as (n m) >> s: with 2^k >= d, s = 31 + k and m = ceil(2^s / d), n m / 2^s is n / d
// and less than n / 2^s < 2^-k <= 1 / d more, which reaches no further integer.
struct Divide {
    uint32_t m, s;
    Divide() = default;
    explicit Divide(int64_t d)
    {
        uint32_t k = 0;
        while ((int64_t(1) << k) < d) ++k;
        s = 31 + k;
        m = (uint32_t)(((uint64_t(1) << s) + (uint64_t)d - 1) / (uint64_t)d);
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (uint32_t)(((uint64_t)n * m) >> s); }
};

// Workspace: for every group its entry state and the (A, B) of its blocks but the last, which the next
// group's entry state holds, side by side so that one wait asks for them together (a row of words for
// every block; none for a single one, which nothing crosses); the tiles' (A, B).  All zeroed by
// the setup kernel; with cu_seqlens each tile's range of offsets.  A column is one block of kCh
// channels of one row of the token axis; tiles, blocks and groups are numbered in the order of
// the scan (from the end in the backward).
struct ScanWork {
    unsigned long long* groups;    // [blocks][cols][kCh]: of a group words (1, entry state), then (A, B) of blocks
    unsigned long long* tile_ab;   // [tiles][cols][kCh]: words (A, B)
    int2* range;                   // [tiles]: offsets cu[x .. y - 1] lie in [first token, first + kTile]
    int64_t cols, tiles, total;    // total = tiles * cols
    Divide by_cols, by_blocks;     // by cols, and by the columns of one row
    int64_t zeroed;                // 16-byte words from groups on
    uint32_t blocks;               // columns of one row
    int log_r;                     // R = 1 << log_r rows of the tensor are one row of the tensor maps
    int64_t mapped;                // tokens (over all rows) that the tensor maps cover
};

// Published words, two channels at once: the complement of A, whose bits are not all ones (arithmetic makes
// no such NaN), so that a word of zeros is one that is not there yet, and B in the high half.  Both come
// back bit for bit: a memory without decay passes thousands of tiles.  Each word is read and written whole,
// so B comes with its A and nothing else has to be ordered.
__device__ __forceinline__ void load_words(const unsigned long long* p, unsigned long long& a, unsigned long long& b)
{
    asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "l"(p) : "memory");
}
__device__ __forceinline__ unsigned long long word_of(float A, float B)
{
    return ((unsigned long long)__float_as_uint(B) << 32) | max(~__float_as_uint(A), 1u);
}
__device__ __forceinline__ bool word_there(unsigned long long w) { return (unsigned)w != 0; }
__device__ __forceinline__ float word_A(unsigned long long w) { return __uint_as_float(~(unsigned)w); }
__device__ __forceinline__ float word_B(unsigned long long w) { return __uint_as_float((unsigned)(w >> 32)); }
__device__ __forceinline__ void store_words(unsigned long long* p, const float (&A)[2], const float (&B)[2])
{
    asm volatile("st.relaxed.gpu.global.v2.u64 [%0], {%1, %2};" ::"l"(p), "l"(word_of(A[0], B[0])), "l"(word_of(A[1], B[1]))
                 : "memory");
}

// exp of two logarithms of decays, within a half step and little more.  The hardware's exponential is
// cheaper, but its errors lean one way and a long memory adds them up (131071 x 1024 fp32: h 5.7e-7 off
// instead of 1.3e-7).  x = n ln 2 + r with |r| <= ln 2 / 2 (ln 2 in two parts, so that r loses nothing);
// e^r = 1 + r + r^2 g(r), g by interpolation of degree 4 at the Chebyshev points of that interval (0.2
// half steps off); times 2^n.  n = -127, where x is cut off (-inf too), makes the scale and the decay 0;
// NaN stays.
__device__ __forceinline__ F2 decay2(F2 l)
{
    constexpr float log2e = 1.4426950408889634f, ln2_hi = 0.693145751953125f,      // 15 bits: n ln2_hi is exact
        ln2_lo = (float)(0.69314718055994531 - 0.693145751953125), magic = 12582912.f,     // 1.5 * 2^23: rounds
        least = (float)(-127 * 0.69314718055994531);
    float a, b;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(l.x()), "f"(least));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(b) : "f"(l.y()), "f"(least));
    const F2 x(a, b), m = fma2(x, both(log2e), both(magic)), n = add2(m, both(-magic));
    const F2 r = fma2(n, both(-ln2_lo), fma2(n, both(-ln2_hi), x));
    F2 p = fma2(r, both(0.0013926198f), both(0.00836319f));
    p = fma2(p, r, both(0.041666556f));
    p = fma2(p, r, both(0.16666576f));
    p = fma2(p, r, both(0.5f));
    p = fma2(p, r, both(1.f));
    p = fma2(p, r, both(1.f));
    // the low bits of m are n; n + 127 is the scale's exponent
    return mul2(p, F2(__int_as_float((__float_as_int(m.x()) << 23) + 0x3f800000),
                      __int_as_float((__float_as_int(m.y()) << 23) + 0x3f800000)));
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

// How rows lie.  kWhole: they start on 16 bytes; a tile is kTile rows of kCh elements.  Otherwise it is R
// boxes of kTile / R rows, and the offset of a token's channel 0 is looked up (Stage::off).  Lane l owns
// channels 2 l, 2 l + 1 as one access, or, where D is odd (kSingle), channels l, l + 32.  (bf16, 100000
// tokens of 1024, 1022, 1023 channels: 168, 208, 232 us.)
constexpr int kSingle = 0, kPairs = 1, kWhole = 2;
template <typename E, int Mode>
struct Rows {
    static constexpr int kBytes = kCh * (int)sizeof(E);
    static constexpr int kPitch = kBytes + (Mode == kWhole ? 0 : 16);
    static constexpr int kPer16 = 16 / (int)sizeof(E);

    // The lane's two channels of the row at `at` bytes.
    static __device__ __forceinline__ F2 get(const unsigned char* base, int at, int lane)
    {
        const E* p = reinterpret_cast<const E*>(base + at);
        if constexpr (Mode == kSingle) return F2(IO<E>::load(p, lane), IO<E>::load(p, lane + 32));
        if constexpr (sizeof(E) == 4) {
            F2 v;
            v.v = reinterpret_cast<const unsigned long long*>(p)[lane];
            return v;
        } else {
            const uint32_t u = reinterpret_cast<const uint32_t*>(p)[lane];
            return F2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
        }
    }
    static __device__ __forceinline__ void put(unsigned char* base, int at, int lane, F2 v)
    {
        static_assert(sizeof(E) == 4, "decays only");
        float* p = reinterpret_cast<float*>(base + at);
        if constexpr (Mode != kSingle) {
            reinterpret_cast<unsigned long long*>(p)[lane] = v.v;
        } else {
            p[lane] = v.x();
            p[lane + 32] = v.y();
        }
    }
    // The same from the tensor itself.
    static __device__ __forceinline__ F2 direct(const E* at, bool on0, bool on1)
    {
        return F2(on0 ? IO<E>::load(at, 0) : 0.f, on1 ? IO<E>::load(at, Mode != kSingle ? 1 : 32) : 0.f);
    }
};

// The lane's two channels, from c0, of a row of a tensor in global memory; on0, on1: which of
// them exist (of a pair both or none).
template <typename E, int Mode>
__device__ __forceinline__ void store_pair(E* at, bool on0, bool on1, F2 v)
{
    if constexpr (Mode != kSingle) {
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
template <int Mode>
__device__ __forceinline__ F2 load_pair(const float* at, bool on0, bool on1)
{
    return F2(at && on0 ? at[0] : 0.f, at && on1 ? at[Mode != kSingle ? 1 : 32] : 0.f);
}

// Tokens of a row that are in a sequence: with cu_seqlens (one row) those behind the last sequence
// are not, and are neither worked on nor written.
__device__ __forceinline__ int64_t tokens_used(const GlrArgs& a)
{
    if (a.cu == nullptr) return a.T;
    const int64_t n = a.cu[a.N];
    return n < 0 ? 0 : n < a.T ? n : a.T;
}

// One stage of the ring.
template <typename T, int Mode, bool Bwd>
struct Stage {
    using La = Rows<float, Mode>;
    using X = Rows<T, Mode>;
    alignas(128) unsigned char la[kTile * La::kPitch];           // log_a, then exp(log_a)
    alignas(128) unsigned char x[kTile * X::kPitch];
    alignas(128) unsigned char y[Bwd ? kTile * X::kPitch : 128]; // dout
    float A[kRuns][kCh], B[kRuns][kCh];                          // runs in the scan's direction
    float fA[Bwd ? kRuns : 1][kCh], fB[Bwd ? kRuns : 1][kCh];    // backward: the forward runs too
    float tA[kCh], tB[kCh], carry[kCh];                          // the tile; what enters it
    int first[kTile], last[kTile];                               // sequences that begin / end there, or -1
    int off[Mode == kWhole ? 1 : kTile];                                // bytes of a token's channel 0: la | x << 16
    int64_t id;                                                  // tile * cols + column; -1: no more
    int marked;                                                  // whether first / last hold anything
    int plain;                                                   // no marks, all tokens there and in the maps
    int folded;                                                  // runs that are there
    uint64_t taken, full, agg, carried, empty;                   // full: the copies, and the loader's notes
    static constexpr uint32_t kCopied = kTile * (La::kPitch + X::kPitch * (Bwd ? 2 : 1));

    __device__ __forceinline__ int la_at(int r) const { return Mode == kWhole ? r * La::kPitch : off[r] & 0xffff; }
    __device__ __forceinline__ int x_at(int r) const { return Mode == kWhole ? r * X::kPitch : (int)((uint32_t)off[r] >> 16); }
};
template <typename T, int Mode, bool Bwd> constexpr int ring_stages()
{
    constexpr int n = (int)((227 * 1024 - 64) / sizeof(Stage<T, Mode, Bwd>));
    return n < 8 ? n : 8;
}

// A worker's wait for its tile q in stage q % NS.  A barrier tells phases apart by their parity alone, so a
// wait may only begin once the phase before has ended; copies land in any order, and a group that takes
// every third tile may be done with tile q - 3 while tile q - NS is still on its way to the stage.  The loader
// goes in order: the wait for `taken` may begin once tile q - NS was taken, which the worker's last tile, a later one,
// shows, and it ends after tile q - NS has left the stage, which ends its phase of `full`.
template <typename S>
__device__ __forceinline__ bool await_tile(S& s, uint32_t parity, int* err)
{
    return umma::mbar_wait(&s.taken, parity, err, kScanBit) && umma::mbar_wait(&s.full, parity, err, kScanBit) && s.id >= 0;
}

// Where a tile lies (tiles, columns and their product fit 31 bits).
struct TileAt {
    uint32_t order, col, i;                      // order: in the scan; i: on the token axis
    int64_t b, t0, row0, c0;                     // row0 = b * T + t0
    __device__ __forceinline__ TileAt(const GlrArgs& a, const ScanWork& w, int64_t id, bool bwd)
    {
        order = w.by_cols((uint32_t)id);
        col = (uint32_t)id - order * (uint32_t)w.cols;
        i = bwd ? (uint32_t)w.tiles - 1 - order : order;
        const uint32_t row = w.by_blocks(col);
        b = row;
        c0 = (int64_t)(col - row * w.blocks) * kCh;
        t0 = (int64_t)i * kTile;
        row0 = b * a.T + t0;
    }
};

// Before a scan: zeroes the published words, finds every tile's offsets, checks
// the offsets, and passes the states of sequences without tokens on.
__global__ void __launch_bounds__(256) glr_setup_kernel(GlrArgs a, ScanWork w, int bwd)
{
    griddep_wait();
    griddep_launch_dependents();
    const int64_t me = (int64_t)blockIdx.x * 256 + threadIdx.x, all = (int64_t)gridDim.x * 256;
    for (int64_t k = me; k < w.zeroed; k += all) reinterpret_cast<uint4*>(w.groups)[k] = make_uint4(0, 0, 0, 0);
    if (a.cu) {
        // few offsets are searched in shared memory: one trip to memory, not one per step
        constexpr int kHeld = 4096;
        __shared__ int32_t held[kHeld];
        const bool hold = a.N < kHeld;
        if (hold)
            for (int64_t n = threadIdx.x; n <= a.N; n += 256) held[n] = a.cu[n];
        __syncthreads();
        const int32_t* cu = hold ? held : a.cu;
        for (int64_t i = me; i < w.tiles; i += all) {
            int at[2];
            for (int k = 0; k < 2; ++k) {
                const int64_t bound = i * kTile + (k ? kTile + 1 : 0);
                int64_t lo = 0, hi = a.N + 1;    // first index with cu[index] >= bound
                while (lo < hi) {
                    const int64_t mid = (lo + hi) >> 1;
                    if (cu[mid] < bound) lo = mid + 1; else hi = mid;
                }
                at[k] = (int)lo;
            }
            w.range[i] = make_int2(at[0], at[1]);
        }
        for (int64_t n = me; n < a.N; n += all)
            if (cu[n + 1] < cu[n] || (n == 0 && (cu[0] != 0 || cu[a.N] != a.T))) atomicOr(a.err, kErrSeqlens);
    }
    const float* from = bwd ? a.dhT : a.h0;
    float* to = bwd ? a.dh0 : a.hT;
    if ((!a.cu && a.T > 0) || to == nullptr) return;
    for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x) {      // a CTA a sequence
        if (a.cu && a.cu[n + 1] > a.cu[n]) continue;
        const int64_t row = bwd ? n : glr_row(a, n, threadIdx.x == 0);
        if (row < 0 || to == from) continue;
        for (int64_t c = threadIdx.x; c < a.D; c += 256) to[row * a.D + c] = from ? from[row * a.D + c] : 0.f;
    }
}

// Tensor maps of log_a, x and dout.
struct ScanMaps {
    CUtensorMap la, x, y;
};

// The loader: one warp.
template <typename T, int Mode, bool Bwd, int NS>
__device__ __forceinline__ void scan_load(const GlrArgs& a, const ScanWork& w, const ScanMaps& maps,
                                          Stage<T, Mode, Bwd>* ring)
{
    using S = Stage<T, Mode, Bwd>;
    const int lane = threadIdx.x % 32;
    const int R = Mode == kWhole ? 1 : 1 << w.log_r;
    const int64_t used = tokens_used(a);
    int64_t next = blockIdx.x;
    int ends = 0;
    for (int64_t q = 0; ends < carry_warps(NS); ++q, next += gridDim.x) {
        S& s = ring[q % NS];
        const int64_t id = next < w.total ? next : -1;
        const TileAt at(a, w, id < 0 ? 0 : id, Bwd);
        int2 range = make_int2(0, 0);
        if (a.cu && id >= 0) range = w.range[at.i];
        if (q >= NS && !umma::mbar_wait(&s.empty, (uint32_t)((q / NS - 1) & 1), a.err, kScanBit)) {
            // given up: the copies under way have to land before the CTA may end
            for (int64_t k = q - NS; k < q; ++k)
                umma::mbar_wait(&ring[k % NS].full, (uint32_t)((k / NS) & 1), a.err, kScanBit);
            return;
        }
        const bool copies = id >= 0 && w.mapped > 0;
        if (lane == 0) {
            s.id = id;
            s.folded = 0;
            umma::mbar_arrive(&s.taken);
            if (copies) tma::expect_tx(&s.full, S::kCopied);
            else umma::mbar_arrive(&s.full);
        }
        __syncwarp();
        if (copies && lane < R) {
            // the box of tokens whose index over all rows is `lane` modulo R
            const int64_t row = (at.row0 - lane + R - 1) >> (Mode == kWhole ? 0 : w.log_r);
            const int64_t x0 = lane * a.D + at.c0;
            const int box = kTile / R;
            const int32_t xa = (int32_t)(x0 & ~(int64_t)(S::La::kPer16 - 1)), xx = (int32_t)(x0 & ~(int64_t)(S::X::kPer16 - 1));
            tma::load_2d(s.la + lane * box * S::La::kPitch, &maps.la, Mode == kWhole ? (int32_t)x0 : xa, (int32_t)row, &s.full);
            tma::load_2d(s.x + lane * box * S::X::kPitch, &maps.x, Mode == kWhole ? (int32_t)x0 : xx, (int32_t)row, &s.full);
            if constexpr (Bwd)
                tma::load_2d(s.y + lane * box * S::X::kPitch, &maps.y, Mode == kWhole ? (int32_t)x0 : xx, (int32_t)row, &s.full);
        }
        if (id < 0) {
            ++ends;                              // one for every worker that takes tiles in turn
        } else {
            if constexpr (Mode != kWhole)
                for (int r = lane; r < kTile; r += 32) {
                    const int place = (int)((at.row0 + r) & (R - 1));
                    const int slot = place * (kTile >> w.log_r) + (r >> w.log_r);
                    const int shift = (int)((place * a.D) & 7);
                    s.off[r] = (slot * S::La::kPitch + (shift & (S::La::kPer16 - 1)) * 4) |
                               (slot * S::X::kPitch + (shift & (S::X::kPer16 - 1)) * (int)sizeof(T)) << 16;
                }
            // sequences that begin or end in the tile
            const bool begins = !a.cu && at.t0 == 0, ends_here = !a.cu && at.t0 + kTile >= a.T;
            const bool marked = a.cu ? range.y > range.x : begins || ends_here;
            if (lane == 0) {
                s.marked = marked;
                s.plain = !marked && at.t0 + kTile <= used && at.row0 + kTile <= w.mapped;
            }
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
    }
}

// An aggregator warp: run `run` of one tile of agg_groups(Bwd), from tile `group` on.
template <typename T, int Mode, bool Bwd, int NS>
__device__ __forceinline__ void scan_aggregate(const GlrArgs& a, const ScanWork& w, Stage<T, Mode, Bwd>* ring,
                                               int group, int run)
{
    using S = Stage<T, Mode, Bwd>;
    const int lane = threadIdx.x % 32, r0 = run * kSteps;
    const int64_t used = tokens_used(a);
    for (int64_t q = group;; q += agg_groups(Bwd)) {
        S& s = ring[q % NS];
        if (!await_tile(s, (uint32_t)((q / NS) & 1), a.err)) return;
        const TileAt at(a, w, s.id, Bwd);
        F2 A(1.f, 1.f), B(0.f, 0.f);
        if (s.plain) {
#pragma unroll 4
            for (int k = 0; k < kSteps; ++k) {
                const int la = s.la_at(r0 + k);
                const F2 l = decay2(S::La::get(s.la, la, lane));
                A = mul2(A, l);
                B = fma2(l, B, S::X::get(s.x, s.x_at(r0 + k), lane));
                S::La::put(s.la, la, lane, l);   // the finishers take the decay from here
            }
            if constexpr (Bwd) {
                *reinterpret_cast<F2*>(&s.fA[run][2 * lane]) = A;
                *reinterpret_cast<F2*>(&s.fB[run][2 * lane]) = B;
                // the product of the decays is the same from either end but for its rounding
                B = F2(0.f, 0.f);
#pragma unroll 4
                for (int k = kSteps - 1; k >= 0; --k)
                    B = mul2(S::La::get(s.la, s.la_at(r0 + k), lane), add2(B, S::X::get(s.y, s.x_at(r0 + k), lane)));
            }
        } else {
            const int live = (int)(used - at.t0 < kTile ? used - at.t0 : kTile);   // tokens that exist (or less than none)
            const int64_t c = at.c0 + (Mode != kSingle ? 2 * lane : lane);
            const bool on0 = c < a.D, on1 = c + (Mode != kSingle ? 1 : 32) < a.D;
            for (int r = r0; r < r0 + kSteps && r < live; ++r) {
                const bool in = at.row0 + r < w.mapped;
                const int64_t e = (at.row0 + r) * a.D + c;
                F2 l = decay2(in ? S::La::get(s.la, s.la_at(r), lane) : S::La::direct(a.log_a + e, on0, on1));
                const F2 x = in ? S::X::get(s.x, s.x_at(r), lane) : S::X::direct((const T*)a.x + e, on0, on1);
                const int n = s.marked ? s.first[r] : -1;
                if (n >= 0) {
                    const int64_t row = Bwd ? n : glr_row(a, n, lane == 0 && at.c0 == 0);
                    const F2 h0 = load_pair<Mode>(a.h0 && row >= 0 ? a.h0 + row * a.D + c : nullptr, on0, on1);
                    A = F2(-1.f, -1.f);
                    B = add2(mul2(l, h0), x);
                    if constexpr (!Bwd) {
                        // the finishers find exp(log_a) h0 here: hT may be written over h0 before they come
                        l = mul2(l, h0);
                        if (a.starts && r == 0)
                            store_pair<float, Mode>(a.starts + (at.b * w.tiles + at.i) * a.D + c, on0, on1, h0);
                    }
                } else {
                    A = mul2(A, l);
                    B = fma2(l, B, x);
                }
                S::La::put(s.la, s.la_at(r), lane, l);
            }
            if constexpr (Bwd) {
                *reinterpret_cast<F2*>(&s.fA[run][2 * lane]) = A;
                *reinterpret_cast<F2*>(&s.fB[run][2 * lane]) = B;
                A = F2(1.f, 1.f);
                B = F2(0.f, 0.f);
                for (int r = (live < r0 + kSteps ? live : r0 + kSteps) - 1; r >= r0; --r) {
                    const int n = s.marked ? s.last[r] : -1;
                    if (n >= 0) {
                        A = F2(-1.f, -1.f);
                        B = load_pair<Mode>(a.dhT ? a.dhT + (int64_t)n * a.D + c : nullptr, on0, on1);
                    }
                    const F2 l = S::La::get(s.la, s.la_at(r), lane);
                    const F2 y = at.row0 + r < w.mapped
                                     ? S::X::get(s.y, s.x_at(r), lane)
                                     : S::X::direct((const T*)a.dout + (at.row0 + r) * a.D + c, on0, on1);
                    A = mul2(A, l);
                    B = mul2(l, add2(B, y));
                }
            }
        }
        *reinterpret_cast<F2*>(&s.A[run][2 * lane]) = A;
        *reinterpret_cast<F2*>(&s.B[run][2 * lane]) = B;
        // the decays written over log_a come before the TMA copy that fills the stage again
        umma::fence_smem_to_async();
        // the last of the tile's runs to be there folds them
        __syncwarp();
        int before = 0;
        if (lane == 0) {
            __threadfence_block();
            before = atomicAdd(&s.folded, 1);
            __threadfence_block();
        }
        if (__shfl_sync(0xffffffffu, before, 0) == kRuns - 1) {
            __syncwarp();                        // what lane 0 has seen of the other runs holds for all lanes
            float tA[2] = {1.f, 1.f}, tB[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kRuns; ++k) {
                const int from = Bwd ? kRuns - 1 - k : k;
                const float2 ra = *reinterpret_cast<const float2*>(&s.A[from][2 * lane]);
                const float2 rb = *reinterpret_cast<const float2*>(&s.B[from][2 * lane]);
                tB[0] = leave(ra.x, rb.x, tB[0]);
                tB[1] = leave(ra.y, rb.y, tB[1]);
                tA[0] = chain(tA[0], ra.x);
                tA[1] = chain(tA[1], ra.y);
            }
            *reinterpret_cast<float2*>(&s.tA[2 * lane]) = make_float2(tA[0], tA[1]);
            *reinterpret_cast<float2*>(&s.tB[2 * lane]) = make_float2(tB[0], tB[1]);
            if (at.order + 1 < w.tiles && at.order % kBlock != kBlock - 1)
                store_words(w.tile_ab + ((int64_t)at.order * w.cols + at.col) * kCh + 2 * lane, tA, tB);
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(&s.agg);
        }
    }
}

// `count` (at most N) published words from p on, `pitch` apart: asked for together, and those that
// are not there yet again together, so that the wait is a few round trips however many are late.
template <int N>
__device__ __forceinline__ void await_words(const unsigned long long* p, int64_t pitch, int count,
                                            unsigned long long (&a)[N], unsigned long long (&b)[N], int* err)
{
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (k < count) load_words(p + k * pitch, a[k], b[k]);
    for (int polls = 0;; ++polls) {
        bool there = true;
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (k < count) there = there && word_there(a[k]) && word_there(b[k]);
        if (__all_sync(0xffffffffu, there)) return;
        if (polls >= kPolls) {
            if (err) atomicOr(err, kErrScanWait);
            return;
        }
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (k < count && !(word_there(a[k]) && word_there(b[k]))) load_words(p + k * pitch, a[k], b[k]);
    }
}
// The run (A, B) followed by a published one.
__device__ __forceinline__ void append(float (&A)[2], float (&B)[2], unsigned long long a, unsigned long long b)
{
    B[0] = leave(word_A(a), word_B(a), B[0]);
    B[1] = leave(word_A(b), word_B(b), B[1]);
    A[0] = chain(A[0], word_A(a));
    A[1] = chain(A[1], word_A(b));
}

// A carrier warp: one tile of carry_warps(NS), from tile `from` on.
template <typename T, int Mode, bool Bwd, int NS>
__device__ __forceinline__ void scan_carry(const GlrArgs& a, const ScanWork& w, Stage<T, Mode, Bwd>* ring, int from)
{
    using S = Stage<T, Mode, Bwd>;
    const int lane = threadIdx.x % 32;
    for (int64_t q = from;; q += carry_warps(NS)) {
        S& s = ring[q % NS];
        if (!umma::mbar_wait(&s.taken, (uint32_t)((q / NS) & 1), a.err, kScanBit) || s.id < 0) return;
        const TileAt at(a, w, s.id, Bwd);
        const int64_t block = at.order / kBlock, g = block / kBlocks, lane2 = at.col * kCh + 2 * lane;
        const int blocks = (int)(block % kBlocks), behind = (int)(at.order % kBlock);   // earlier ones of the group, the block
        const bool more = at.order + 1 < w.tiles, last = behind == kBlock - 1;
        const int64_t pitch = w.cols * kCh;
        unsigned long long v0[kBlock], v1[kBlock];
        // the block's earlier tiles as one run
        float rA[2] = {1.f, 1.f}, rB[2] = {0.f, 0.f};
        if (behind > 0) {
            await_words(w.tile_ab + block * kBlock * pitch + lane2, pitch, behind, v0, v1, a.err);
#pragma unroll
            for (int k = 0; k < kBlock - 1; ++k)
                if (k < behind) append(rA, rB, v0[k], v1[k]);
        }
        if (!umma::mbar_wait(&s.agg, (uint32_t)((q / NS) & 1), a.err, kScanBit)) return;
        const float2 tA = *reinterpret_cast<const float2*>(&s.tA[2 * lane]);
        const float2 tB = *reinterpret_cast<const float2*>(&s.tB[2 * lane]);
        const float A[2] = {tA.x, tA.y}, B[2] = {tB.x, tB.y};
        unsigned long long* group = w.groups + g * kBlocks * pitch + lane2;
        if (more && last && blocks < kBlocks - 1) {
            const float bA[2] = {chain(rA[0], A[0]), chain(rA[1], A[1])};
            const float bB[2] = {leave(A[0], B[0], rB[0]), leave(A[1], B[1], rB[1])};
            store_words(group + (blocks + 1) * pitch, bA, bB);
        }
        // the group's entry state (the first group has none), its earlier blocks, then the run
        const int none = g == 0 ? 1 : 0, count = blocks + 1 - none;
        float carry[2] = {0.f, 0.f};
        if (count > 0) {
            await_words(group + none * pitch, pitch, count, v0, v1, a.err);
            float pA[2] = {1.f, 1.f}, pB[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kBlocks; ++k)
                if (k < count && k + none > 0) append(pA, pB, v0[k], v1[k]);
            if (none == 0) {
                carry[0] = word_B(v0[0]);
                carry[1] = word_B(v1[0]);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                rB[e] = leave(rA[e], rB[e], pB[e]);
                rA[e] = chain(pA[e], rA[e]);
            }
        }
        carry[0] = leave(rA[0], rB[0], carry[0]);
        carry[1] = leave(rA[1], rB[1], carry[1]);
        if (more && last && blocks == kBlocks - 1) {
            const float one[2] = {1.f, 1.f}, out[2] = {leave(A[0], B[0], carry[0]), leave(A[1], B[1], carry[1])};
            store_words(group + kBlocks * pitch, one, out);
        }
        *reinterpret_cast<float2*>(&s.carry[2 * lane]) = make_float2(carry[0], carry[1]);
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(&s.carried);
    }
}

// A finisher warp: run `run` of one tile of kFinGroups, from tile `group` on.
template <typename T, int Mode, bool Bwd, int NS>
__device__ __forceinline__ void scan_finish(const GlrArgs& a, const ScanWork& w, Stage<T, Mode, Bwd>* ring,
                                            int group, int run)
{
    using S = Stage<T, Mode, Bwd>;
    const int lane = threadIdx.x % 32, r0 = run * kSteps;
    const int64_t used = tokens_used(a);
    for (int64_t q = group;; q += kFinGroups) {
        S& s = ring[q % NS];
        if (!await_tile(s, (uint32_t)((q / NS) & 1), a.err)) return;
        const TileAt at(a, w, s.id, Bwd);
        const int live = (int)(used - at.t0 < kTile ? used - at.t0 : kTile);     // tokens that exist (or less than none)
        const int64_t c = at.c0 + (Mode != kSingle ? 2 * lane : lane);
        const bool on0 = c < a.D, on1 = c + (Mode != kSingle ? 1 : 32) < a.D;
        F2 enter(0.f, 0.f);                      // backward: the kept entry state, asked for before the wait
        if constexpr (Bwd) enter = load_pair<Mode>(a.starts + (at.b * w.tiles + at.i) * a.D + c, on0, on1);
        if (!umma::mbar_wait(&s.carried, (uint32_t)((q / NS) & 1), a.err, kScanBit)) return;
        const bool marked = s.marked != 0;
        // x or dout of a token
        const auto value = [&](const unsigned char* stage, const void* tensor, int r) {
            return at.row0 + r < w.mapped ? S::X::get(stage, s.x_at(r), lane)
                                          : S::X::direct((const T*)tensor + (at.row0 + r) * a.D + c, on0, on1);
        };
        float h[2];
        if constexpr (!Bwd) {
            h[0] = s.carry[2 * lane];
            h[1] = s.carry[2 * lane + 1];
            for (int k = 0; k < run; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) h[e] = leave(s.A[k][2 * lane + e], s.B[k][2 * lane + e], h[e]);
            F2 H(h[0], h[1]);
            if (a.starts && run == 0 && !(marked && s.first[0] >= 0))
                store_pair<float, Mode>(a.starts + (at.b * w.tiles + at.i) * a.D + c, on0, on1, H);
            T* out = (T*)a.out + (at.row0 + r0) * a.D + c;
            if (s.plain && a.out) {
#pragma unroll 4
                for (int r = r0; r < r0 + kSteps; ++r, out += a.D) {
                    H = fma2(S::La::get(s.la, s.la_at(r), lane), H, S::X::get(s.x, s.x_at(r), lane));
                    store_pair<T, Mode>(out, on0, on1, H);
                }
            } else {
                for (int r = r0; r < live && r < r0 + kSteps; ++r, out += a.D) {
                    const F2 l = S::La::get(s.la, s.la_at(r), lane), x = value(s.x, a.x, r);
                    H = marked && s.first[r] >= 0 ? add2(l, x) : fma2(l, H, x);
                    if (a.out) store_pair<T, Mode>(out, on0, on1, H);
                    const int n = marked && a.hT ? s.last[r] : -1;
                    if (n >= 0) {
                        const int64_t row = glr_row(a, n, false);
                        if (row >= 0) store_pair<float, Mode>(a.hT + row * a.D + c, on0, on1, H);
                    }
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
            if (s.plain) {
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    before[k] = H;
                    H = fma2(S::La::get(s.la, s.la_at(r0 + k), lane), H, S::X::get(s.x, s.x_at(r0 + k), lane));
                }
                T* to = (T*)a.dx + (at.row0 + r0 + kSteps - 1) * a.D + c;
                float* ta = a.dlog_a + (at.row0 + r0 + kSteps - 1) * a.D + c;
#pragma unroll
                for (int k = kSteps - 1; k >= 0; --k, to -= a.D, ta -= a.D) {
                    G = add2(G, S::X::get(s.y, s.x_at(r0 + k), lane));
                    store_pair<T, Mode>(to, on0, on1, G);
                    G = mul2(G, S::La::get(s.la, s.la_at(r0 + k), lane));
                    store_pair<float, Mode>(ta, on0, on1, mul2(G, before[k]));
                }
            } else {
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const int r = r0 + k;
                    if (r >= live) break;
                    const int n = marked ? s.first[r] : -1;
                    if (n >= 0)
                        H = load_pair<Mode>(a.h0 ? a.h0 + (int64_t)n * a.D + c : nullptr, on0, on1);
                    before[k] = H;
                    H = fma2(S::La::get(s.la, s.la_at(r), lane), H, value(s.x, a.x, r));
                }
#pragma unroll
                for (int k = kSteps - 1; k >= 0; --k) {
                    const int r = r0 + k;
                    if (r >= live) continue;
                    const int n = marked ? s.last[r] : -1;
                    if (n >= 0)
                        G = load_pair<Mode>(a.dhT ? a.dhT + (int64_t)n * a.D + c : nullptr, on0, on1);
                    G = add2(G, value(s.y, a.dout, r));
                    const int64_t to = (at.row0 + r) * a.D + c;
                    store_pair<T, Mode>((T*)a.dx + to, on0, on1, G);
                    G = mul2(G, S::La::get(s.la, s.la_at(r), lane));
                    store_pair<float, Mode>(a.dlog_a + to, on0, on1, mul2(G, before[k]));
                    const int m = marked && a.dh0 ? s.first[r] : -1;
                    if (m >= 0) store_pair<float, Mode>(a.dh0 + (int64_t)m * a.D + c, on0, on1, G);
                }
            }
        }
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(&s.empty);
    }
}

template <typename T, int Mode, bool Bwd>
__global__ void __launch_bounds__(scan_threads(ring_stages<T, Mode, Bwd>(), Bwd), 1)
glr_scan_kernel(GlrArgs a, ScanWork w, const __grid_constant__ ScanMaps maps)
{
    griddep_wait();
    using S = Stage<T, Mode, Bwd>;
    constexpr int NS = ring_stages<T, Mode, Bwd>();
    static_assert(NS > agg_groups(Bwd) && NS > kFinGroups, "every group meets an end, and ends take a stage each");
    extern __shared__ __align__(128) unsigned char smem[];
    S* ring = reinterpret_cast<S*>(smem);
    int warp = threadIdx.x / 32;
    if (threadIdx.x < NS) {
        S& s = ring[threadIdx.x];
        umma::mbar_init(&s.taken, 1);
        umma::mbar_init(&s.full, 2);             // the copies, and the loader's notes
        umma::mbar_init(&s.agg, 1);
        umma::mbar_init(&s.carried, 1);
        umma::mbar_init(&s.empty, kRuns);
        umma::fence_mbar_init();
    }
    __syncthreads();
    constexpr int kAggWarps = agg_groups(Bwd) * kRuns;
    if (warp < kAggWarps) return scan_aggregate<T, Mode, Bwd, NS>(a, w, ring, warp / kRuns, warp % kRuns);
    warp -= kAggWarps;
    if (warp < kFinWarps) return scan_finish<T, Mode, Bwd, NS>(a, w, ring, warp / kRuns, warp % kRuns);
    warp -= kFinWarps;
    if (warp < carry_warps(NS)) return scan_carry<T, Mode, Bwd, NS>(a, w, ring, warp);
    scan_load<T, Mode, Bwd, NS>(a, w, maps, ring);
}

// One token per sequence: read and written once, V channels a thread (one access each where rows
// start on 16 bytes: V = 4, or 8 for bf16).
template <typename T, int V>
__global__ void __launch_bounds__(128)
glr_step_kernel(const T* __restrict__ x, const float* __restrict__ log_a, float* __restrict__ state,
                const int32_t* __restrict__ slots, T* __restrict__ out, int64_t P, int64_t D,
                int* __restrict__ err)
{
    const int64_t n = blockIdx.x;
    const int64_t c = ((int64_t)blockIdx.y * 128 + threadIdx.x) * V;
    if (c >= D) return;
    struct alignas(V == 1 ? sizeof(T) : V * sizeof(T)) Io { T v[V]; };
    struct alignas(V == 1 ? 4 : 16) Quad { float v[V == 1 ? 1 : 4]; };
    constexpr int Q = V == 1 ? 1 : V / 4, W = V == 1 ? 1 : 4;
    const Io xi = *reinterpret_cast<const Io*>(x + n * D + c);
    Quad l[Q], s[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) l[q] = *reinterpret_cast<const Quad*>(log_a + n * D + c + W * q);
    int64_t row = n;
    Io o = {};
    if (slots) {
        row = slots[n];
        if (row >= P && c == 0 && err) atomicOr(err, kErrSeqlens);
        if (row < 0 || row >= P) {
            *reinterpret_cast<Io*>(out + n * D + c) = o;
            return;
        }
    }
    float* at = state + row * D + c;
#pragma unroll
    for (int q = 0; q < Q; ++q) s[q] = *reinterpret_cast<const Quad*>(at + W * q);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
#pragma unroll
        for (int e = 0; e < W; ++e) {
            s[q].v[e] = expf(l[q].v[e]) * s[q].v[e] + IO<T>::load(xi.v, W * q + e);
            IO<T>::store(o.v, W * q + e, s[q].v[e]);
        }
        *reinterpret_cast<Quad*>(at + W * q) = s[q];
    }
    *reinterpret_cast<Io*>(out + n * D + c) = o;
}

namespace {

template <typename T, int Mode, bool Bwd>
cudaError_t launch_scan(const GlrArgs& a, cudaStream_t st)
{
    ScanWork w = {};
    w.cols = a.B * ((a.D + kCh - 1) / kCh);
    w.tiles = (a.T + kTile - 1) / kTile;
    w.total = w.tiles * w.cols;
    w.blocks = (uint32_t)((a.D + kCh - 1) / kCh);
    w.by_cols = Divide(w.cols);
    w.by_blocks = Divide(w.blocks);
    StreamBuffer buf;
    // a single tile per column waits for nothing: no setup, unless offsets or sequences without
    // tokens want looking at
    if (w.tiles > 1 || a.cu || a.T == 0) {
        const int64_t blocks = (w.tiles + kBlock - 1) / kBlock, rows = blocks > 1 ? blocks : 0;
        const int64_t words = w.tiles > 1 ? (rows * w.cols + w.total) * kCh : 0, ranges = a.cu ? (w.tiles + 1) / 2 * 2 : 0;
        const cudaError_t e = buf.alloc((size_t)((words + ranges) * 8), st);
        if (e != cudaSuccess) return e;
        w.groups = static_cast<unsigned long long*>(buf.ptr);
        w.tile_ab = w.groups + rows * w.cols * kCh;
        w.range = reinterpret_cast<int2*>(w.groups + words);
        w.zeroed = words / 2;
        const int64_t work = w.zeroed / 8 + (a.cu ? w.tiles : 0) + (a.cu || a.T == 0 ? a.N * 256 : 0);
        const int64_t ctas = (work + 255) / 256;
        LaunchScope scope(st, K_GLR_SETUP);
        const cudaError_t s = launch_pdl(glr_setup_kernel, dim3((unsigned)(ctas < 296 ? ctas < 1 ? 1 : ctas : 296)),
                                         dim3(256), 0, st, a, w, Bwd ? 1 : 0);
        if (s != cudaSuccess) return s;
    }
    if (w.total == 0) return cudaSuccess;
    constexpr int smem = ring_stages<T, Mode, Bwd>() * (int)sizeof(Stage<T, Mode, Bwd>);
    const auto kernel = glr_scan_kernel<T, Mode, Bwd>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // rows of R tokens have a stride of 16 bytes
    constexpr bool bf16 = sizeof(T) == 2;
    if (Mode != kWhole) w.log_r = a.D * (int64_t)sizeof(T) % 8 == 0 ? 1 : a.D * (int64_t)sizeof(T) % 4 == 0 ? 2 : 3;
    const int64_t R = int64_t(1) << w.log_r, rows = a.B * a.T / R;
    w.mapped = rows * R;
    ScanMaps maps = {};
    if (rows > 0) {
        using S = Stage<T, Mode, Bwd>;
        const auto map = [&](CUtensorMap* m, const void* p, bool half, int pitch) {
            const int e = half ? 2 : 4;
            return make_tensor_map_2d(m, p, half, (uint64_t)(R * a.D), (uint64_t)rows, (uint64_t)(R * a.D * e),
                                      (uint32_t)(pitch / e), (uint32_t)(kTile / R), false);
        };
        cudaError_t m = map(&maps.la, a.log_a, false, S::La::kPitch);
        if (m == cudaSuccess) m = map(&maps.x, a.x, bf16, S::X::kPitch);
        if (m == cudaSuccess && Bwd) m = map(&maps.y, a.dout, bf16, S::X::kPitch);
        if (m != cudaSuccess) return m;
    }
    LaunchScope scope(st, Bwd ? K_GLR_BWD : K_GLR_FWD);
    const int64_t sms = device_sm_count();
    const dim3 grid((unsigned)(w.total < sms ? w.total : sms)), block(scan_threads(ring_stages<T, Mode, Bwd>(), Bwd));
    if (w.tiles == 1) return launch_pdl(glr_scan_kernel<T, Mode, Bwd>, grid, block, smem, st, a, w, maps);
    return launch_coop(kernel, grid, block, smem, st, a, w, maps);
}

template <typename T, bool Bwd>
cudaError_t launch_scan_io(const GlrArgs& a, cudaStream_t st)
{
    if (a.D * (int64_t)sizeof(T) % 16 == 0) return launch_scan<T, kWhole, Bwd>(a, st);
    return a.D % 2 == 0 ? launch_scan<T, kPairs, Bwd>(a, st) : launch_scan<T, kSingle, Bwd>(a, st);
}

template <bool Bwd>
cudaError_t launch_scan_t(const GlrArgs& a, cudaStream_t st)
{
    return a.io == KDA_IO_F32 ? launch_scan_io<float, Bwd>(a, st) : launch_scan_io<__nv_bfloat16, Bwd>(a, st);
}

}  // namespace

cudaError_t launch_glr_fwd(const GlrArgs& a, cudaStream_t st) { return launch_scan_t<false>(a, st); }
cudaError_t launch_glr_bwd(const GlrArgs& a, cudaStream_t st) { return launch_scan_t<true>(a, st); }

namespace {

template <typename T, int V>
cudaError_t launch_step(const void* x, const float* log_a, float* state, const int32_t* slots, void* out, int64_t N,
                        int64_t P, int64_t D, int* err, cudaStream_t st)
{
    LaunchScope scope(st, K_GLR_STEP);
    glr_step_kernel<T, V><<<dim3((unsigned)N, (unsigned)((D + 128 * V - 1) / (128 * V))), 128, 0, st>>>(
        (const T*)x, log_a, state, slots, (T*)out, P, D, err);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_glr_step(const void* x, const float* log_a, float* state, const int32_t* slots,
                            void* out, int64_t N, int64_t P, int64_t D, kda_io_dtype_t io, int* err,
                            cudaStream_t st)
{
    if (io == KDA_IO_F32)
        return D % 4 == 0 ? launch_step<float, 4>(x, log_a, state, slots, out, N, P, D, err, st)
                          : launch_step<float, 1>(x, log_a, state, slots, out, N, P, D, err, st);
    return D % 8 == 0 ? launch_step<__nv_bfloat16, 8>(x, log_a, state, slots, out, N, P, D, err, st)
                      : launch_step<__nv_bfloat16, 1>(x, log_a, state, slots, out, N, P, D, err, st);
}

}  // namespace kda

using namespace kda;

namespace {

// Channels of one call: grid.y and the 32-bit tile arithmetic of the kernels.
constexpr int64_t kMaxChannels = int64_t(1) << 20;
constexpr int64_t kMaxTokens = 0x7fffffffLL - 2 * kTile;   // 32-bit coordinates
constexpr int64_t kMaxRows = int64_t(1) << 40;

// Rows, channels and tokens; `rows` = 1 with cu_seqlens.
kda_status_t glr_check_sizes(int64_t B, int64_t T, int64_t D, kda_io_dtype_t io, bool packed)
{
    if (B < 0 || T < 0 || D < 0) return KDA_ERR_INVALID_ARG;
    if (io != KDA_IO_F32 && io != KDA_IO_BF16) return KDA_ERR_UNSUPPORTED;
    if (D > kMaxChannels || B > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
    if (T > kMaxTokens || (B > 0 && T > kMaxTokens / B)) return KDA_ERR_UNSUPPORTED;
    // tile numbers are 32-bit
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
    const int64_t nh = (slots ? P : B) * D * 4;
    if (n > 0) {
        if (!tensor_ok(x) || !tensor_ok(log_a) || !tensor_ok(out)) return KDA_ERR_INVALID_ARG;
        const int64_t ns = rows * ((T + KDA_GLR_TILE - 1) / KDA_GLR_TILE) * D * 4;
        if (overlap(out, n * e, x, n * e) || overlap(out, n * e, log_a, n * 4) ||
            overlap(out, n * e, h0, nh) || overlap(out, n * e, hT, nh) || overlap(out, n * e, starts, ns) ||
            overlap(hT, nh, x, n * e) || overlap(hT, nh, log_a, n * 4) || overlap(hT, nh, starts, ns) ||
            overlap(starts, ns, x, n * e) || overlap(starts, ns, log_a, n * 4) || overlap(starts, ns, h0, nh))
            return KDA_ERR_INVALID_ARG;
    }
    if (hT != h0 && overlap(hT, nh, h0, nh)) return KDA_ERR_INVALID_ARG;     // without tokens too: hT = h0 then
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
    if (D > kMaxChannels || N > 0x7fffffffLL || P > kMaxRows) return KDA_ERR_UNSUPPORTED;
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
    if (P > kMaxRows) return KDA_ERR_UNSUPPORTED;
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
    if (overlap(dh0, nh, dhT, nh)) return KDA_ERR_INVALID_ARG;               // without tokens dh0 = dhT
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
