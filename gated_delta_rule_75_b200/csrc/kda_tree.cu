// A tree of drafted tokens over cached states.
//
// Node i continues its parent's state (the cached state S0 for parent -1); with P(i, j) the
// product of the decays alpha on the path from j (exclusive) to i (inclusive),
//
//     A_ij  = sum_c k_ic P_c(i, j) k_jc,     B_ij = sum_c q_ic P_c(i, j) k_jc      (j an ancestor)
//     u_i   = beta_i (v_i - S0^T (P(i, root) k_i) - sum_j A_ij u_j)
//     o_i   = scale (S0^T (P(i, root) q_i) + sum_j B_ij u_j + (q_i . k_i) u_i)
//
// so no node's state is ever formed, and S0 is read once for all of them.  The products of
// decays come from walking up the path one factor at a time: every factor is at most 1, so any
// decay rate is safe, and the last one is the row that multiplies S0.
//
// A head's state is 64 KiB at d = 128, its 16 drafted tokens 24 KiB: 2 us of an SM's share of the
// memory, next to 1 MFLOP of products with S0 (4 for 64 nodes), which mma.sync took 1.6 (6.5) us of
// an SM for, so they are on tcgen05: 0.3 (0.8) us.  What bounds the kernel is the latency of its
// steps: 20,600 (29,300) cycles, of which 5,100 (6,000) are loads, 5,400 (5,000) the products and 3,400
// (8,000) the levels; three CTAs of an SM cover one another up to 16 nodes, two up to 32, and the
// state of the CTA that follows is brought into the L2 meanwhile.  64 x 16 nodes, 32 heads: 68 us, 2.7 TB/s;
// 40 x 61 nodes: 142 us.
// One CTA for one (sequence, head).  The walking warps, eight lanes a node:
//   1. alpha, k into shared memory; depths, order by depth;
//   2. walk up the node's path, every lane 16 (8) channels: the dots with every ancestor (three
//      shuffles each), then the node's two rows, kept in registers;
//   3. the rows (keys, then queries) as bf16 summands in shared memory.
// Meanwhile four more warps bring S0 there, as bf16 summands too.  Then one thread issues the
// product, transposed, D^T = S0^T rows^T: M = dv, N = rows, so that N and the tensor memory follow
// the number of nodes.  Rows and S0 are split into three bf16 summands each, which hold all 24 bits of
// an fp32 value whatever the I/O type (two would take 59 and 125 us, and round the state to 17 bits).
// Products down to 2^-16 of the largest are taken, those of a weight into sums of their own: an addition
// in tensor memory truncates, and the sums that reach full size take 8 that way, not 48 (128 terms: 1.4e-7
// off, 1.4e-6 with all in the same sums).  Then, all warps:
//   4. D^T to shared memory; level by level, a warp a node: u_i and o_i.
#include "kda_common.cuh"
#include "kda_f32x2.cuh"
#include "kda_internal.h"
#include "kda_umma.cuh"

namespace kda {

// Nodes of one sequence's tree, checked: a parent must come before its child.
__device__ __forceinline__ int tree_parent(const int32_t* parents, int i, int* err)
{
    int p = parents[i];
    if (p < -1 || p >= i) {
        if (err) atomicOr(err, kErrSeqlens);
        p = -1;
    }
    return p;
}

// Four channels of q, k or v.
template <typename T> __device__ __forceinline__ float4 load4(const T* p);
template <> __device__ __forceinline__ float4 load4<float>(const float* p) { return *reinterpret_cast<const float4*>(p); }
template <> __device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p)
{
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}
using umma::pack_bf16;

// Four channels in shared memory, as pairs.
struct Four { F2 a, b; };
__device__ __forceinline__ Four four(const float* p)
{
    const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(p);
    Four f;
    f.a.v = u.x;
    f.b.v = u.y;
    return f;
}

// (x, y) as three bf16 pairs, the largest first, whose sum is x, y: each takes 8 of the 24 bits.
constexpr int kSummands = 3;
__device__ __forceinline__ void split(float x, float y, uint32_t (&s)[kSummands])
{
#pragma unroll
    for (int i = 0; i < kSummands; ++i) {
        s[i] = pack_bf16(x, y);
        x -= __uint_as_float(s[i] << 16);
        y -= __uint_as_float(s[i] & 0xffff0000u);
    }
}

// Eight lanes for every node walk; four more warps bring S0.
constexpr int tree_walkers(int KB) { return 8 * KB; }
constexpr int kTreeStagers = 128;
// CTAs of an SM, by their registers and shared memory.
constexpr int tree_per_sm(int KB, int io_bytes) { return KB == 64 ? 1 : KB == 32 ? (io_bytes == 2 ? 2 : 1) : (io_bytes == 2 ? 3 : 2); }
constexpr int kTreeErrBit = 2;                             // "operand MMAs" of the error word

// Shared memory of a CTA for trees of up to KB nodes.
template <int DK, int DV, int KB, int IoBytes>
struct TreeSmem {
    static constexpr int NS = kSummands, kPairs = KB * (KB + 1) / 2;
    // S0 comes in one piece, or, where that lets another CTA onto the SM, 64 rows at a time
    static constexpr int kPieces = tree_per_sm(KB, IoBytes) > 1 ? DK / 64 : 1, kRows = DK / kPieces;
    static constexpr int kColumns = KB == 16 ? 128 : KB == 32 ? 256 : 512;     // of tensor memory
    static_assert(NS * 2 * KB <= kColumns, "sums of NS weights for the rows of keys and queries");
    static constexpr int kState = kRows * DV * 2;          // bytes of one summand of a piece
    // with dv = 64 the upper half of the M = 128 operand is whatever follows: its rows are not used
    static constexpr int kSlack = DV == 64 ? kRows * 128 : 0;
    static constexpr int kA = 2 * KB * DK * 4, kB = NS * 2 * KB * DK * 2, kC = 2 * KB * DV * 4;
    static constexpr int kRegion = kA > kB ? (kA > kC ? kA : kC) : (kB > kC ? kB : kC);
    // S0: [NS] of blocks of 64 columns, [kRows][64] bf16 each, 128-byte swizzle (M-major operand)
    alignas(1024) unsigned char state[NS * kState + kSlack];
    // alpha, k [KB][DK]; then the rows, [NS] of blocks of 64 channels, [2 KP][64] bf16 each, 128-byte
    // swizzle (K-major operand); then the products with S0 [2][KB][DV], whose first half becomes u
    alignas(1024) unsigned char region[kRegion];
    float2 ab[kPairs];                                     // A, B of a node, by place on its path, itself at 0
    float beta[KB];
    int par[KB], depth[KB], off[KB], order[KB], level_end[KB + 1];
    uint64_t done[kPieces];                                // the products
    uint32_t tmem;
    unsigned char anc[kPairs];                             // the node at that place
};

template <int Bytes> __device__ __forceinline__ void prefetch_l2(const void* p)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "n"(Bytes) : "memory");
}

// Everything that the CTA of sequence n, head h reads, by 128 threads.
template <typename T, int DK, int DV>
__device__ __forceinline__ void prefetch_item(const TreeArgs& a, int64_t n, int64_t h, int tid)
{
    const int64_t row = a.slots ? a.slots[n] : n;
    const int live = a.num_nodes ? a.num_nodes[n] : (int)a.K;
    if (tid == 127 && row >= 0 && row < a.P) prefetch_l2<DK * DV * 4>(a.state + (row * a.H + h) * (int64_t)DK * DV);
    if (tid >= live || tid >= a.K) return;
    const int64_t tok = (n * a.K + tid) * a.H + h;
    prefetch_l2<DK * 4>(a.log_alpha + tok * DK);
    prefetch_l2<DK * sizeof(T)>((const T*)a.k + tok * DK);
    prefetch_l2<DK * sizeof(T)>((const T*)a.q + tok * DK);
    prefetch_l2<DV * sizeof(T)>((const T*)a.v + tok * DV);
}

// The walking warps, the staging warps.
template <int KB> __device__ __forceinline__ void walkers_sync()
{
    asm volatile("bar.sync 1, %0;" ::"n"(tree_walkers(KB)) : "memory");
}
// Whether all staging threads say so.
__device__ __forceinline__ bool stagers_all(bool ok)
{
    int all;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbar.red.and.pred q, 2, %2, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
                 : "=r"(all)
                 : "r"((int)ok), "n"(kTreeStagers)
                 : "memory");
    return all != 0;
}

template <typename T, int DK, int DV, int KB>
__global__ void __launch_bounds__(tree_walkers(KB) + kTreeStagers, tree_per_sm(KB, sizeof(T))) tree_fwd_kernel(const TreeArgs a)
{
    constexpr int NS = kSummands;
    using Smem = TreeSmem<DK, DV, KB, sizeof(T)>;
    constexpr int kQuads = DK / 32;                        // float4 channel groups of a lane in the walk
    constexpr int kWalkers = tree_walkers(KB), kThreads = kWalkers + kTreeStagers, kStageWarp = kWalkers / 32;
    extern __shared__ __align__(1024) unsigned char raw[];
    Smem& sm = *reinterpret_cast<Smem*>(raw);
    float* alpha = reinterpret_cast<float*>(sm.region);
    float* kf = alpha + KB * DK;
    const int K = (int)a.K, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int64_t n = blockIdx.x / a.H, h = blockIdx.x % a.H;

    int64_t row = n;
    if (a.slots) {
        row = a.slots[n];
        if (row >= a.P && tid == 0) atomicOr(a.err, kErrSeqlens);
        if (row >= a.P) row = -1;
    }
    const float* S0 = row < 0 ? nullptr : a.state + (row * a.H + h) * (int64_t)DK * DV;
    int live = K;
    if (a.num_nodes) {
        live = a.num_nodes[n];
        if ((live < 0 || live > K) && tid == 0) atomicOr(a.err, kErrSeqlens);
        live = live < 0 ? 0 : live > K ? K : live;
    }
    if (live == 0) return;
    const int64_t tok0 = (n * K) * a.H + h;                // node i: tok0 + i * H
    const int KP = (live + 15) / 16 * 16;                  // rows of keys, and of queries
    if (warp == kStageWarp) {
        umma::tmem_alloc(&sm.tmem, Smem::kColumns);
        umma::tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < Smem::kPieces; ++i) umma::mbar_init(&sm.done[i], 1);
        umma::fence_mbar_init();
    }
    float* prod = reinterpret_cast<float*>(sm.region);
    // S0, by the staging warps: a row (two rows of 64 columns) a warp at a time
    constexpr int kPerRow = DV / 4, kStep = kTreeStagers / kPerRow;
    constexpr int kLoads = Smem::kRows / kStep < 16 ? Smem::kRows / kStep : 16;      // rows of a thread on their way
    static_assert(Smem::kRows % (kLoads * kStep) == 0, "whole rounds");
    const int mine = tid - kWalkers, sc = mine % kPerRow * 4, sr = mine / kPerRow;
    float4 s[kLoads];
    const auto ask = [&](int piece, int k0) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            s[i] = __ldcs(reinterpret_cast<const float4*>(S0 + (piece * Smem::kRows + k0 + sr + i * kStep) * DV + sc));
    };
    const auto put = [&](int k0) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            uint32_t lo[NS], hi[NS];
            split(s[i].x, s[i].y, lo);
            split(s[i].z, s[i].w, hi);
            const uint32_t to = sc / 64 * (Smem::kRows * 128) + umma::sw128_offset(k0 + sr + i * kStep, sc % 64);
#pragma unroll
            for (int e = 0; e < NS; ++e)
                *reinterpret_cast<uint2*>(sm.state + e * Smem::kState + to) = make_uint2(lo[e], hi[e]);
        }
    };
    // The products with one piece, by one thread.  Summand i of S0 times summand j of the rows goes into sums
    // i + j, so the first sums, which alone reach full size, take only one addition for 16 channels; the rows'
    // summands lie side by side, and one MMA takes all that a summand of S0 is multiplied by
    const auto multiply = [&](int piece) {
        const uint64_t ad = umma::make_desc(umma::smem_u32(sm.state), Smem::kRows * 128, 1024);
        const uint64_t bd = umma::make_desc(umma::smem_u32(sm.region), 16, 1024);
        const uint32_t block = NS * 2 * KP * 128 / 16;     // 64 channels of the rows, in descriptor units
#pragma unroll
        for (int ks = 0; ks < Smem::kRows / 16; ++ks) {
            const int step = piece * (Smem::kRows / 16) + ks;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const uint64_t at = ad + (i * Smem::kState + ks * 2048) / 16, bt = bd + step / 4 * block + step % 4 * 2;
                const int columns = (NS - i) * 2 * KP, most = columns > 256 ? 256 : columns;
                umma::mma_bf16(sm.tmem + i * 2 * KP, at, bt, umma::make_idesc_bf16(128, most, true, false), step + i > 0);
                if (KB == 64 && columns > most)
                    umma::mma_bf16(sm.tmem + i * 2 * KP + most, at, bt + most * 128 / 16,
                                   umma::make_idesc_bf16(128, columns - most, true, false), step + i > 0);
            }
        }
        umma::commit(&sm.done[piece]);
    };
    if (warp >= kStageWarp) {
        if (S0) {
#pragma unroll 1
            for (int k0 = 0; k0 < Smem::kRows; k0 += kLoads * kStep) {
                ask(0, k0);
                put(k0);
            }
            if (Smem::kPieces > 1) ask(1, 0);
        }
        // what the CTA that follows this one on the SM will read goes into the L2 meanwhile, or memory
        // would idle while this one computes
        const int64_t next = (int64_t)blockIdx.x + a.resident;
        if (next < a.N * a.H) prefetch_item<T, DK, DV>(a, next / a.H, next % a.H, mine);
    } else {
        if (tid < live) {
            sm.par[tid] = tree_parent(a.parents + n * K, tid, a.err);
            sm.beta[tid] = a.beta[tok0 + tid * a.H];
            // q and v are asked for when a node's turn comes: into the L2 meanwhile
#pragma unroll
            for (int c = 0; c < DK * (int)sizeof(T); c += 128)
                asm volatile("prefetch.global.L2 [%0];" ::"l"((const char*)a.q + (tok0 + tid * a.H) * DK * sizeof(T) + c));
#pragma unroll
            for (int c = 0; c < DV * (int)sizeof(T); c += 128)
                asm volatile("prefetch.global.L2 [%0];" ::"l"((const char*)a.v + (tok0 + tid * a.H) * DV * sizeof(T) + c));
        }
        if (tid <= KB) sm.level_end[tid] = 0;
        constexpr int kAhead = 4;                              // quads of alpha and k a thread has on their way
        const int quads = live * (DK / 4);
        for (int e0 = tid; e0 < quads; e0 += kWalkers * kAhead) {
            float4 g[kAhead];
            struct alignas(4 * sizeof(T)) Raw { T v[4]; } k[kAhead];
#pragma unroll
            for (int r = 0; r < kAhead; ++r) {
                const int e = min(e0 + r * kWalkers, quads - 1);         // the last one again past the end
                const int64_t at = (tok0 + e / (DK / 4) * a.H) * DK + e % (DK / 4) * 4;
                g[r] = __ldcs(reinterpret_cast<const float4*>(a.log_alpha + at));
                k[r] = *reinterpret_cast<const Raw*>((const T*)a.k + at);
            }
#pragma unroll
            for (int r = 0; r < kAhead; ++r) {
                const int e = min(e0 + r * kWalkers, quads - 1);
                *reinterpret_cast<float4*>(alpha + 4 * e) = make_float4(expf(g[r].x), expf(g[r].y), expf(g[r].z), expf(g[r].w));
                *reinterpret_cast<float4*>(kf + 4 * e) = load4(k[r].v);
            }
        }
        walkers_sync<KB>();
        if (tid < live) {
            int d = 1;                                         // nodes on the path, itself too
            for (int j = sm.par[tid]; j >= 0; j = sm.par[j]) ++d;
            sm.depth[tid] = d;
        }
        walkers_sync<KB>();
        if (tid < live) {
            const int mine = sm.depth[tid];
            int off = 0, pos = 0;
            for (int j = 0; j < live; ++j) {
                const int d = sm.depth[j];
                off += j < tid ? d : 0;
                pos += d < mine || (d == mine && j < tid);
            }
            sm.off[tid] = off;
            sm.order[pos] = tid;
            atomicMax(&sm.level_end[mine], pos + 1);
        }
        walkers_sync<KB>();

        // 2. the walks: lane l of a group holds channels 4 (l + 8 m) .. + 3
        const int l8 = lane % 8;
        F2 wk[kQuads][2], wq[kQuads][2];
        const int node = warp * 4 + lane / 8 < live ? sm.order[warp * 4 + lane / 8] : -1;
        {
            const int i = node;
            int j = -1, place = 0;
            float2 dot = make_float2(0.f, 0.f);
            if (i >= 0) {
                j = sm.par[i];
                place = sm.off[i];
                F2 self = both(0.f);
#pragma unroll
                for (int m = 0; m < kQuads; ++m) {
                    const int c = 4 * (l8 + 8 * m);
                    const float4 q = load4((const T*)a.q + (tok0 + i * a.H) * DK + c);
                    const Four k = four(kf + i * DK + c), g = four(alpha + i * DK + c);
                    const F2 q0(q.x, q.y), q1(q.z, q.w);
                    self = fma2(q1, k.b, fma2(q0, k.a, self));
                    wk[m][0] = mul2(k.a, g.a);
                    wk[m][1] = mul2(k.b, g.b);
                    wq[m][0] = mul2(q0, g.a);
                    wq[m][1] = mul2(q1, g.b);
                }
                dot.y = self.x() + self.y();
            }
            int at_node = i;                                   // the node whose dots are in `dot`
            // every lane of the warp goes round as often as its longest path asks
            while (__any_sync(0xffffffffu, at_node >= 0)) {
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) {
                    dot.x += __shfl_xor_sync(0xffffffffu, dot.x, o);
                    dot.y += __shfl_xor_sync(0xffffffffu, dot.y, o);
                }
                if (at_node >= 0 && l8 == 0) {
                    sm.ab[place] = dot;
                    sm.anc[place] = (unsigned char)at_node;
                }
                ++place;
                at_node = j;
                if (j >= 0) {
                    F2 x = both(0.f), y = both(0.f);
#pragma unroll
                    for (int m = 0; m < kQuads; ++m) {
                        const int c = 4 * (l8 + 8 * m);
                        const Four k = four(kf + j * DK + c), g = four(alpha + j * DK + c);
                        x = fma2(wk[m][1], k.b, fma2(wk[m][0], k.a, x));
                        y = fma2(wq[m][1], k.b, fma2(wq[m][0], k.a, y));
                        wk[m][0] = mul2(wk[m][0], g.a);
                        wk[m][1] = mul2(wk[m][1], g.b);
                        wq[m][0] = mul2(wq[m][0], g.a);
                        wq[m][1] = mul2(wq[m][1], g.b);
                    }
                    dot = make_float2(x.x() + x.y(), y.x() + y.y());
                    j = sm.par[j];
                }
            }
        }
        walkers_sync<KB>();                                        // alpha and k are done with

        // 3. the rows
        if (S0) {
            if (node >= 0)
#pragma unroll
                    for (int m = 0; m < kQuads; ++m)
#pragma unroll
                        for (int which = 0; which < 2; ++which) {
                            const F2 x = which ? wq[m][0] : wk[m][0], y = which ? wq[m][1] : wk[m][1];
                            uint32_t lo[NS], hi[NS];
                            split(x.x(), x.y(), lo);
                            split(y.x(), y.y(), hi);
                            const int c = 4 * (l8 + 8 * m);
                            // (the rows of a summand are a multiple of 8, where the swizzle repeats)
                            const uint32_t to = c / 64 * (NS * 2 * KP * 128) + umma::sw128_offset(which * KP + node, c % 64);
#pragma unroll
                            for (int e = 0; e < NS; ++e)
                                *reinterpret_cast<uint2*>(sm.region + e * (2 * KP * 128) + to) = make_uint2(lo[e], hi[e]);
                        }
        }
    }
    umma::fence_smem_to_async();
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    bool fine = true;
    if (S0) {
        if (tid == 0) multiply(0);
        if (Smem::kPieces > 1 && warp >= kStageWarp) {
            // the first piece's products, another thread's, have read their operands and come before the second's
            // in the sums; if they do not end, the second piece is left out and so is its signal
            const bool first = __all_sync(0xffffffffu, umma::mbar_wait(&sm.done[0], 0, a.err, kTreeErrBit));
            umma::fence_after_sync();
            for (int k0 = 0; first && k0 < Smem::kRows; k0 += kLoads * kStep) {
                if (k0 > 0) ask(1, k0);
                put(k0);
            }
            umma::fence_smem_to_async();
            if (stagers_all(first) && tid == kWalkers) multiply(1);
        }
    }
    // a thread's column and its first 16 rows: v is asked for before the wait.  Lane = column of S0,
    // TMEM column = row; the warps of one quarter of the lanes take 16 rows in turn
    const int col = warp % 4 * 32 + lane;
    T v0[16];
    const auto load_v = [&](int r0, T (&v)[16]) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (r0 + e < live && col < DV) v[e] = ((const T*)a.v)[(tok0 + (r0 + e) * a.H) * DV + col];
    };
    load_v(warp / 4 * 16, v0);
    if (S0) {
        fine = umma::block_wait(&sm.done[Smem::kPieces - 1], 0, a.err, kTreeErrBit);
        umma::fence_after_sync();
    }
    if (fine && warp % 4 * 32 < DV)
        for (int c0 = warp / 4 * 16; c0 < 2 * KP; c0 += kThreads / 128 * 16) {
            float x[16] = {};
            if (S0) {
                const uint32_t from = sm.tmem + ((uint32_t)(warp % 4 * 32) << 16) + c0;
#pragma unroll
                for (int i = NS - 1; i >= 0; --i) {        // the smallest sums first
                    float y[16];
                    umma::tmem_ld16(from + i * 2 * KP, y);
                    umma::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] += y[e];
                }
            }
            if (c0 < KP) {                                 // keys: v - S0^T (..)
                if (c0 >= kThreads / 128 * 16) load_v(c0, v0);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (c0 + e < live) prod[(c0 + e) * DV + col] = IO<T>::load(v0, e) - x[e];
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) prod[(KB + c0 - KP + e) * DV + col] = x[e];
            }
        }
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    if (warp == kStageWarp) umma::tmem_dealloc(sm.tmem, Smem::kColumns);
    if (!fine) return;

    // 4. level by level; a lane holds CPL columns
    constexpr int CPL = DV / 32;
    struct alignas(4 * CPL) Cols { float v[CPL]; };
    for (int done = 0, level = 1; done < live; ++level) {
        const int end = sm.level_end[level];
        for (int at = done + warp; at < end; at += kThreads / 32) {
            const int i = sm.order[at], off = sm.off[i];
            Cols vk = *reinterpret_cast<const Cols*>(prod + i * DV + CPL * lane);
            Cols pq = *reinterpret_cast<const Cols*>(prod + (KB + i) * DV + CPL * lane);
            const int64_t to = (tok0 + i * a.H) * DV + CPL * lane;
#pragma unroll 4
            for (int p = 1; p < level; ++p) {
                const float2 ab = sm.ab[off + p];
                const Cols u = *reinterpret_cast<const Cols*>(prod + sm.anc[off + p] * DV + CPL * lane);
#pragma unroll
                for (int e = 0; e < CPL; ++e) {
                    vk.v[e] -= ab.x * u.v[e];
                    pq.v[e] += ab.y * u.v[e];
                }
            }
            const float self = sm.ab[off].y, b = sm.beta[i];
            Cols o;
#pragma unroll
            for (int e = 0; e < CPL; ++e) {
                vk.v[e] *= b;
                o.v[e] = a.scale * (pq.v[e] + self * vk.v[e]);
            }
            *reinterpret_cast<Cols*>(prod + i * DV + CPL * lane) = vk;
            if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<Cols*>((T*)a.out + to) = o;
            } else if constexpr (CPL == 4) {
                *reinterpret_cast<uint2*>((T*)a.out + to) = make_uint2(pack_bf16(o.v[0], o.v[1]), pack_bf16(o.v[2], o.v[3]));
            } else {
                *reinterpret_cast<uint32_t*>((T*)a.out + to) = pack_bf16(o.v[0], o.v[1]);
            }
        }
        done = end;
        __syncthreads();
    }
}

// The accepted path's tokens applied to the cached state, in place: the decode step's
// arithmetic once per token, with the state in registers from the first to the last, so that
// it is read and written once however long the path (bound by memory: 128 KiB a head at
// d = 128).  One CTA of 256 threads for kCommitCols columns of one (sequence, head): columns
// go their own way, and more, smaller CTAs on an SM mix loads, arithmetic and stores better.
// The tokens of up to kCommitAhead places of the path are brought in together, while the state
// is on its way.
constexpr int kCommitAhead = 8, kCommitCols = 64;

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(256, 4) tree_commit_kernel(const TreeArgs a)
{
    constexpr int DB = kCommitCols, TPR = DB / 4;      // columns; threads per state row (float4 each)
    constexpr int RG = 256 / TPR;      // row groups
    constexpr int RPT = DK / RG;       // rows per thread
    __shared__ float sk[kCommitAhead][DK], sa[kCommitAhead][DK], sv[kCommitAhead][DB], se[DB], sb[kCommitAhead];
    __shared__ float4 red[RG][TPR];
    __shared__ int par[KDA_TREE_MAX_NODES], path[KDA_TREE_MAX_NODES];   // accepted node first
    __shared__ int count;
    const int tid = threadIdx.x, c4 = tid % TPR, rg = tid / TPR;
    const int64_t item = blockIdx.x / (DV / DB), n = item / a.H, h = item % a.H;
    const int c0 = (int)(blockIdx.x % (DV / DB)) * DB;
    const int K = (int)a.K;
    const int64_t sl = a.slots ? a.slots[n] : n;
    const int last = a.accepted[n];
    if (tid < K) par[tid] = a.parents[n * K + tid];
    if (sl >= a.P || last >= K || last < -1) {
        if (tid == 0) atomicOr(a.err, kErrSeqlens);
        return;
    }
    if (sl < 0 || last < 0) return;
    float4* S4 = reinterpret_cast<float4*>(a.state + (sl * a.H + h) * (int64_t)DK * DV + c0);
    float4 s[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r) s[r] = __ldcs(&S4[(rg * RPT + r) * (DV / 4) + c4]);
    __syncthreads();
    if (tid == 0) {
        int c = 0;
        for (int i = last; i >= 0; i = tree_parent(par, i, a.err)) path[c++] = i;
        count = c;
    }
    __syncthreads();
    for (int left = count; left > 0; left -= kCommitAhead) {
        const int now = left < kCommitAhead ? left : kCommitAhead;
        for (int e = tid; e < now * DK; e += 256) {
            const int64_t tok = (n * K + path[left - 1 - e / DK]) * a.H + h;
            sk[e / DK][e % DK] = IO<T>::load((const T*)a.k, tok * DK + e % DK);
            sa[e / DK][e % DK] = expf(__ldcs(a.log_alpha + tok * DK + e % DK));
        }
        for (int e = tid; e < now * DB; e += 256) {
            const int64_t tok = (n * K + path[left - 1 - e / DB]) * a.H + h;
            sv[e / DB][e % DB] = IO<T>::load((const T*)a.v, tok * DV + c0 + e % DB);
        }
        if (tid < now) sb[tid] = a.beta[(n * K + path[left - 1 - tid]) * a.H + h];
        __syncthreads();
        for (int p = 0; p < now; ++p) {
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                const float al = sa[p][rg * RPT + r], kk = sk[p][rg * RPT + r];
                s[r].x *= al; s[r].y *= al; s[r].z *= al; s[r].w *= al;
                acc.x += kk * s[r].x; acc.y += kk * s[r].y; acc.z += kk * s[r].z; acc.w += kk * s[r].w;
            }
            red[rg][c4] = acc;
            __syncthreads();
            for (int j = tid; j < DB; j += 256) {
                float vh = 0.f;
#pragma unroll
                for (int g = 0; g < RG; ++g) vh += reinterpret_cast<const float*>(&red[g][0])[j];
                se[j] = sb[p] * (sv[p][j] - vh);
            }
            __syncthreads();
            const float4 e = reinterpret_cast<const float4*>(se)[c4];
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                const float kk = sk[p][rg * RPT + r];
                s[r].x += kk * e.x; s[r].y += kk * e.y; s[r].z += kk * e.z; s[r].w += kk * e.w;
            }
        }
        __syncthreads();               // the tokens' places are filled again
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r) __stcs(&S4[(rg * RPT + r) * (DV / 4) + c4], s[r]);
}

namespace {

template <typename T, int DK, int DV, int KB>
cudaError_t tree_fwd_kb(TreeArgs a, cudaStream_t st)
{
    constexpr int smem = (int)sizeof(TreeSmem<DK, DV, KB, sizeof(T)>);
    const cudaError_t e = cudaFuncSetAttribute(tree_fwd_kernel<T, DK, DV, KB>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    a.resident = device_sm_count() * tree_per_sm(KB, sizeof(T));
    LaunchScope scope(st, K_TREE_FWD);
    tree_fwd_kernel<T, DK, DV, KB><<<(unsigned)(a.N * a.H), tree_walkers(KB) + kTreeStagers, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int DK, int DV>
cudaError_t tree_fwd_t(const TreeArgs& a, cudaStream_t st)
{
    // shared memory and registers for the next power of two of nodes
    if (a.K <= 16) return tree_fwd_kb<T, DK, DV, 16>(a, st);
    if (a.K <= 32) return tree_fwd_kb<T, DK, DV, 32>(a, st);
    return tree_fwd_kb<T, DK, DV, 64>(a, st);
}

template <typename T, int DK, int DV>
cudaError_t tree_commit_t(const TreeArgs& a, cudaStream_t st)
{

    LaunchScope scope(st, K_TREE_COMMIT);
    tree_commit_kernel<T, DK, DV><<<(unsigned)(a.N * a.H * (DV / kCommitCols)), 256, 0, st>>>(a);
    return cudaGetLastError();
}

#define KDA_TREE_BY_DIMS(F, T)                                      \
    do {                                                            \
        if (a.dk == 128 && a.dv == 128) return F<T, 128, 128>(a, st); \
        if (a.dk == 128) return F<T, 128, 64>(a, st);                \
        if (a.dv == 128) return F<T, 64, 128>(a, st);                \
        return F<T, 64, 64>(a, st);                                 \
    } while (0)

}  // namespace

cudaError_t launch_tree_fwd(const TreeArgs& a, cudaStream_t st)
{
    if (a.io == KDA_IO_F32) KDA_TREE_BY_DIMS(tree_fwd_t, float);
    KDA_TREE_BY_DIMS(tree_fwd_t, __nv_bfloat16);
}

cudaError_t launch_tree_commit(const TreeArgs& a, cudaStream_t st)
{
    if (a.io == KDA_IO_F32) KDA_TREE_BY_DIMS(tree_commit_t, float);
    KDA_TREE_BY_DIMS(tree_commit_t, __nv_bfloat16);
}

}  // namespace kda

using namespace kda;

namespace {

bool tree_dim_ok(int64_t d) { return d == 64 || d == 128; }

// Sizes that both entry points refuse; KDA_OK with *empty set when there is nothing to do.
kda_status_t tree_check(int64_t N, int64_t P, int64_t K, int64_t H, int64_t dk, int64_t dv, kda_io_dtype_t io,
                        bool* empty)
{
    if (N < 0 || P < 0 || K < 0 || H < 0) return KDA_ERR_INVALID_ARG;
    if (io != KDA_IO_F32 && io != KDA_IO_BF16) return KDA_ERR_UNSUPPORTED;
    if (!tree_dim_ok(dk) || !tree_dim_ok(dv) || K > KDA_TREE_MAX_NODES) return KDA_ERR_UNSUPPORTED;
    if (N > 0x7fffffffLL || H > 0x7fffffffLL || N * H > 0x3fffffffLL) return KDA_ERR_UNSUPPORTED;
    if (H > 0 && P > (int64_t(1) << 40) / H) return KDA_ERR_UNSUPPORTED;
    *empty = N == 0 || H == 0 || K == 0;
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status_t kda_tree_fwd(const void* q, const void* k, const void* v, const float* log_alpha,
                          const float* beta, const float* state, const int32_t* slots,
                          const int32_t* parents, const int32_t* num_nodes, void* out, int64_t N,
                          int64_t P, int64_t K, int64_t H, int64_t dk, int64_t dv, float scale,
                          kda_io_dtype_t io_dtype, cudaStream_t stream)
{
    bool empty = false;
    const kda_status_t s = tree_check(N, slots ? P : N, K, H, dk, dv, io_dtype, &empty);
    if (s != KDA_OK || empty) return s;
    if (!tensor_ok(q) || !tensor_ok(k) || !tensor_ok(v) || !tensor_ok(log_alpha) || !tensor_ok(out))
        return KDA_ERR_INVALID_ARG;
    if (!(slots && P == 0) && !tensor_ok(state)) return KDA_ERR_INVALID_ARG;
    if (!beta || !parents || !is_aligned(beta, 4) || !is_aligned(parents, 4) || !is_aligned(slots, 4) ||
        !is_aligned(num_nodes, 4))
        return KDA_ERR_INVALID_ARG;
    const int64_t t = N * K * H, e = io_dtype == KDA_IO_F32 ? 4 : 2, no = t * dv * e;
    if (overlap(out, no, q, t * dk * e) || overlap(out, no, k, t * dk * e) || overlap(out, no, v, no) ||
        overlap(out, no, log_alpha, t * dk * 4) || overlap(out, no, beta, t * 4) ||
        overlap(out, no, state, (slots ? P : N) * H * dk * dv * 4) || overlap(out, no, parents, N * K * 4) ||
        overlap(out, no, slots, N * 4) || overlap(out, no, num_nodes, N * 4))
        return KDA_ERR_INVALID_ARG;
    TreeArgs a = {};
    a.q = q; a.k = k; a.v = v; a.log_alpha = log_alpha; a.beta = beta; a.state = const_cast<float*>(state);
    a.slots = slots; a.parents = parents; a.num_nodes = num_nodes; a.out = out;
    a.N = N; a.P = slots ? P : N; a.K = K; a.H = H; a.dk = (int)dk; a.dv = (int)dv; a.scale = scale; a.io = io_dtype;
    cudaError_t err = library_error_word(&a.err);
    if (err == cudaSuccess) err = launch_tree_fwd(a, stream);
    return finish_call(err, stream);
}

kda_status_t kda_tree_commit(const void* k, const void* v, const float* log_alpha, const float* beta,
                             float* state, const int32_t* slots, const int32_t* parents,
                             const int32_t* accepted, int64_t N, int64_t P, int64_t K, int64_t H,
                             int64_t dk, int64_t dv, kda_io_dtype_t io_dtype, cudaStream_t stream)
{
    bool empty = false;
    const kda_status_t s = tree_check(N, slots ? P : N, K, H, dk, dv, io_dtype, &empty);
    if (s != KDA_OK || empty) return s;
    if (!tensor_ok(k) || !tensor_ok(v) || !tensor_ok(log_alpha)) return KDA_ERR_INVALID_ARG;
    if (!(slots && P == 0) && !tensor_ok(state)) return KDA_ERR_INVALID_ARG;
    if (!beta || !parents || !accepted || !is_aligned(beta, 4) || !is_aligned(parents, 4) ||
        !is_aligned(slots, 4) || !is_aligned(accepted, 4))
        return KDA_ERR_INVALID_ARG;
    const int64_t t = N * K * H, e = io_dtype == KDA_IO_F32 ? 4 : 2;
    const int64_t ns = (slots ? P : N) * H * dk * dv * 4;
    if (overlap(state, ns, k, t * dk * e) || overlap(state, ns, v, t * dv * e) ||
        overlap(state, ns, log_alpha, t * dk * 4) || overlap(state, ns, beta, t * 4) ||
        overlap(state, ns, parents, N * K * 4) || overlap(state, ns, slots, N * 4) ||
        overlap(state, ns, accepted, N * 4))
        return KDA_ERR_INVALID_ARG;
    TreeArgs a = {};
    a.k = k; a.v = v; a.log_alpha = log_alpha; a.beta = beta; a.state = state;
    a.slots = slots; a.parents = parents; a.accepted = accepted;
    a.N = N; a.P = slots ? P : N; a.K = K; a.H = H; a.dk = (int)dk; a.dv = (int)dv; a.io = io_dtype;
    cudaError_t err = library_error_word(&a.err);
    if (err == cudaSuccess) err = launch_tree_commit(a, stream);
    return finish_call(err, stream);
}

}  // extern "C"
