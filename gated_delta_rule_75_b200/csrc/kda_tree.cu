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
#include "kda_common.cuh"
#include "kda_internal.h"

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

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One CTA of 256 threads for one (sequence, head).
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(256) tree_fwd_kernel(TreeArgs a)
{
    constexpr int CPL = DK / 32;
    extern __shared__ float sm[];
    const int K = (int)a.K;
    float* alpha = sm;                       // [K][DK]
    float* kk = alpha + K * DK;              // [K][DK]
    float* W = kk + K * DK;                  // [2K][DK]: decayed keys, decayed queries
    float* AB = W + 2 * K * DK;              // [K][K][2]: by place on the path, self at 0
    float* bet = AB + 2 * K * K;             // [K]
    int* par = reinterpret_cast<int*>(bet + K);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int64_t n = blockIdx.x / a.H, h = blockIdx.x % a.H;

    int live = K;
    if (a.num_nodes) {
        live = a.num_nodes[n];
        if ((live < 0 || live > K) && tid == 0) atomicOr(a.err, kErrSeqlens);
        live = live < 0 ? 0 : live > K ? K : live;
    }
    int64_t row = n;
    if (a.slots) {
        row = a.slots[n];
        if (row >= a.P && tid == 0) atomicOr(a.err, kErrSeqlens);
        if (row >= a.P) row = -1;
    }
    const float* S0 = row < 0 ? nullptr : a.state + (row * a.H + h) * (int64_t)DK * DV;
    const int64_t tok0 = (n * K) * a.H + h;  // node i: tok0 + i * H
    for (int i = tid; i < live; i += 256) {
        par[i] = tree_parent(a.parents + n * K, i, a.err);
        bet[i] = a.beta[tok0 + i * a.H];
    }
    for (int i = tid; i < live * DK; i += 256) {
        const int64_t at = (tok0 + (i / DK) * a.H) * DK + i % DK;
        alpha[i] = expf(a.log_alpha[at]);
        kk[i] = IO<T>::load((const T*)a.k, at);
    }
    __syncthreads();
    for (int i = warp; i < live; i += 8) {   // one warp walks up one node's path
        float wk[CPL], wq[CPL], dot = 0.f;
#pragma unroll
        for (int r = 0; r < CPL; ++r) {
            const int c = r * 32 + lane;
            const float q = IO<T>::load((const T*)a.q, (tok0 + i * a.H) * DK + c);
            dot += q * kk[i * DK + c];
            wk[r] = kk[i * DK + c] * alpha[i * DK + c];
            wq[r] = q * alpha[i * DK + c];
        }
        dot = warp_sum(dot);
        if (lane == 0) AB[2 * (i * K) + 1] = dot;
        int place = 1;
        for (int j = par[i]; j >= 0; j = par[j], ++place) {
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int r = 0; r < CPL; ++r) {
                const int c = r * 32 + lane;
                x += wk[r] * kk[j * DK + c];
                y += wq[r] * kk[j * DK + c];
                wk[r] *= alpha[j * DK + c];
                wq[r] *= alpha[j * DK + c];
            }
            x = warp_sum(x);
            y = warp_sum(y);
            if (lane == 0) {
                AB[2 * (i * K + place)] = x;
                AB[2 * (i * K + place) + 1] = y;
            }
        }
#pragma unroll
        for (int r = 0; r < CPL; ++r) {
            W[i * DK + r * 32 + lane] = wk[r];
            W[(K + i) * DK + r * 32 + lane] = wq[r];
        }
    }
    __syncthreads();
    // one thread a column of S0: the products, then the nodes in order
    if (tid >= DV) return;
    float u[64];
    for (int i = 0; i < live; ++i) {
        float pk = 0.f, pq = 0.f;
        if (S0)
            for (int c = 0; c < DK; ++c) {
                const float s = S0[c * DV + tid];
                pk += W[i * DK + c] * s;
                pq += W[(K + i) * DK + c] * s;
            }
        int place = 1;
        for (int j = par[i]; j >= 0; j = par[j], ++place) {
            pk += AB[2 * (i * K + place)] * u[j];
            pq += AB[2 * (i * K + place) + 1] * u[j];
        }
        const int64_t at = (tok0 + i * a.H) * DV + tid;
        u[i] = bet[i] * (IO<T>::load((const T*)a.v, at) - pk);
        IO<T>::store((T*)a.out, at, a.scale * (pq + AB[2 * (i * K) + 1] * u[i]));
    }
}

// The accepted path's tokens applied to the cached state, in place: the decode step's
// arithmetic once per token, with the state in registers from the first to the last.
// One CTA of 256 threads for one (sequence, head).
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(256) tree_commit_kernel(TreeArgs a)
{
    constexpr int TPR = DV / 4;        // threads per state row (float4 each)
    constexpr int RG = 256 / TPR;      // row groups
    constexpr int RPT = DK / RG;       // rows per thread
    __shared__ float sk[DK], sa[DK], sv[DV], se[DV];
    __shared__ float4 red[RG][TPR];
    __shared__ int path[64];           // accepted node first
    __shared__ int count;
    const int tid = threadIdx.x, c4 = tid % TPR, rg = tid / TPR;
    const int64_t n = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const int K = (int)a.K;
    const int64_t sl = a.slots ? a.slots[n] : n;
    const int last = a.accepted[n];
    if (sl >= a.P || last >= K || last < -1) {
        if (tid == 0) atomicOr(a.err, kErrSeqlens);
        return;
    }
    if (sl < 0 || last < 0) return;
    float4* S4 = reinterpret_cast<float4*>(a.state + (sl * a.H + h) * (int64_t)DK * DV);
    float4 s[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r) s[r] = __ldcs(&S4[(rg * RPT + r) * TPR + c4]);
    if (tid == 0) {
        int c = 0;
        for (int i = last; i >= 0; i = tree_parent(a.parents + n * K, i, a.err)) path[c++] = i;
        count = c;
    }
    __syncthreads();
    for (int p = count - 1; p >= 0; --p) {
        const int64_t tok = (n * K + path[p]) * a.H + h;
        for (int i = tid; i < DK; i += 256) {
            sk[i] = IO<T>::load((const T*)a.k, tok * DK + i);
            sa[i] = expf(a.log_alpha[tok * DK + i]);
        }
        for (int j = tid; j < DV; j += 256) sv[j] = IO<T>::load((const T*)a.v, tok * DV + j);
        const float b = a.beta[tok];
        __syncthreads();
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < RPT; ++r) {
            const float al = sa[rg * RPT + r], kk = sk[rg * RPT + r];
            s[r].x *= al; s[r].y *= al; s[r].z *= al; s[r].w *= al;
            acc.x += kk * s[r].x; acc.y += kk * s[r].y; acc.z += kk * s[r].z; acc.w += kk * s[r].w;
        }
        red[rg][c4] = acc;
        __syncthreads();
        for (int j = tid; j < DV; j += 256) {
            float vh = 0.f;
#pragma unroll
            for (int g = 0; g < RG; ++g) vh += reinterpret_cast<const float*>(&red[g][0])[j];
            se[j] = b * (sv[j] - vh);
        }
        __syncthreads();
        const float4 e = reinterpret_cast<const float4*>(se)[c4];
#pragma unroll
        for (int r = 0; r < RPT; ++r) {
            const float kk = sk[rg * RPT + r];
            s[r].x += kk * e.x; s[r].y += kk * e.y; s[r].z += kk * e.z; s[r].w += kk * e.w;
        }
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r) __stcs(&S4[(rg * RPT + r) * TPR + c4], s[r]);
}

namespace {

template <typename T, int DK, int DV>
cudaError_t tree_fwd_t(const TreeArgs& a, cudaStream_t st)
{
    const size_t smem = (size_t)(4 * a.K * DK + 2 * a.K * a.K + a.K) * 4 + (size_t)a.K * 4;
    const cudaError_t e = cudaFuncSetAttribute(tree_fwd_kernel<T, DK, DV>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    LaunchScope scope(st, K_TREE_FWD);
    tree_fwd_kernel<T, DK, DV><<<(unsigned)(a.N * a.H), 256, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int DK, int DV>
cudaError_t tree_commit_t(const TreeArgs& a, cudaStream_t st)
{
    LaunchScope scope(st, K_TREE_COMMIT);
    tree_commit_kernel<T, DK, DV><<<(unsigned)(a.N * a.H), 256, 0, st>>>(a);
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
    if (N > 0x7fffffffLL || H > 0x7fffffffLL || N * H > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
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
