// Gated linear recurrence, h_t = exp(log_a_t) h_{t-1} + x_t per channel: the
// elementwise sibling of the delta rule (a vector state, the same per-channel
// decay).  One thread walks one channel of one sequence.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {

// Row of h0 / hT / the pool that holds sequence n's state; -1: none.
__device__ __forceinline__ int64_t glr_row(const GlrArgs& a, int64_t n, bool report)
{
    if (a.slots == nullptr) return n;
    const int64_t s = a.slots[n];
    if (s >= a.P && report && a.err) atomicOr(a.err, kErrSeqlens);
    return s >= 0 && s < a.P ? s : -1;
}

template <typename T>
__global__ void __launch_bounds__(128) glr_fwd_kernel(GlrArgs a)
{
    const int64_t n = blockIdx.x;
    const int64_t c = (int64_t)blockIdx.y * 128 + threadIdx.x;
    if (c >= a.D) return;
    int64_t bos, eos;
    const int64_t T_total = a.B * a.T;
    seq_range(a.cu, n, a.T, T_total, bos, eos);
    if (a.cu && c == 0 && (a.cu[n + 1] < a.cu[n] || a.cu[0] != 0 || a.cu[a.N] != T_total))
        atomicOr(a.err, kErrSeqlens);
    const int64_t row = glr_row(a, n, c == 0);
    float h = a.h0 && row >= 0 ? a.h0[row * a.D + c] : 0.f;
    const int64_t tiles = (a.T + KDA_GLR_TILE - 1) / KDA_GLR_TILE;
    for (int64_t t = bos; t < eos; ++t) {
        const int64_t b = t / a.T, tb = t - b * a.T;
        if (a.starts && tb % KDA_GLR_TILE == 0)
            a.starts[(b * tiles + tb / KDA_GLR_TILE) * a.D + c] = h;
        h = expf(a.log_a[t * a.D + c]) * h + IO<T>::load((const T*)a.x, t * a.D + c);
        if (a.out) IO<T>::store((T*)a.out, t * a.D + c, h);
    }
    if (a.hT && row >= 0) a.hT[row * a.D + c] = h;
}

template <typename T>
__global__ void __launch_bounds__(128) glr_bwd_kernel(GlrArgs a)
{
    const int64_t n = blockIdx.x;
    const int64_t c = (int64_t)blockIdx.y * 128 + threadIdx.x;
    if (c >= a.D) return;
    int64_t bos, eos;
    const int64_t T_total = a.B * a.T;
    seq_range(a.cu, n, a.T, T_total, bos, eos);
    if (a.cu && c == 0 && (a.cu[n + 1] < a.cu[n] || a.cu[0] != 0 || a.cu[a.N] != T_total))
        atomicOr(a.err, kErrSeqlens);
    const float h0 = a.h0 ? a.h0[n * a.D + c] : 0.f;
    const int64_t tiles = (a.T + KDA_GLR_TILE - 1) / KDA_GLR_TILE;
    float g = a.dhT ? a.dhT[n * a.D + c] : 0.f;
    float before[KDA_GLR_TILE];
    for (int64_t end = eos; end > bos;) {
        const int64_t b = (end - 1) / a.T, tile = (end - 1 - b * a.T) / KDA_GLR_TILE;
        const int64_t first = b * a.T + tile * KDA_GLR_TILE;
        const int64_t from = first > bos ? first : bos;
        float h = from == bos ? h0 : a.starts[(b * tiles + tile) * a.D + c];
        for (int64_t t = from; t < end; ++t) {
            before[t - from] = h;
            h = expf(a.log_a[t * a.D + c]) * h + IO<T>::load((const T*)a.x, t * a.D + c);
        }
        for (int64_t t = end - 1; t >= from; --t) {
            g += IO<T>::load((const T*)a.dout, t * a.D + c);
            IO<T>::store((T*)a.dx, t * a.D + c, g);
            g *= expf(a.log_a[t * a.D + c]);
            a.dlog_a[t * a.D + c] = g * before[t - from];
        }
        end = from;
    }
    if (a.dh0) a.dh0[n * a.D + c] = g;
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

cudaError_t launch_glr_fwd(const GlrArgs& a, cudaStream_t st)
{
    LaunchScope scope(st, K_GLR_FWD);
    const dim3 grid((unsigned)a.N, (unsigned)((a.D + 127) / 128));
    if (a.io == KDA_IO_F32) glr_fwd_kernel<float><<<grid, 128, 0, st>>>(a);
    else glr_fwd_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_glr_bwd(const GlrArgs& a, cudaStream_t st)
{
    LaunchScope scope(st, K_GLR_BWD);
    const dim3 grid((unsigned)a.N, (unsigned)((a.D + 127) / 128));
    if (a.io == KDA_IO_F32) glr_bwd_kernel<float><<<grid, 128, 0, st>>>(a);
    else glr_bwd_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>(a);
    return cudaGetLastError();
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
                if (overlap(res[i].p, res[i].n, q.p, q.n) && !(res[i].p == dh0 && q.p == dhT && dh0 == dhT))
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
