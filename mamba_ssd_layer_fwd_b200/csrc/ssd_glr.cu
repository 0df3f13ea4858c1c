// Gated linear recurrence (include/ssd_glr.h): a state of one value a channel,
//     q = exp(A_log) sigmoid(r),  a = exp(-q),  h <- a h + sqrt(1 - a^2) sigmoid(i) x,
// forward, backward and single-token step.  One thread walks one channel of
// one sequence.
#include "ssd_glr.cuh"
#include "ssd_glr.h"

namespace ssd {
namespace {

constexpr int kThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kThreads)
glr_fwd_kernel(GlrArgs g, T *__restrict__ y, float *__restrict__ final_states, float *__restrict__ chunk_states)
{
    const int c = blockIdx.y * kThreads + threadIdx.x, s = blockIdx.x;
    const SeqSpan span = seq_span(g, s, blockIdx.y == 0 && threadIdx.x == 0);
    if (c >= g.D) return;
    const float rate = expf(g.A_log[c]);
    float h = g.init ? g.init[(size_t)s * g.D + c] : 0.0f;
    for (long long t = span.lo; t < span.hi; ++t) {
        const long long in_row = g.cu ? t : t - span.lo;
        if (chunk_states && in_row % SSD_GLR_CHUNK == 0)
            chunk_states[((g.cu ? 0 : (long long)s * g.nchunk) + in_row / SSD_GLR_CHUNK) * g.D + c] = h;
        const Gate k = gate(to_f32(static_cast<const T *>(g.r)[t * g.rs + c]),
                            to_f32(static_cast<const T *>(g.i)[t * g.is + c]), rate);
        h = fmaf(k.a, h, k.m * k.si * to_f32(static_cast<const T *>(g.x)[t * g.xs + c]));
        if (y) y[t * g.D + c] = from_f32<T>(h);
    }
    if (final_states) final_states[(size_t)s * g.D + c] = h;
}

template <typename T, typename G>
__global__ void __launch_bounds__(kThreads)
glr_bwd_kernel(GlrArgs g, const float *__restrict__ chunk_states, const T *__restrict__ dy,
               const float *__restrict__ dfinal, G *__restrict__ dx, G *__restrict__ dr, G *__restrict__ di,
               float *__restrict__ dA_part, float *__restrict__ dinit)
{
    const int c = blockIdx.y * kThreads + threadIdx.x, s = blockIdx.x;
    const SeqSpan span = seq_span(g, s, blockIdx.y == 0 && threadIdx.x == 0);
    if (c >= g.D) return;
    const float rate = expf(g.A_log[c]);
    float carry = dfinal ? dfinal[(size_t)s * g.D + c] : 0.0f;
    float dA = 0.0f;
    const long long row0 = g.cu ? 0 : span.lo;
    float h[SSD_GLR_CHUNK];                                  // state before each token of a chunk
    for (long long k = (span.hi - 1 - row0) / SSD_GLR_CHUNK; span.hi > span.lo; --k) {
        const long long lo = max(row0 + k * SSD_GLR_CHUNK, span.lo);
        const long long hi = min(row0 + (k + 1) * SSD_GLR_CHUNK, span.hi);
        float v = lo > span.lo || (lo - row0) % SSD_GLR_CHUNK == 0
                      ? chunk_states[((g.cu ? 0 : (long long)s * g.nchunk) + k) * g.D + c]
                      : (g.init ? g.init[(size_t)s * g.D + c] : 0.0f);
        for (long long t = lo; t < hi; ++t) {
            h[t - lo] = v;
            const Gate q = gate(to_f32(static_cast<const T *>(g.r)[t * g.rs + c]),
                                to_f32(static_cast<const T *>(g.i)[t * g.is + c]), rate);
            v = fmaf(q.a, v, q.m * q.si * to_f32(static_cast<const T *>(g.x)[t * g.xs + c]));
        }
        for (long long t = hi - 1; t >= lo; --t) {
            const float x = to_f32(static_cast<const T *>(g.x)[t * g.xs + c]);
            const Gate q = gate(to_f32(static_cast<const T *>(g.r)[t * g.rs + c]),
                                to_f32(static_cast<const T *>(g.i)[t * g.is + c]), rate);
            const float gt = to_f32(dy[t * g.D + c]) + carry;
            const float gm = gt * q.m * q.si;
            // q dm/dq = q a^2 / m stays finite as q -> 0
            const float dqq = q.a * (q.q * q.a * q.inv_m * gt * q.si * x - q.q * gt * h[t - lo]);
            dx[t * g.D + c] = from_f32<G>(gm);
            di[t * g.D + c] = from_f32<G>(gm * x * q.osi);
            dr[t * g.D + c] = from_f32<G>(dqq * q.osr);
            dA += dqq;
            carry = q.a * gt;
        }
        if (lo == span.lo) break;
    }
    dA_part[(size_t)s * g.D + c] = dA;
    if (dinit) dinit[(size_t)s * g.D + c] = carry;
}

__global__ void __launch_bounds__(kThreads) glr_dA_kernel(int n, int D, const float *__restrict__ part, float *__restrict__ dA)
{
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= D) return;
    float v = 0.0f;
    for (int k = 0; k < n; ++k) v += part[(size_t)k * D + c];
    dA[c] = v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
glr_step_kernel(long long n, int D, const T *__restrict__ x, const T *__restrict__ r, const T *__restrict__ i,
                long long xs, long long rs, long long is, const float *__restrict__ A_log, float *__restrict__ state,
                T *__restrict__ y)
{
    const long long k = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (k >= n) return;
    const long long row = k / D;
    const int c = (int)(k - row * D);
    const Gate q = gate(to_f32(r[row * rs + c]), to_f32(i[row * is + c]), expf(A_log[c]));
    const float h = fmaf(q.a, state[k], q.m * q.si * to_f32(x[row * xs + c]));
    state[k] = h;
    y[k] = from_f32<T>(h);
}

bool valid_dtype(ssd_dtype t) { return t == SSD_DTYPE_F32 || t == SSD_DTYPE_BF16; }
size_t elem_size(ssd_dtype t) { return t == SSD_DTYPE_BF16 ? 2 : 4; }
bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

ssd_status validate(const ssd_glr_params *p)
{
    if (!p || p->batch < 1 || p->seqlen < 0 || p->channels < 1 || p->num_seqs < 0) return SSD_ERR_INVALID_ARG;
    if (p->num_seqs > 0 && p->batch != 1) return SSD_ERR_INVALID_ARG;
    if (!valid_dtype(p->io_dtype) || (p->grad_dtype != SSD_DTYPE_F32 && p->grad_dtype != p->io_dtype))
        return SSD_ERR_INVALID_ARG;
    if (p->x_stride < p->channels || p->r_stride < p->channels || p->i_stride < p->channels)
        return SSD_ERR_INVALID_ARG;
    const int64_t lim = int64_t(1) << 31;
    if ((int64_t)p->batch * p->seqlen >= lim - 1024 || p->x_stride >= lim || p->r_stride >= lim || p->i_stride >= lim ||
        p->num_seqs > (1 << 20) || p->channels >= (1 << 22))
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

constexpr size_t kAlign = 256;
size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
int nseq_of(const ssd_glr_params &p) { return p.num_seqs > 0 ? p.num_seqs : p.batch; }
int64_t chunks_of(const ssd_glr_params &p) { return ((int64_t)p.seqlen + SSD_GLR_CHUNK - 1) / SSD_GLR_CHUNK; }

GlrArgs args_of(const ssd_glr_params &p, const void *x, const void *r, const void *i, const float *A_log,
                const float *init, const int32_t *cu, void *ws)
{
    GlrArgs g;
    g.x = x; g.r = r; g.i = i; g.A_log = A_log; g.init = init; g.cu = cu;
    g.xs = p.x_stride; g.rs = p.r_stride; g.is = p.i_stride;
    g.D = p.channels; g.T = p.seqlen; g.nseq = nseq_of(p); g.nchunk = (int)chunks_of(p);
    g.status = static_cast<int *>(ws);
    return g;
}

template <typename T>
cudaError_t fwd(const GlrArgs &g, void *y, float *fin, float *chunks, cudaStream_t st)
{
    const dim3 grid(g.nseq, (g.D + kThreads - 1) / kThreads);
    glr_fwd_kernel<T><<<grid, kThreads, 0, st>>>(g, static_cast<T *>(y), fin, chunks);
    return cudaGetLastError();
}

template <typename T, typename G>
cudaError_t bwd(const GlrArgs &g, const float *chunks, const void *dy, const float *dfinal, void *dx, void *dr, void *di,
                float *part, float *dA, float *dinit, cudaStream_t st)
{
    const dim3 grid(g.nseq, (g.D + kThreads - 1) / kThreads);
    glr_bwd_kernel<T, G><<<grid, kThreads, 0, st>>>(g, chunks, static_cast<const T *>(dy), dfinal, static_cast<G *>(dx),
                                                    static_cast<G *>(dr), static_cast<G *>(di), part, dinit);
    glr_dA_kernel<<<grid.y, kThreads, 0, st>>>(g.nseq, g.D, part, dA);
    return cudaGetLastError();
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_glr_fwd_workspace_size(const ssd_glr_params *p)
{
    return validate(p) == SSD_OK ? kAlign : 0;
}

size_t ssd_glr_bwd_workspace_size(const ssd_glr_params *p, int with_chunk_states)
{
    if (validate(p) != SSD_OK) return 0;
    size_t n = kAlign + align_up((size_t)nseq_of(*p) * p->channels * sizeof(float));
    if (!with_chunk_states) n += align_up((size_t)p->batch * chunks_of(*p) * p->channels * sizeof(float));
    return n;
}

ssd_status ssd_glr_fwd(const ssd_glr_params *p, const void *x, const void *r, const void *i, const float *A_log,
                       const float *initial_states, const int32_t *cu_seqlens, void *y, float *final_states,
                       float *chunk_states, void *workspace, size_t workspace_bytes, void *stream)
{
    const ssd_status v = validate(p);
    if (v != SSD_OK) return v;
    const size_t es = elem_size(p->io_dtype);
    if (!A_log || !workspace || !aligned(workspace, kAlign) || workspace_bytes < ssd_glr_fwd_workspace_size(p))
        return SSD_ERR_INVALID_ARG;
    if (p->seqlen > 0 && (!x || !r || !i || !y)) return SSD_ERR_INVALID_ARG;
    if ((p->num_seqs > 0) != (cu_seqlens != nullptr)) return SSD_ERR_INVALID_ARG;
    if (!aligned(x, es) || !aligned(r, es) || !aligned(i, es) || !aligned(y, es)) return SSD_ERR_INVALID_ARG;
    for (const void *q : {(const void *)A_log, (const void *)initial_states, (const void *)cu_seqlens,
                          (const void *)final_states, (const void *)chunk_states})
        if (!aligned(q, 4)) return SSD_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(workspace, 0, sizeof(int), st) != cudaSuccess) return SSD_ERR_CUDA;
    const GlrArgs g = args_of(*p, x, r, i, A_log, initial_states, cu_seqlens, workspace);
    const cudaError_t e = p->io_dtype == SSD_DTYPE_BF16 ? fwd<__nv_bfloat16>(g, y, final_states, chunk_states, st)
                                                        : fwd<float>(g, y, final_states, chunk_states, st);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_glr_bwd(const ssd_glr_params *p, const void *x, const void *r, const void *i, const float *A_log,
                       const float *initial_states, const int32_t *cu_seqlens, const float *chunk_states,
                       const void *dy, const float *dfinal_states, void *dx, void *dr, void *di, float *dA_log,
                       float *dinitial_states, void *workspace, size_t workspace_bytes, void *stream)
{
    const ssd_status v = validate(p);
    if (v != SSD_OK) return v;
    const size_t es = elem_size(p->io_dtype), gs = elem_size(p->grad_dtype);
    if (!A_log || !dA_log || !workspace || !aligned(workspace, kAlign) ||
        workspace_bytes < ssd_glr_bwd_workspace_size(p, chunk_states != nullptr))
        return SSD_ERR_INVALID_ARG;
    if (p->seqlen > 0 && (!x || !r || !i || !dy || !dx || !dr || !di)) return SSD_ERR_INVALID_ARG;
    if ((p->num_seqs > 0) != (cu_seqlens != nullptr)) return SSD_ERR_INVALID_ARG;
    if (!aligned(x, es) || !aligned(r, es) || !aligned(i, es) || !aligned(dy, es) || !aligned(dx, gs) ||
        !aligned(dr, gs) || !aligned(di, gs))
        return SSD_ERR_INVALID_ARG;
    for (const void *q : {(const void *)A_log, (const void *)initial_states, (const void *)cu_seqlens,
                          (const void *)chunk_states, (const void *)dfinal_states, (const void *)dA_log,
                          (const void *)dinitial_states})
        if (!aligned(q, 4)) return SSD_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(workspace, 0, sizeof(int), st) != cudaSuccess) return SSD_ERR_CUDA;
    const GlrArgs g = args_of(*p, x, r, i, A_log, initial_states, cu_seqlens, workspace);
    char *ws = static_cast<char *>(workspace);
    float *part = reinterpret_cast<float *>(ws + kAlign);
    const float *chunks = chunk_states;
    const bool bf = p->io_dtype == SSD_DTYPE_BF16;
    if (!chunks) {
        float *c = reinterpret_cast<float *>(ws + kAlign + align_up((size_t)g.nseq * g.D * sizeof(float)));
        const cudaError_t e = bf ? fwd<__nv_bfloat16>(g, nullptr, nullptr, c, st) : fwd<float>(g, nullptr, nullptr, c, st);
        if (e != cudaSuccess) return SSD_ERR_CUDA;
        chunks = c;
    }
    cudaError_t e;
    if (bf && p->grad_dtype == SSD_DTYPE_BF16)
        e = bwd<__nv_bfloat16, __nv_bfloat16>(g, chunks, dy, dfinal_states, dx, dr, di, part, dA_log, dinitial_states, st);
    else if (bf)
        e = bwd<__nv_bfloat16, float>(g, chunks, dy, dfinal_states, dx, dr, di, part, dA_log, dinitial_states, st);
    else
        e = bwd<float, float>(g, chunks, dy, dfinal_states, dx, dr, di, part, dA_log, dinitial_states, st);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_glr_step(const ssd_glr_step_params *p, const void *x, const void *r, const void *i, const float *A_log,
                        float *state, void *y, void *stream)
{
    if (!p || p->batch < 0 || p->channels < 1 || !valid_dtype(p->io_dtype) || p->x_stride < p->channels ||
        p->r_stride < p->channels || p->i_stride < p->channels)
        return SSD_ERR_INVALID_ARG;
    if (p->batch == 0) return SSD_OK;
    const size_t es = elem_size(p->io_dtype);
    if (!x || !r || !i || !A_log || !state || !y || !aligned(x, es) || !aligned(r, es) || !aligned(i, es) ||
        !aligned(y, es) || !aligned(A_log, 4) || !aligned(state, 4))
        return SSD_ERR_INVALID_ARG;
    const long long n = (long long)p->batch * p->channels, blocks = (n + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffLL) return SSD_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p->io_dtype == SSD_DTYPE_BF16) {
        typedef __nv_bfloat16 T;
        glr_step_kernel<T><<<(unsigned)blocks, kThreads, 0, st>>>(
            n, p->channels, static_cast<const T *>(x), static_cast<const T *>(r), static_cast<const T *>(i),
            p->x_stride, p->r_stride, p->i_stride, A_log, state, static_cast<T *>(y));
    } else {
        typedef float T;
        glr_step_kernel<T><<<(unsigned)blocks, kThreads, 0, st>>>(
            n, p->channels, static_cast<const T *>(x), static_cast<const T *>(r), static_cast<const T *>(i),
            p->x_stride, p->r_stride, p->i_stride, A_log, state, static_cast<T *>(y));
    }
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
