// Layer norm forward and backward (include/ssd_norm.h).
//     y = (u - mean) rstd w + b,   u = x | round(x + residual) | x silu(z)
// One CTA normalises one group of a row; the weight's gradient is a second
// kernel over columns.
#include "ssd_common.cuh"
#include "ssd_norm.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;

struct NormArgs {
    const void *x, *z, *res, *dy, *dres;
    const float *w, *b, *mean, *rstd;
    long long xs, zs, rows;
    int D, G, P;
    float eps;
};

__device__ __forceinline__ float block_sum(float v)
{
    __shared__ float part[kThreads / 32];
    __shared__ float total;
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        float t = 0.0f;
        for (int k = 0; k < kThreads / 32; ++k) t += part[k];
        total = t;
    }
    __syncthreads();
    const float t = total;
    __syncthreads();
    return t;
}

template <typename T>
__device__ __forceinline__ float input(const NormArgs &a, long long row, int c)
{
    float u = to_f32(static_cast<const T *>(a.x)[row * a.xs + c]);
    if (a.res) u = to_f32(from_f32<T>(u + to_f32(static_cast<const T *>(a.res)[row * a.D + c])));
    if (a.z) {
        const float z = to_f32(static_cast<const T *>(a.z)[row * a.zs + c]);
        u *= z / (1.0f + expf(-z));
    }
    return u;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_fwd_kernel(NormArgs a, T *__restrict__ y, T *__restrict__ sum, float *__restrict__ mean, float *__restrict__ rstd)
{
    const long long unit = blockIdx.x, row = unit / a.G;
    const int g = (int)(unit - row * a.G), c0 = g * a.P;
    float v = 0.0f;
    for (int c = threadIdx.x; c < a.P; c += kThreads) v += input<T>(a, row, c0 + c);
    const float mu = block_sum(v) / a.P;
    v = 0.0f;
    for (int c = threadIdx.x; c < a.P; c += kThreads) {
        const float d = input<T>(a, row, c0 + c) - mu;
        v = fmaf(d, d, v);
    }
    const float rs = 1.0f / sqrtf(block_sum(v) / a.P + a.eps);
    if (threadIdx.x == 0) {
        if (mean) mean[unit] = mu;
        if (rstd) rstd[unit] = rs;
    }
    for (int c = threadIdx.x; c < a.P; c += kThreads) {
        const float u = input<T>(a, row, c0 + c);
        const size_t at = (size_t)row * a.D + c0 + c;
        if (sum) sum[at] = from_f32<T>(u);
        y[at] = from_f32<T>(fmaf((u - mu) * rs, a.w[c0 + c], a.b ? a.b[c0 + c] : 0.0f));
    }
}

template <typename T, typename Gr>
__global__ void __launch_bounds__(kThreads) norm_dx_kernel(NormArgs a, Gr *__restrict__ dx, Gr *__restrict__ dz)
{
    const long long unit = blockIdx.x, row = unit / a.G;
    const int g = (int)(unit - row * a.G), c0 = g * a.P;
    const float mu = a.mean[unit], rs = a.rstd[unit];
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x; c < a.P; c += kThreads) {
        const float wd = to_f32(static_cast<const T *>(a.dy)[row * a.D + c0 + c]) * a.w[c0 + c];
        s1 += wd;
        s2 = fmaf(wd, (input<T>(a, row, c0 + c) - mu) * rs, s2);
    }
    s1 = block_sum(s1) / a.P;
    s2 = block_sum(s2) / a.P;
    for (int c = threadIdx.x; c < a.P; c += kThreads) {
        const size_t at = (size_t)row * a.D + c0 + c;
        const float wd = to_f32(static_cast<const T *>(a.dy)[at]) * a.w[c0 + c];
        float du = rs * (wd - s1 - (input<T>(a, row, c0 + c) - mu) * rs * s2);
        if (a.z) {
            const float z = to_f32(static_cast<const T *>(a.z)[row * a.zs + c0 + c]);
            const float sg = 1.0f / (1.0f + expf(-z));
            dz[at] = from_f32<Gr>(du * to_f32(static_cast<const T *>(a.x)[row * a.xs + c0 + c]) * sg * (1.0f + z * (1.0f - sg)));
            du *= z * sg;
        }
        if (a.dres) du += to_f32(static_cast<const Gr *>(a.dres)[at]);
        dx[at] = from_f32<Gr>(du);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_dw_kernel(NormArgs a, float *__restrict__ dw, float *__restrict__ db)
{
    const int c = blockIdx.x;
    float s1 = 0.0f, s2 = 0.0f;
    for (long long row = threadIdx.x; row < a.rows; row += kThreads) {
        const long long unit = row * a.G + c / a.P;
        const float dy = to_f32(static_cast<const T *>(a.dy)[row * a.D + c]);
        s1 += dy;
        s2 = fmaf(dy, (input<T>(a, row, c) - a.mean[unit]) * a.rstd[unit], s2);
    }
    s1 = block_sum(s1);
    s2 = block_sum(s2);
    if (threadIdx.x == 0) {
        dw[c] = s2;
        if (db) db[c] = s1;
    }
}

bool valid_dtype(ssd_dtype t) { return t == SSD_DTYPE_F32 || t == SSD_DTYPE_BF16; }
size_t elem_size(ssd_dtype t) { return t == SSD_DTYPE_BF16 ? 2 : 4; }
bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

ssd_status validate(const ssd_layer_norm_params *p, bool gate)
{
    if (!p || p->rows < 0 || p->dim < 1 || p->ngroups < 1 || p->dim % p->ngroups != 0) return SSD_ERR_INVALID_ARG;
    if (!valid_dtype(p->io_dtype) || (p->grad_dtype != SSD_DTYPE_F32 && p->grad_dtype != p->io_dtype))
        return SSD_ERR_INVALID_ARG;
    if (!(p->eps >= 0.0f) || p->x_stride < p->dim || (gate && p->z_stride < p->dim)) return SSD_ERR_INVALID_ARG;
    const int64_t lim = int64_t(1) << 31;
    if (p->rows * p->ngroups >= lim || p->rows >= lim || p->x_stride >= lim || (gate && p->z_stride >= lim) ||
        p->dim / p->ngroups > SSD_LAYER_NORM_MAX_GROUP)
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

NormArgs args_of(const ssd_layer_norm_params &p, const void *x, const void *z, const float *w)
{
    NormArgs a{};
    a.x = x; a.z = z; a.w = w;
    a.xs = p.x_stride; a.zs = p.z_stride; a.rows = p.rows;
    a.D = p.dim; a.G = p.ngroups; a.P = p.dim / p.ngroups;
    a.eps = p.eps;
    return a;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status ssd_layer_norm_fwd(const ssd_layer_norm_params *p, const void *x, const void *residual, const void *z,
                              const float *weight, const float *bias, void *y, void *sum, float *mean, float *rstd,
                              void *stream)
{
    const ssd_status v = validate(p, z != nullptr);
    if (v != SSD_OK) return v;
    if ((residual != nullptr) != (sum != nullptr) || (residual && z)) return SSD_ERR_INVALID_ARG;
    if (!weight || (p->rows > 0 && (!x || !y))) return SSD_ERR_INVALID_ARG;
    const size_t es = elem_size(p->io_dtype);
    for (const void *q : {x, residual, z, (const void *)y, (const void *)sum})
        if (!aligned(q, es)) return SSD_ERR_INVALID_ARG;
    for (const void *q : {(const void *)weight, (const void *)bias, (const void *)mean, (const void *)rstd})
        if (!aligned(q, 4)) return SSD_ERR_INVALID_ARG;
    if (p->rows == 0) return SSD_OK;
    NormArgs a = args_of(*p, x, z, weight);
    a.res = residual; a.b = bias;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)(p->rows * p->ngroups);
    if (p->io_dtype == SSD_DTYPE_BF16)
        norm_fwd_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a, static_cast<__nv_bfloat16 *>(y),
                                                                  static_cast<__nv_bfloat16 *>(sum), mean, rstd);
    else
        norm_fwd_kernel<float><<<grid, kThreads, 0, st>>>(a, static_cast<float *>(y), static_cast<float *>(sum), mean, rstd);
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

size_t ssd_layer_norm_bwd_workspace_size(const ssd_layer_norm_params *p)
{
    return validate(p, false) == SSD_OK ? 256 : 0;
}

ssd_status ssd_layer_norm_bwd(const ssd_layer_norm_params *p, const void *x, const void *z, const float *weight,
                              const float *mean, const float *rstd, const void *dy, const void *dresidual, void *dx,
                              void *dz, float *dweight, float *dbias, void *workspace, size_t workspace_bytes,
                              void *stream)
{
    const ssd_status v = validate(p, z != nullptr);
    if (v != SSD_OK) return v;
    if ((z != nullptr) != (dz != nullptr) || (dresidual && z)) return SSD_ERR_INVALID_ARG;
    if (!weight || !dweight || !workspace || !aligned(workspace, 256) ||
        workspace_bytes < ssd_layer_norm_bwd_workspace_size(p))
        return SSD_ERR_INVALID_ARG;
    if (p->rows > 0 && (!x || !mean || !rstd || !dy || !dx)) return SSD_ERR_INVALID_ARG;
    const size_t es = elem_size(p->io_dtype), gs = elem_size(p->grad_dtype);
    for (const void *q : {x, z, dy})
        if (!aligned(q, es)) return SSD_ERR_INVALID_ARG;
    for (const void *q : {dresidual, (const void *)dx, (const void *)dz})
        if (!aligned(q, gs)) return SSD_ERR_INVALID_ARG;
    for (const void *q : {weight, mean, rstd, (const float *)dweight, (const float *)dbias})
        if (!aligned(q, 4)) return SSD_ERR_INVALID_ARG;
    NormArgs a = args_of(*p, x, z, weight);
    a.mean = mean; a.rstd = rstd; a.dy = dy; a.dres = dresidual;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    typedef __nv_bfloat16 B;
    const unsigned grid = (unsigned)(p->rows * p->ngroups);
    const bool bf = p->io_dtype == SSD_DTYPE_BF16;
    if (grid > 0) {
        if (bf && p->grad_dtype == SSD_DTYPE_BF16)
            norm_dx_kernel<B, B><<<grid, kThreads, 0, st>>>(a, static_cast<B *>(dx), static_cast<B *>(dz));
        else if (bf)
            norm_dx_kernel<B, float><<<grid, kThreads, 0, st>>>(a, static_cast<float *>(dx), static_cast<float *>(dz));
        else
            norm_dx_kernel<float, float><<<grid, kThreads, 0, st>>>(a, static_cast<float *>(dx), static_cast<float *>(dz));
    }
    if (bf)
        norm_dw_kernel<B><<<p->dim, kThreads, 0, st>>>(a, dweight, dbias);
    else
        norm_dw_kernel<float><<<p->dim, kThreads, 0, st>>>(a, dweight, dbias);
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
