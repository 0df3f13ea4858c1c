// Layer norm forward and backward (include/ssd_norm.h).
//     y = (u - mean) rstd w + b,   u = x | round(x + residual) | x silu(z)
//     du = rstd (w dy - mean(w dy) - xhat mean(w dy xhat)),  dw = sum dy xhat,  db = sum dy
//
// All four kernels are bound by HBM: every input is read once, into registers,
// and the statistics are taken there.  Groups of up to kTeamMax elements are
// held by 8, 16 or 32 lanes of a warp (a block's output norm has groups of 64
// channels: eight lanes with 16 bytes each, four groups a warp), longer ones
// by a CTA.  A thread loads 16 bytes at a time where rows are aligned to that,
// single elements otherwise.
//
// Backward: a thread keeps its columns over all the rows that its CTA walks and
// sums dw and db in registers; the CTAs' sums go to the workspace and a second
// kernel adds them in order, so results do not depend on timing.
#include <algorithm>
#include <atomic>
#include <initializer_list>

#include "ssd_common.cuh"
#include "ssd_norm.h"
#include "ssd_tc_prims.cuh"

namespace ssd {
namespace {

struct NormArgs {
    const void *x, *z, *res, *dy, *dres;
    const float *w, *b, *mean, *rstd;
    long long xs, zs, rows;
    int D, G, P;
    float eps;
};

enum Mode { kPlain, kResidual, kGate };

// V elements at an address aligned to all of them (V > 1: 16 bytes)
template <typename T, int V> struct alignas(sizeof(T) * V) Pack {
    T v[V];
};
template <typename T, int V>
__device__ __forceinline__ void unpack(const Pack<T, V> &p, float (&f)[V])
{
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = to_f32(p.v[k]);
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T *p)
{
    return *reinterpret_cast<const Pack<T, V> *>(p);
}
// V values at an address aligned to min(16 bytes, all of them)
template <typename T, int V>
__device__ __forceinline__ void store_values(T *p, const float (&f)[V])
{
    constexpr int N = V * (int)sizeof(T) > 16 ? 16 / (int)sizeof(T) : V;
#pragma unroll
    for (int k = 0; k < V; k += N) {
        Pack<T, N> o;
#pragma unroll
        for (int q = 0; q < N; ++q) o.v[q] = from_f32<T>(f[k + q]);
        *reinterpret_cast<Pack<T, N> *>(p + k) = o;
    }
}
template <typename T, int V>
__device__ __forceinline__ void load_values(const T *p, float (&f)[V])
{
    constexpr int N = V * (int)sizeof(T) > 16 ? 16 / (int)sizeof(T) : V;
#pragma unroll
    for (int k = 0; k < V; k += N) {
        const Pack<T, N> o = load_pack<T, N>(p + k);
#pragma unroll
        for (int q = 0; q < N; ++q) f[k + q] = to_f32(o.v[q]);
    }
}

// V values of type T as they lie in memory
template <typename T, int V> struct Raw {
    static constexpr int N = V * (int)sizeof(T) > 16 ? 16 / (int)sizeof(T) : V;
    Pack<T, N> p[V / N];
    __device__ __forceinline__ void load(const T *from)
    {
#pragma unroll
        for (int k = 0; k < V / N; ++k) p[k] = load_pack<T, N>(from + k * N);
    }
    __device__ __forceinline__ float value(int v) const { return to_f32(p[v / N].v[v % N]); }
};

__device__ __forceinline__ float rcp_fast(float v)
{
    float o;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(o) : "f"(v));
    return o;
}
__device__ __forceinline__ float sigmoid(float z) { return rcp_fast(1.0f + tc::ex2_approx(z * -1.4426950408889634f)); }

// Sum over `lanes` (a power of two) neighbouring lanes, in all of them.
__device__ __forceinline__ float team_sum(float v, int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the CTA (whole warps, at most 32), in all threads.  One barrier;
// `slots` must not be the ones of the call before.
__device__ __forceinline__ float cta_sum(float v, float *slots)
{
    v = team_sum(v, 32);
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) slots[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < nw ? slots[lane] : 0.0f;
    return team_sum(v, 32);
}

// ---------------------------------------------------------------- forward

// One unit (a group of a row): lane `t` of its team of n holds the vectors t,
// t + n, ... of V channels.  Sum is a callable that adds a value over the team.
template <typename T, int V, int NV, Mode M, typename Sum>
__device__ __forceinline__ void norm_unit(const NormArgs &a, long long row, int g, int t, int n, bool live, T *y, T *sum,
                                          float *mean, float *rstd, Sum team)
{
    const int c0 = g * a.P;
    const T *x = static_cast<const T *>(a.x) + row * a.xs + c0;
    const T *z = M == kGate ? static_cast<const T *>(a.z) + row * a.zs + c0 : nullptr;
    const long long at = row * a.D + c0;
    Pack<T, V> xr[NV], zr[M == kPlain ? 1 : NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (t + k * n) * V;
        if (live && c < a.P) {
            xr[k] = load_pack<T, V>(x + c);
            if (M == kGate) zr[k] = load_pack<T, V>(z + c);
            if (M == kResidual) zr[k] = load_pack<T, V>(static_cast<const T *>(a.res) + at + c);
        }
    }
    float u[NV][V], s = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (t + k * n) * V;
        const bool in = live && c < a.P;
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float f = 0.0f;
            if (in) {
                f = to_f32(xr[k].v[v]);
                if (M == kGate) {
                    const float zv = to_f32(zr[k].v[v]);
                    f *= zv * sigmoid(zv);
                }
                if (M == kResidual) f = to_f32(from_f32<T>(f + to_f32(zr[k].v[v])));
            }
            u[k][v] = o[v] = f;
            s += f;
        }
        if (M == kResidual && in) store_values<T, V>(sum + at + c, o);
    }
    const float inv = 1.0f / a.P;
    s = team(s);
    float mu = s * inv;
    mu = fmaf(fmaf(-mu, (float)a.P, s), inv, mu);   // s / P rounded once: a row of one value has no spread
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const bool in = live && (t + k * n) * V < a.P;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            u[k][v] -= mu;
            if (in) s = fmaf(u[k][v], u[k][v], s);
        }
    }
    const float rs = rsqrtf(fmaf(team(s), inv, a.eps));
    if (!live) return;
    if (t == 0) {
        if (mean) mean[row * a.G + g] = mu;
        if (rstd) rstd[row * a.G + g] = rs;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (t + k * n) * V;
        if (c >= a.P) break;
        float w[V], b[V], o[V];
        load_values<float, V>(a.w + c0 + c, w);
        if (a.b) load_values<float, V>(a.b + c0 + c, b);
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = fmaf(u[k][v] * rs, w[v], a.b ? b[v] : 0.0f);
        store_values<T, V>(y + at + c, o);
    }
}

constexpr int kTeamThreads = 256;

// lanes: 8, 16 or 32 with lanes V NV >= P
template <typename T, int V, int NV, Mode M>
__global__ void __launch_bounds__(kTeamThreads)
norm_fwd_team_kernel(NormArgs a, int lanes, T *__restrict__ y, T *__restrict__ sum, float *__restrict__ mean,
                     float *__restrict__ rstd)
{
    const unsigned unit = blockIdx.x * (kTeamThreads / lanes) + threadIdx.x / lanes;
    const unsigned row = unit / a.G;
    norm_unit<T, V, NV, M>(a, row, unit - row * a.G, threadIdx.x & (lanes - 1), lanes, row < a.rows, y, sum, mean, rstd,
                           [&](float v) { return team_sum(v, lanes); });
}

template <typename T, int V, int NV, Mode M>
__global__ void __launch_bounds__(1024)
norm_fwd_cta_kernel(NormArgs a, T *__restrict__ y, T *__restrict__ sum, float *__restrict__ mean, float *__restrict__ rstd)
{
    __shared__ float slots[2][32];
    int turn = 0;
    const unsigned unit = blockIdx.x, row = unit / a.G;
    norm_unit<T, V, NV, M>(a, row, unit - row * a.G, threadIdx.x, blockDim.x, true, y, sum, mean, rstd,
                           [&](float v) { return cta_sum(v, slots[turn++]); });
}

// ---------------------------------------------------------------- backward

// A thread's V columns of one row.
template <int V> struct Cols {
    float xh[V], wd[V], dy[V];      // xhat, w dy, dy
    float x[V], z[V], sz[V];        // gate: x, z, sigmoid(z)
};

template <typename T, int V, bool GATE>
__device__ __forceinline__ void columns(const Pack<T, V> &x, const Pack<T, V> &z, const Pack<T, V> &dy,
                                        const float (&w)[V], float mu, float rs, Cols<V> &o)
{
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float u = to_f32(x.v[v]);
        if (GATE) {
            o.x[v] = u;
            o.z[v] = to_f32(z.v[v]);
            o.sz[v] = sigmoid(o.z[v]);
            u *= o.z[v] * o.sz[v];
        }
        o.xh[v] = (u - mu) * rs;
        o.dy[v] = to_f32(dy.v[v]);
        o.wd[v] = o.dy[v] * w[v];
    }
}

template <typename G, int V, bool GATE>
__device__ __forceinline__ void write_columns(const Cols<V> &k, float rs, float s1, float s2, bool has_res,
                                              const Raw<G, V> &dres, G *dx, G *dz)
{
    float o[V], oz[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float du = rs * (k.wd[v] - s1 - k.xh[v] * s2);
        if (GATE) {
            o[v] = du * k.z[v] * k.sz[v];
            oz[v] = du * k.x[v] * (k.sz[v] * fmaf(k.z[v], 1.0f - k.sz[v], 1.0f));
        } else {
            o[v] = has_res ? du + dres.value(v) : du;
        }
    }
    store_values<G, V>(dx, o);
    if (GATE) store_values<G, V>(dz, oz);
}

// Warps of a CTA share 32 / lanes neighbouring groups and take rows in turn.
// part: [CTA of the columns][2][D].
template <typename T, typename G, int V, int NV, bool GATE>
__global__ void __launch_bounds__(kTeamThreads)
norm_bwd_team_kernel(NormArgs a, int lanes, int ncols, G *__restrict__ dx, G *__restrict__ dz, float *__restrict__ part)
{
    constexpr int W = kTeamThreads / 32;
    __shared__ float red[W][32 * V];
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5, t = lane & (lanes - 1);
    const int col = blockIdx.x % ncols, split = blockIdx.x / ncols, nsplit = gridDim.x / ncols;
    const int g = col * (32 / lanes) + lane / lanes, c0 = g * a.P;
    const bool live = g < a.G;
    const float inv = 1.0f / a.P;
    float w[NV][V], dw[NV][V], db[NV][V];
    bool in[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (t + k * lanes) * V;
        in[k] = live && c < a.P;
#pragma unroll
        for (int v = 0; v < V; ++v) w[k][v] = dw[k][v] = db[k][v] = 0.0f;
        if (in[k]) load_values<float, V>(a.w + c0 + c, w[k]);
    }
    for (long long row = (long long)split * W + wp; row < a.rows; row += (long long)nsplit * W) {
        const T *x = static_cast<const T *>(a.x) + row * a.xs + c0;
        const T *z = GATE ? static_cast<const T *>(a.z) + row * a.zs + c0 : nullptr;
        const long long at = row * a.D + c0;
        Pack<T, V> xr[NV], zr[GATE ? NV : 1], dr[NV];
        Raw<G, V> res[GATE ? 1 : NV];
        float mu = 0.0f, rs = 0.0f;
        if (live) mu = a.mean[row * a.G + g], rs = a.rstd[row * a.G + g];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (t + k * lanes) * V;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (!in[k]) xr[k].v[v] = dr[k].v[v] = zr[GATE ? k : 0].v[v] = from_f32<T>(0.0f);
            if (in[k]) {
                xr[k] = load_pack<T, V>(x + c);
                dr[k] = load_pack<T, V>(static_cast<const T *>(a.dy) + at + c);
                if (GATE) zr[k] = load_pack<T, V>(z + c);
                if (!GATE && a.dres) res[k].load(static_cast<const G *>(a.dres) + at + c);
            }
        }
        Cols<V> cl[NV];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            columns<T, V, GATE>(xr[k], zr[GATE ? k : 0], dr[k], w[k], mu, rs, cl[k]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s1 += cl[k].wd[v];
                s2 = fmaf(cl[k].wd[v], cl[k].xh[v], s2);
                dw[k][v] = fmaf(cl[k].dy[v], cl[k].xh[v], dw[k][v]);
                db[k][v] += cl[k].dy[v];
            }
        }
        s1 = team_sum(s1, lanes) * inv;
        s2 = team_sum(s2, lanes) * inv;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (in[k]) {
                const long long o = at + (t + k * lanes) * V;
                write_columns<G, V, GATE>(cl[k], rs, s1, s2, a.dres != nullptr, res[GATE ? 0 : k], dx + o, GATE ? dz + o : nullptr);
            }
    }
    // the warps' sums, in order
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < V; ++v) red[wp][lane * V + v] = q ? db[k][v] : dw[k][v];
            __syncthreads();
            for (int j = threadIdx.x; j < 32 * V; j += kTeamThreads) {
                const int l = j / V, gj = col * (32 / lanes) + l / lanes, c = ((l & (lanes - 1)) + k * lanes) * V + j % V;
                if (gj < a.G && c < a.P) {
                    float s = 0.0f;
#pragma unroll
                    for (int i = 0; i < W; ++i) s += red[i][j];
                    part[((long long)split * 2 + q) * a.D + gj * a.P + c] = s;
                }
            }
        }
}

// A CTA keeps one group's columns and walks rows, R at a time: their sums meet
// at one barrier.  RING: thread 0 copies rows `nst` ahead into shared memory
// (rows aligned to 16 bytes), so HBM reads go on through the reduction;
// otherwise threads load their own columns.  The weights stay in registers
// where a thread has eight elements, and are read again for each row, from L1,
// where it has sixteen.
constexpr int kMaxStages = 6;

template <typename T, typename G, int V, int NV, int R, bool GATE, bool RING, int MAXT>
__global__ void __launch_bounds__(MAXT, 1)
norm_bwd_cta_kernel(NormArgs a, int nst, G *__restrict__ dx, G *__restrict__ dz, float *__restrict__ part)
{
    extern __shared__ __align__(128) char ring[];
    __shared__ float2 red[2][R][32];
    __shared__ uint64_t full[kMaxStages];
    __shared__ int abort_wait;
    constexpr bool KEEP = V * NV <= 8;
    const int t = threadIdx.x, n = blockDim.x, lane = t & 31, wp = t >> 5, nw = n >> 5;
    const int g = blockIdx.x % a.G, split = blockIdx.x / a.G, nsplit = gridDim.x / a.G, c0 = g * a.P;
    const float inv = 1.0f / a.P;
    const bool has_res = !GATE && a.dres != nullptr;
    const int row_t = a.P * (int)sizeof(T), row_g = has_res ? a.P * (int)sizeof(G) : 0;
    const int stage_bytes = (GATE ? 3 : 2) * row_t + row_g;
    const int count = split < a.rows ? (int)((a.rows - split + nsplit - 1) / nsplit) : 0;     // rows of this CTA
    const auto send = [&](int q) {                  // the CTA's q-th row
        const int stage = q % nst;
        char *to = ring + (size_t)stage * stage_bytes;
        const long long row = split + (long long)q * nsplit, at = row * a.D + c0;
        tc::mbar_arrive_expect_tx(&full[stage], stage_bytes);
        tc::bulk_load(to, static_cast<const T *>(a.x) + row * a.xs + c0, row_t, &full[stage]);
        tc::bulk_load(to + row_t, static_cast<const T *>(a.dy) + at, row_t, &full[stage]);
        if (GATE) tc::bulk_load(to + 2 * row_t, static_cast<const T *>(a.z) + row * a.zs + c0, row_t, &full[stage]);
        if (has_res) tc::bulk_load(to + 2 * row_t, static_cast<const G *>(a.dres) + at, row_g, &full[stage]);
    };
    if (RING && t == 0) {
        abort_wait = 0;
        for (int k = 0; k < nst; ++k) tc::mbar_init(&full[k], 1);
        tc::mbar_fence_init();
        for (int q = 0; q < min(nst, count); ++q) send(q);
    }
    float dw[NV][V], db[NV][V], w[KEEP ? NV : 1][V];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (t + k * n) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) dw[k][v] = db[k][v] = w[KEEP ? k : 0][v] = 0.0f;
        if (KEEP && c < a.P) load_values<float, V>(a.w + c0 + c, w[k]);
    }
    __syncthreads();
    float mu_next[R], rs_next[R];
    const auto stats = [&](int q, float &mu, float &rs) {
        mu = rs = 0.0f;
        if (q < count) {
            const long long at = (split + (long long)q * nsplit) * a.G + g;
            mu = a.mean[at], rs = a.rstd[at];
        }
    };
#pragma unroll
    for (int r = 0; r < R; ++r) stats(r, mu_next[r], rs_next[r]);
    int stage = 0, parity = 0, turn = 0;
    for (int q = 0; q < count; q += R) {
        float mu[R], rs[R];
        Pack<T, V> xr[R][NV], zr[R][GATE ? NV : 1], dr[R][NV];
        Raw<G, V> res[R][GATE ? 1 : NV];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mu[r] = mu_next[r], rs[r] = rs_next[r];
            stats(q + R + r, mu_next[r], rs_next[r]);
            const bool there = q + r < count;
            const long long row = split + (long long)(q + r) * nsplit, at = row * a.D + c0;
            const char *here = ring + (size_t)stage * stage_bytes;
            // a copy that does not arrive (2 s) is not waited for again: the row is then read in place
            const bool staged = RING && there && tc::mbar_wait(&full[stage], parity, &abort_wait);
            const T *x = staged ? reinterpret_cast<const T *>(here) : static_cast<const T *>(a.x) + row * a.xs + c0;
            const T *dy = staged ? reinterpret_cast<const T *>(here + row_t) : static_cast<const T *>(a.dy) + at;
            const T *z = !GATE ? nullptr : staged ? reinterpret_cast<const T *>(here + 2 * row_t)
                                                  : static_cast<const T *>(a.z) + row * a.zs + c0;
            const G *dres = !has_res ? nullptr : staged ? reinterpret_cast<const G *>(here + 2 * row_t)
                                                        : static_cast<const G *>(a.dres) + at;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (t + k * n) * V;
                if (there && c < a.P) {
                    xr[r][k] = load_pack<T, V>(x + c);
                    dr[r][k] = load_pack<T, V>(dy + c);
                    if (GATE) zr[r][k] = load_pack<T, V>(z + c);
                    if (!GATE && has_res) res[r][k].load(dres + c);
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) xr[r][k].v[v] = dr[r][k].v[v] = zr[r][GATE ? k : 0].v[v] = from_f32<T>(0.0f);
                }
            }
            if (++stage == nst) stage = 0, parity ^= 1;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                Cols<V> cl;
                const int c = (t + k * n) * V;
                float wk[V];
#pragma unroll
                for (int v = 0; v < V; ++v) wk[v] = KEEP ? w[KEEP ? k : 0][v] : 0.0f;
                if (!KEEP && c < a.P) load_values<float, V>(a.w + c0 + c, wk);
                columns<T, V, GATE>(xr[r][k], zr[r][GATE ? k : 0], dr[r][k], wk, mu[r], rs[r], cl);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    s1 += cl.wd[v];
                    s2 = fmaf(cl.wd[v], cl.xh[v], s2);
                    dw[k][v] = fmaf(cl.dy[v], cl.xh[v], dw[k][v]);
                    db[k][v] += cl.dy[v];
                }
            }
            s1 = team_sum(s1, 32);
            s2 = team_sum(s2, 32);
            if (lane == 0) red[turn][r][wp] = make_float2(s1, s2);
        }
        __syncthreads();                            // the rows are in registers: their stages are free
        if (RING && t == 0)
            for (int r = 0; r < R; ++r)
                if (q + r + nst < count) send(q + r + nst);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (q + r >= count) break;
            float2 s = make_float2(0.0f, 0.0f);
            if (lane < nw) s = red[turn][r][lane];
            const float s1 = team_sum(s.x, 32) * inv, s2 = team_sum(s.y, 32) * inv;
            const long long at = (split + (long long)(q + r) * nsplit) * a.D + c0;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (t + k * n) * V;
                if (c >= a.P) break;
                Cols<V> cl;
                float wk[V];
                if (KEEP) {
#pragma unroll
                    for (int v = 0; v < V; ++v) wk[v] = w[KEEP ? k : 0][v];
                } else {
                    load_values<float, V>(a.w + c0 + c, wk);
                }
                columns<T, V, GATE>(xr[r][k], zr[r][GATE ? k : 0], dr[r][k], wk, mu[r], rs[r], cl);
                write_columns<G, V, GATE>(cl, rs[r], s1, s2, has_res, res[r][GATE ? 0 : k], dx + at + c, GATE ? dz + at + c : nullptr);
            }
        }
        turn ^= 1;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (t + k * n) * V;
        if (c >= a.P) break;
        store_values<float, V>(part + ((long long)split * 2) * a.D + c0 + c, dw[k]);
        store_values<float, V>(part + ((long long)split * 2 + 1) * a.D + c0 + c, db[k]);
    }
}

// dw and db: the sums of n parts [n][2][D].  A CTA has 32 columns of one of
// them; eight warps take every eighth part and their sums are added in order.
__global__ void __launch_bounds__(256)
norm_dw_kernel(int n, int D, const float *__restrict__ part, float *__restrict__ dw, float *__restrict__ db)
{
    __shared__ float sums[8][32];
    float *out = blockIdx.y ? db : dw;
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < D) {
        const float *p = part + (long long)blockIdx.y * D + c;
        int k = wp;
        for (; k + 24 < n; k += 32)
#pragma unroll
            for (int u = 0; u < 4; ++u) s[u] += p[(long long)(k + 8 * u) * 2 * D];
        for (; k < n; k += 8) s[0] += p[(long long)k * 2 * D];
    }
    sums[wp][lane] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    if (wp == 0 && c < D) {
        float v = 0.0f;
        for (int k = 0; k < 8; ++k) v += sums[k][lane];
        out[c] = v;
    }
}

// ---------------------------------------------------------------- host side

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
    if (p->rows >= lim || p->x_stride >= lim || (gate && p->z_stride >= lim) || p->dim >= lim - 1024 ||
        p->rows * p->ngroups >= lim - 1024 || p->dim / p->ngroups > SSD_LAYER_NORM_MAX_GROUP)
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

// Whether rows and groups start on 16-byte boundaries, `v` elements of x's type.
bool wide(const NormArgs &a, int v, std::initializer_list<const void *> ptrs)
{
    if (a.P % v || a.xs % v || (a.z && a.zs % v)) return false;
    for (const void *q : ptrs)
        if (!aligned(q, 16)) return false;
    return true;
}

int sm_count()
{
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
        cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

int lanes_of(int P, int V)
{
    int lanes = 8;
    while (lanes < 32 && lanes * V < P) lanes *= 2;
    return lanes;
}

// Whole warps that hold `vecs` vectors, nv a thread.
int threads_of(int vecs, int nv) { return ((vecs + nv - 1) / nv + 31) / 32 * 32; }

template <typename T, int V, int NV, Mode M>
void fwd_team(const NormArgs &a, T *y, T *sum, float *mean, float *rstd, cudaStream_t st)
{
    const int lanes = lanes_of(a.P, V);
    const unsigned per = kTeamThreads / lanes, units = (unsigned)(a.rows * a.G);
    norm_fwd_team_kernel<T, V, NV, M><<<(units + per - 1) / per, kTeamThreads, 0, st>>>(a, lanes, y, sum, mean, rstd);
}

template <typename T, int V, int NV, Mode M>
void fwd_cta(const NormArgs &a, T *y, T *sum, float *mean, float *rstd, cudaStream_t st)
{
    norm_fwd_cta_kernel<T, V, NV, M>
        <<<(unsigned)(a.rows * a.G), threads_of((a.P + V - 1) / V, NV), 0, st>>>(a, y, sum, mean, rstd);
}

// V elements a load (16 bytes or one).  A team holds up to 32 elements a lane,
// a CTA's thread up to 16: 512 threads have 8192 elements, 1024 the longest group.
template <typename T, int V, Mode M>
void fwd_mode(const NormArgs &a, void *y_, void *sum_, float *mean, float *rstd, cudaStream_t st)
{
    T *y = static_cast<T *>(y_), *sum = static_cast<T *>(sum_);
    const int vecs = (a.P + V - 1) / V;
    if constexpr (V == 1) {
        if (a.P <= 32) fwd_team<T, 1, 1, M>(a, y, sum, mean, rstd, st);
        else if (a.P <= 128) fwd_team<T, 1, 4, M>(a, y, sum, mean, rstd, st);
        else if (a.P <= 512) fwd_team<T, 1, 16, M>(a, y, sum, mean, rstd, st);
        else if (a.P <= 2048) fwd_cta<T, 1, 4, M>(a, y, sum, mean, rstd, st);
        else fwd_cta<T, 1, 16, M>(a, y, sum, mean, rstd, st);
    } else {
        constexpr int S = 16 / V;                   // vectors in 16 elements
        if (vecs <= 32) fwd_team<T, V, 1, M>(a, y, sum, mean, rstd, st);
        else if (vecs <= 64) fwd_team<T, V, 2, M>(a, y, sum, mean, rstd, st);
        else if (vecs <= 128) fwd_team<T, V, 4, M>(a, y, sum, mean, rstd, st);
        else if (vecs <= 384) fwd_cta<T, V, 1, M>(a, y, sum, mean, rstd, st);
        else if (vecs <= 1024 || S == 2) fwd_cta<T, V, 2, M>(a, y, sum, mean, rstd, st);
        else fwd_cta<T, V, S, M>(a, y, sum, mean, rstd, st);
    }
}

template <typename T, int V>
void fwd(const NormArgs &a, void *y, void *sum, float *mean, float *rstd, cudaStream_t st)
{
    if (a.res) fwd_mode<T, V, kResidual>(a, y, sum, mean, rstd, st);
    else if (a.z) fwd_mode<T, V, kGate>(a, y, sum, mean, rstd, st);
    else fwd_mode<T, V, kPlain>(a, y, sum, mean, rstd, st);
}

// The backward's CTA: eight elements a thread and two rows at a time up to 768
// threads (80 registers; one row with a gate), then sixteen and one row.
constexpr int kCtaThreads = 768;
int vectors_of(int vecs, int V) { return (vecs * V <= 8 * kCtaThreads ? 8 : 16) / V; }

// How the backward splits a call; the same for any alignment, so that the
// workspace can be sized before it is known.
struct Split {
    bool team;
    int lanes, ncols, nsplit, per_sm;
};

// CTAs that fit an SM's registers, 80 a thread (64 to 128 in CTAs of sixteen elements a thread: one).
int ctas_per_sm(int P, int V)
{
    const int vecs = (P + V - 1) / V, nv = vectors_of(vecs, V);
    return nv * V == 8 ? std::max(1, std::min(8, 65536 / (80 * threads_of(vecs, nv)))) : 1;
}

Split split_of(const ssd_layer_norm_params &p, int V)
{
    const int P = p.dim / p.ngroups;
    Split s{};
    s.team = P <= (V == 1 ? 256 : 512);             // at most 16 elements a lane (8: rows of single elements)
    const int64_t rows = std::max<int64_t>(p.rows, 1);
    if (s.team) {
        s.lanes = lanes_of(P, V);
        s.ncols = (p.ngroups + 32 / s.lanes - 1) / (32 / s.lanes);
        const int64_t most = (rows + kTeamThreads / 32 - 1) / (kTeamThreads / 32);
        s.nsplit = (int)std::min<int64_t>(most, std::max(1, sm_count() * 4 / s.ncols));
    } else {
        s.per_sm = ctas_per_sm(P, V);
        s.ncols = p.ngroups;
        s.nsplit = (int)std::min<int64_t>(rows, std::max(1, (sm_count() * s.per_sm + s.ncols - 1) / s.ncols));
    }
    return s;
}

struct BwdOut {
    void *dx, *dz;
    float *part;
};

template <typename T, typename G, int V, int NV, bool GATE>
cudaError_t bwd_team(const NormArgs &a, const Split &s, const BwdOut &o, cudaStream_t st)
{
    norm_bwd_team_kernel<T, G, V, NV, GATE><<<(unsigned)(s.ncols * s.nsplit), kTeamThreads, 0, st>>>(
        a, s.lanes, s.ncols, static_cast<G *>(o.dx), static_cast<G *>(o.dz), o.part);
    return cudaGetLastError();
}

template <typename T, typename G, int V, int NV, int R, bool GATE, int MAXT>
cudaError_t bwd_cta(const NormArgs &a, const Split &s, const BwdOut &o, cudaStream_t st)
{
    constexpr bool RING = V > 1;
    const auto kernel = norm_bwd_cta_kernel<T, G, V, NV, R, GATE, RING, MAXT>;
    size_t smem = 0;
    int nst = 1;
    if (RING) {
        // R stages at least: with 16 elements a thread the longest group's one has 192 KB, with 8 three have 216 KB
        const size_t stage = (size_t)a.P * ((GATE ? 3 : 2) * sizeof(T) + (a.dres ? sizeof(G) : 0));
        nst = (int)std::min<size_t>(kMaxStages, std::max<size_t>(R, (size_t)216 * 1024 / s.per_sm / stage));
        smem = nst * stage;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    kernel<<<(unsigned)(s.ncols * s.nsplit), threads_of((a.P + V - 1) / V, NV), smem, st>>>(
        a, nst, static_cast<G *>(o.dx), static_cast<G *>(o.dz), o.part);
    return cudaGetLastError();
}

template <typename T, typename G, int V, bool GATE>
cudaError_t bwd_gate(const NormArgs &a, const Split &s, const BwdOut &o, cudaStream_t st)
{
    const int vecs = (a.P + V - 1) / V;
    if constexpr (V == 1) {
        if (s.team) {
            if (a.P <= 32) return bwd_team<T, G, 1, 1, GATE>(a, s, o, st);
            return a.P <= 128 ? bwd_team<T, G, 1, 4, GATE>(a, s, o, st) : bwd_team<T, G, 1, 8, GATE>(a, s, o, st);
        }
    } else {
        if (s.team) {
            if (vecs <= 32) return bwd_team<T, G, V, 1, GATE>(a, s, o, st);
            if (vecs <= 64) return bwd_team<T, G, V, 2, GATE>(a, s, o, st);
            if constexpr (V == 4) return bwd_team<T, G, V, 4, GATE>(a, s, o, st);
        }
    }
    if (vectors_of(vecs, V) * V == 8) return bwd_cta<T, G, V, 8 / V, GATE ? 1 : 2, GATE, kCtaThreads>(a, s, o, st);
    if (vecs * V <= 8192) return bwd_cta<T, G, V, 16 / V, 1, GATE, 512>(a, s, o, st);
    return bwd_cta<T, G, V, 16 / V, 1, GATE, 1024>(a, s, o, st);
}

template <typename T, typename G, int V>
cudaError_t bwd(const NormArgs &a, const Split &s, const BwdOut &o, cudaStream_t st)
{
    return a.z ? bwd_gate<T, G, V, true>(a, s, o, st) : bwd_gate<T, G, V, false>(a, s, o, st);
}

size_t part_bytes(const ssd_layer_norm_params &p, int V) { return (size_t)split_of(p, V).nsplit * 2 * p.dim * sizeof(float); }

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
    const bool w16 = wide(a, 16 / (int)es, {x, residual, z, y, sum, weight, bias});
    if (p->io_dtype == SSD_DTYPE_BF16) {
        if (w16) fwd<__nv_bfloat16, 8>(a, y, sum, mean, rstd, st);
        else fwd<__nv_bfloat16, 1>(a, y, sum, mean, rstd, st);
    } else {
        if (w16) fwd<float, 4>(a, y, sum, mean, rstd, st);
        else fwd<float, 1>(a, y, sum, mean, rstd, st);
    }
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

size_t ssd_layer_norm_bwd_workspace_size(const ssd_layer_norm_params *p)
{
    if (validate(p, false) != SSD_OK) return 0;
    return std::max(part_bytes(*p, 1), part_bytes(*p, p->io_dtype == SSD_DTYPE_BF16 ? 8 : 4)) + 256;
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
    const int W = 16 / (int)es, V = wide(a, W, {x, z, weight, dy, dresidual, dx, dz}) ? W : 1;
    const Split s = split_of(*p, V);
    const BwdOut o{dx, dz, static_cast<float *>(workspace)};
    int parts = 0;
    if (p->rows > 0) {
        typedef __nv_bfloat16 H;
        const bool bf = p->io_dtype == SSD_DTYPE_BF16, gb = p->grad_dtype == SSD_DTYPE_BF16;
        cudaError_t e;
        if (bf && gb) e = V == 8 ? bwd<H, H, 8>(a, s, o, st) : bwd<H, H, 1>(a, s, o, st);
        else if (bf) e = V == 8 ? bwd<H, float, 8>(a, s, o, st) : bwd<H, float, 1>(a, s, o, st);
        else e = V == 4 ? bwd<float, float, 4>(a, s, o, st) : bwd<float, float, 1>(a, s, o, st);
        if (e != cudaSuccess) return SSD_ERR_CUDA;
        parts = s.nsplit;
    }
    norm_dw_kernel<<<dim3((p->dim + 31) / 32, dbias ? 2 : 1), 256, 0, st>>>(parts, p->dim, o.part, dweight, dbias);
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
