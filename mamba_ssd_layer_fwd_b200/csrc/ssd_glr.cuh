// Device arithmetic of the gated linear recurrence (ssd_glr.cu): the gates of
// one element, and the spans of sequences.
#pragma once

#include "ssd_common.cuh"

namespace ssd {

struct GlrArgs {
    const void *x, *r, *i;
    long long xs, rs, is;       // elements between tokens
    const float *A_log, *init;
    const int32_t *cu;          // NULL: nseq rows of T tokens; else one row of T tokens
    int *status;
    int D, T, nseq, nchunk;     // nchunk = ceil(T / SSD_GLR_CHUNK)
};

__device__ __forceinline__ float min_nan(float a, float b)   // NaN if either is
{
    float v;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ float ex2_approx(float v)
{
    float o;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(o) : "f"(v));
    return o;
}
__device__ __forceinline__ float rcp_approx(float v)
{
    float o;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(o) : "f"(v));
    return o;
}
__device__ __forceinline__ float rsqrt_approx(float v)
{
    float o;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(o) : "f"(v));
    return o;
}

struct Gate {
    float a, m, inv_m;          // exp(-q), sqrt(1 - a^2), 1 / m (finite at m = 0)
    float q;                    // exp(A_log) sigmoid(r)
    float si, osi, osr;         // sigmoid(i), sigmoid(-i), sigmoid(-r)
};

// One element's gates.  Four special-function operations: the two sigmoids
// share one reciprocal (exponents clamped so that the product of the
// denominators stays below 2^125), and exp(-q) is taken on the FMA units, since
// the special-function unit (16 lanes a clock and SM) would otherwise bound the
// kernels.  1 - a^2 = -e (1 + a) needs e = exp(-q) - 1 to full relative
// precision for small q: q = n ln2 + f (two-term ln2, the usual argument
// reduction), e = 2^-n p + (2^-n - 1) with p = exp(-f) - 1 from its Taylor
// series (|f| <= ln2 / 2: next term below 2e-8 of p).
__device__ __forceinline__ Gate gate(float r, float i, float rate)
{
    constexpr float kLog2e = 1.4426950408889634f;
    Gate g;
    const float er = ex2_approx(min_nan(r * -kLog2e, 62.0f));
    const float ei = ex2_approx(min_nan(i * -kLog2e, 62.0f));
    const float dr = 1.0f + er, di = 1.0f + ei;
    const float inv = rcp_approx(dr * di);
    const float sr = di * inv;
    g.si = dr * inv;
    g.osr = er * sr;
    g.osi = ei * g.si;
    const float q = min_nan(rate * sr, 87.0f);
    g.q = q;
    const float k = fmaf(q, kLog2e, 12582912.0f);           // 1.5 * 2^23: the sum's low bits are rint(q log2 e)
    const float n = k - 12582912.0f;
    float f = fmaf(n, 0.693359375f, -q);                    // -(q - n ln2), ln2 = 0.693359375 - 2.12194440e-4
    f = fmaf(n, -2.12194440e-4f, f);
    const float s = __int_as_float((127 << 23) - (__float_as_int(k) << 23));
    float p = fmaf(f, 1.0f / 5040.0f, 1.0f / 720.0f);
    p = fmaf(p, f, 1.0f / 120.0f);
    p = fmaf(p, f, 1.0f / 24.0f);
    p = fmaf(p, f, 1.0f / 6.0f);
    p = fmaf(p, f, 0.5f);
    p = fmaf(p * f, f, f);                                  // exp(f) - 1
    g.a = fmaf(s, p, s);
    const float e = fmaf(s, p, s - 1.0f);
    const float w = -e * (1.0f + g.a);                      // 1 - a^2
    g.inv_m = rsqrt_approx(fmaxf(w, 1.17549435e-38f));
    g.m = w * g.inv_m;
    return g;
}

// ---------------------------------------------------------------- vectors of V adjacent channels
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T v[V];
};

// Read once, so it is kept out of L1.
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_stream(const T *p)
{
    union {
        Vec<T, V> v;
        uint16_t h;
        uint32_t w[4];
    } u;
    if constexpr (sizeof(T) * V == 2)
        asm volatile("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=h"(u.h) : "l"(p));
    else if constexpr (sizeof(T) * V == 4)
        asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(u.w[0]) : "l"(p));
    else if constexpr (sizeof(T) * V == 8)
        asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(u.w[0]), "=r"(u.w[1]) : "l"(p));
    else
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.w[0]), "=r"(u.w[1]), "=r"(u.w[2]), "=r"(u.w[3]) : "l"(p));
    return u.v;
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const float (&f)[V])
{
    Vec<T, V> o;
#pragma unroll
    for (int k = 0; k < V; ++k) o.v[k] = from_f32<T>(f[k]);
    *reinterpret_cast<Vec<T, V> *>(p) = o;
}

template <int V>
__device__ __forceinline__ void load_f32(const float *p, float (&f)[V])
{
    const Vec<float, V> o = *reinterpret_cast<const Vec<float, V> *>(p);
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = o.v[k];
}

// ---------------------------------------------------------------- maps h -> A h + B
// A row's updates compose to such maps.  In a packed batch the first token of a
// sequence forgets what came before it: there A is exactly 0, and "A h" is left
// out rather than multiplied, so that a state that is not finite stays in its
// own sequence.
template <bool PACKED>
__device__ __forceinline__ float apply_map(float A, float B, float h)
{
    const float v = fmaf(A, h, B);
    return PACKED && A == 0.0f ? B : v;
}

// (A, B) <- (A2, B2) after (A, B)
template <bool PACKED>
__device__ __forceinline__ void compose_map(float &A, float &B, float A2, float B2)
{
    const bool cut = PACKED && A2 == 0.0f;
    B = cut ? B2 : fmaf(A2, B, B2);
    A = cut ? 0.0f : A * A2;
}

// ---------------------------------------------------------------- waits between CTAs
__device__ __forceinline__ int ld_acquire(const int *p)
{
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_release(int *p, int v)
{
    asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ uint64_t now_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Until *flag is set; after 2 s, or as soon as another wait of the call has
// given up, records the timeout and returns false.
__device__ __forceinline__ bool wait_flag(const int *flag, int *status)
{
    if (ld_acquire(flag)) return true;
    const uint64_t t0 = now_ns();
    for (uint32_t it = 1;; ++it) {
        if (ld_acquire(flag)) return true;
        if ((it & 127u) == 0) {
            if (*reinterpret_cast<volatile int *>(status) == kDevTimeout) return false;
            if (now_ns() - t0 > 2000000000ull) {
                atomicExch(status, kDevTimeout);
                return false;
            }
        }
    }
}

}  // namespace ssd
