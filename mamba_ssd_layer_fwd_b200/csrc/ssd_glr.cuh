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

struct SeqSpan {
    long long lo, hi;           // tokens of the sequence on the flattened axis, 0 <= lo <= hi
};

// Tokens of sequence s; a cu_seqlens that is not 0 = c0 <= ... <= T is recorded
// (`report`) and clamped, so that no access leaves the buffers.
__device__ __forceinline__ SeqSpan seq_span(const GlrArgs &g, int s, bool report)
{
    if (!g.cu) return {(long long)s * g.T, (long long)(s + 1) * g.T};
    const int a = g.cu[s], b = g.cu[s + 1];
    if (report && (a > b || (s == 0 && a != 0) || (s == g.nseq - 1 && b != g.T))) set_status(g.status, kDevBadSeqlens);
    const int lo = min(max(a, 0), g.T);
    return {lo, min(max(b, lo), g.T)};
}

}  // namespace ssd
