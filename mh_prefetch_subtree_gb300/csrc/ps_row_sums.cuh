// Sums over a logits row relative to a reference, and how a row is finished from
// them: shared by the scoring kernels (ps_score_rows.cu has the formulation).
#pragma once

#include <math.h>

#include "ps_internal.cuh"

namespace ps {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2f = 0.6931471805599453f;
constexpr float kLimit = 1.8446744073709552e19f;   // 2^64: largest chunk sum kept as is
constexpr uint32_t kAbsent = 0x7fc0deadu;           // "token not in this part" (a NaN payload
                                                    // no bf16/f32 logit converts to)
// Entropy variant: logits below -1e30 (that is, -inf) are raised to -1e30, so
// that 2^y * y is 0 * (finite) = 0 instead of 0 * (-inf) = NaN.  The exponential
// of such a value is 0 either way; NaN is kept (the max propagates it).
constexpr uint32_t kFloorBf16x2 = 0xf14af14au;      // (-1.0009e30, -1.0009e30) as bf16x2
constexpr float kFloorF32 = -1.0e30f;

template <int DT>
struct Elem;
template <>
struct Elem<PS_BF16> {
    static constexpr int kSize = 2;
    static constexpr uint32_t kNegInfWord = 0xff80ff80u;
    static constexpr uint32_t kFloorWord = 0xf14af14au;   // two bf16 -1.0009e30
    static constexpr uint16_t kFloorElem = 0xf14au;
};
template <>
struct Elem<PS_F32> {
    static constexpr int kSize = 4;
    static constexpr uint32_t kNegInfWord = 0xff800000u;
    static constexpr uint32_t kFloorWord = 0xf149f2cau;   // -1.0e30f
};
// Values at or below this are taken as absent (-inf) when the maximum is sought.
constexpr float kAbsentBelow = -9.0e29f;

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ float max_nan_f32(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// NP == kAllPowers or kPowersTo4: one pass serves several temperatures whose
// 1/tau is 1, 2, 4 or 8 (the MultiTryMH set {0.25, 0.5, 1} among them): from
// 2^y the powers 2^(2y), 2^(4y) (and, for kAllPowers, 2^(8y)) are squares,
// and their sums are kept side by side.
constexpr int kAllPowers = 16;     // sums of 2^(2y), 2^(4y), 2^(8y)
constexpr int kPowersTo4 = 17;     // sums of 2^(2y), 2^(4y)

template <int NP>
__host__ __device__ constexpr bool multi_tau() { return NP == kAllPowers || NP == kPowersTo4; }

template <int NP>
__host__ __device__ constexpr int n_tau_sums() {
    return NP == kAllPowers ? 3 : (NP == kPowersTo4 ? 2 : 1);
}

// Running sums of one lane (or one merged part) relative to reference R.
// st[k] is the tau sum (multi-temperature: the sum of 2^(2^(k+1) y)).
struct Acc {
    float R;
    float s1;
    float st[3];
    float y1;
};

__device__ __forceinline__ Acc acc_empty() { return Acc{-INFINITY, 0.f, {0.f, 0.f, 0.f}, 0.f}; }

// One pair of logits v: accumulate 2^x into a1, 2^(g x) into at[0] (or the
// three power sums into at[0..2]) and 2^x x into ay, with x = v L - R.  For a
// general g the tau exponent g x = v (g L) - g R is formed from v directly
// (GL2, nGR2), so that it does not wait for x.
template <int NP, bool ENT>
__device__ __forceinline__ void step2(float2 v, float2 L2, float2 nR2, float2 GL2, float2 nGR2,
                                      float2 &a1, float2 (&at)[3], float2 &ay) {
    const float2 x = __ffma2_rn(v, L2, nR2);
    const float2 e = make_float2(ex2(x.x), ex2(x.y));
    a1 = __fadd2_rn(a1, e);
    if constexpr (ENT) ay = __ffma2_rn(e, x, ay);
    if constexpr (NP == 2) {
        at[0] = __fadd2_rn(at[0], __fmul2_rn(e, e));
    } else if constexpr (NP == 4) {
        const float2 e2 = __fmul2_rn(e, e);
        at[0] = __fadd2_rn(at[0], __fmul2_rn(e2, e2));
    } else if constexpr (NP == 8) {
        const float2 e2 = __fmul2_rn(e, e);
        const float2 e4 = __fmul2_rn(e2, e2);
        at[0] = __fadd2_rn(at[0], __fmul2_rn(e4, e4));
    } else if constexpr (multi_tau<NP>()) {
        const float2 e2 = __fmul2_rn(e, e);
        const float2 e4 = __fmul2_rn(e2, e2);
        at[0] = __fadd2_rn(at[0], e2);
        at[1] = __fadd2_rn(at[1], e4);
        if constexpr (NP == kAllPowers) at[2] = __fadd2_rn(at[2], __fmul2_rn(e4, e4));
    } else if constexpr (NP == 0) {
        const float2 xt = __ffma2_rn(v, GL2, nGR2);
        at[0] = __fadd2_rn(at[0], make_float2(ex2(xt.x), ex2(xt.y)));
    }
}

__device__ __forceinline__ float hsum4(const float2 (&a)[4]) {
    const float2 s01 = __fadd2_rn(a[0], a[1]), s23 = __fadd2_rn(a[2], a[3]);
    const float2 s = __fadd2_rn(s01, s23);
    return s.x + s.y;
}

// Sums of one lane's VPL vectors relative to reference R: c1, ct[0..NS-1], cy.
// CLAMP (entropy only) raises -inf inputs to a large negative finite value
// first, so that 2^y y is 0 rather than NaN there; without it the caller must
// see to it that no -inf is in q (a NaN sum sends the chunk down the slow path).
template <int DT, int NP, bool ENT, int VPL, bool CLAMP = ENT>
__device__ __forceinline__ void sum_vecs(const uint4 (&q)[VPL], float R, float g, float &c1,
                                         float (&ct)[3], float &cy) {
    const float2 L2 = make_float2(kLog2e, kLog2e);
    const float2 nR2 = make_float2(-R, -R);
    const float2 GL2 = make_float2(g * kLog2e, g * kLog2e);
    const float2 nGR2 = make_float2(-g * R, -g * R);
    float2 a1[4], at[4][3], ay[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        a1[j] = make_float2(0.f, 0.f);
        at[j][0] = at[j][1] = at[j][2] = make_float2(0.f, 0.f);
        ay[j] = make_float2(0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
        if constexpr (DT == PS_BF16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (ENT && CLAMP) w[j] = max_nan_bf16x2(w[j], kFloorBf16x2);
                const float2 v = make_float2(__uint_as_float(w[j] << 16),
                                             __uint_as_float(w[j] & 0xffff0000u));
                step2<NP, ENT>(v, L2, nR2, GL2, nGR2, a1[j], at[j], ay[j]);
            }
        } else {
            float f[4] = {__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]),
                          __uint_as_float(w[3])};
            if constexpr (ENT && CLAMP) {
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = max_nan_f32(f[j], kFloorF32);
            }
            step2<NP, ENT>(make_float2(f[0], f[1]), L2, nR2, GL2, nGR2, a1[(i & 1) * 2],
                           at[(i & 1) * 2], ay[(i & 1) * 2]);
            step2<NP, ENT>(make_float2(f[2], f[3]), L2, nR2, GL2, nGR2, a1[(i & 1) * 2 + 1],
                           at[(i & 1) * 2 + 1], ay[(i & 1) * 2 + 1]);
        }
    }
    c1 = hsum4(a1);
    if constexpr (NP == 1) {
        ct[0] = c1;
    } else {
#pragma unroll
        for (int k = 0; k < n_tau_sums<NP>(); ++k) {
            const float2 t[4] = {at[0][k], at[1][k], at[2][k], at[3][k]};
            ct[k] = hsum4(t);
        }
    }
    cy = ENT ? hsum4(ay) : 0.f;
}

// Rescale factor of tau sum k when the reference moves by d (log2 units).
template <int NP>
__device__ __forceinline__ float tau_scale(float d, float g, int k) {
    if constexpr (NP == 0) return ex2(d * g);
    else if constexpr (multi_tau<NP>()) return ex2(d * (float)(2 << k));
    else return ex2(d * (float)NP);
}

// Moves the reference of `a` from a.R to Rn >= a.R.  With y' = y - D,
// D = Rn - R: sum 2^y' = 2^-D S1 and sum 2^y' y' = 2^-D (Y1 - D S1).
template <int NP, bool ENT>
__device__ __forceinline__ Acc rebase(Acc a, float Rn, float g) {
    if (a.R == -INFINITY) {            // empty so far (or only -inf): nothing to move
        a.R = Rn;
        return a;
    }
    const float d = a.R - Rn;          // <= 0
    const float f = ex2(d);
    if constexpr (ENT) a.y1 = f * fmaf(d, a.s1, a.y1);
    a.s1 *= f;
    if constexpr (NP != 1) {
#pragma unroll
        for (int k = 0; k < n_tau_sums<NP>(); ++k) a.st[k] *= tau_scale<NP>(d, g, k);
    }
    a.R = Rn;
    return a;
}

// Load one lane's VPL vectors of a stage; vectors past the chunk read as -inf
// (or, with FLOOR, as the large negative finite floor).
template <int DT, int VPL, bool FLOOR = false>
__device__ __forceinline__ void load_vecs(const uint4 *v4, int nvec, int lane,
                                          uint4 (&q)[VPL]) {
    if (nvec == VPL * 32) {                    // a full chunk: no predication
#pragma unroll
        for (int i = 0; i < VPL; ++i) q[i] = v4[lane + 32 * i];
        return;
    }
    const uint32_t ni = FLOOR ? Elem<DT>::kFloorWord : Elem<DT>::kNegInfWord;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int idx = lane + 32 * i;
        q[i] = idx < nvec ? v4[idx] : make_uint4(ni, ni, ni, ni);
    }
}

// Adds a chunk's sums to the running ones.
template <int NP, bool ENT>
__device__ __forceinline__ void add_chunk(Acc &a, float c1, const float (&ct)[3], float cy) {
    a.s1 += c1;
    if constexpr (NP != 1) {
#pragma unroll
        for (int k = 0; k < n_tau_sums<NP>(); ++k) a.st[k] += ct[k];
    }
    if constexpr (ENT) a.y1 += cy;
}

// The largest of a chunk's sums (the one that overflows first).
template <int NP>
__device__ __forceinline__ float chunk_peak(float c1, const float (&ct)[3]) {
    return fmaxf(c1, ct[n_tau_sums<NP>() - 1]);
}

// Merge part b into a (each relative to its own reference).
template <int NP, bool ENT>
__device__ __forceinline__ Acc merge_part(Acc a, Acc b, float g) {
    const float M = fmaxf(a.R, b.R);
    if (M == -INFINITY) {              // both parts saw only -inf logits
        a.s1 += b.s1;                  // keeps a NaN poison, else 0
        a.st[0] += b.st[0];
        a.st[1] += b.st[1];
        a.st[2] += b.st[2];
        a.y1 += b.y1;
        return a;
    }
    a = rebase<NP, ENT>(a, M, g);
    b = rebase<NP, ENT>(b, M, g);
    const float z[3] = {b.st[0], b.st[1], b.st[2]};
    add_chunk<NP, ENT>(a, b.s1, z, b.y1);
    return a;
}

template <int NP, bool ENT>
__device__ __forceinline__ Acc warp_merge(Acc a, float g) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        Acc b;
        b.R = __shfl_xor_sync(0xffffffffu, a.R, off);
        b.s1 = __shfl_xor_sync(0xffffffffu, a.s1, off);
#pragma unroll
        for (int k = 0; k < 3; ++k)
            b.st[k] = (NP != 1 && k < n_tau_sums<NP>())
                          ? __shfl_xor_sync(0xffffffffu, a.st[k], off) : 0.f;
        b.y1 = ENT ? __shfl_xor_sync(0xffffffffu, a.y1, off) : 0.f;
        a = merge_part<NP, ENT>(a, b, g);
    }
    return a;
}

// -ln(1 + 2^a) in float64 (the value is computed in float, except for the tiny
// tail, whose magnitude is below float's range).
__device__ __forceinline__ double neg_log1p_exp2(float a) {
    if (a > 24.f) return -(double)(a * kLn2f + log1pf(exp2f(-a)));
    if (a > -120.f) return -(double)log1pf(exp2f(a));
    return -exp2((double)a);
}

// Entropy in nats from S1, Y1 (the sums without the token) and the token's
// exponent t, all relative to the same reference (the general form, for
// shifts outside the range the fast form handles).
__device__ double entropy_nats_wide(double s1, double y1, double t) {
    const bool tok = t != -INFINITY;
    const double m = fmax(tok ? t : -INFINITY, log2(s1));
    const double et = tok ? exp2(t - m) : 0.0;
    const double zs = s1 * exp2(-m) + et;
    const double ms = y1 * exp2(-m) + (tok ? t * et : 0.0);
    return 0.6931471805599453 * (m + log2(zs) - ms / zs);
}

// The same with an integer shift m >= every exponent (m = ceil(max(t,
// log2 S1))): Z = S1 2^-m + 2^(t-m) lies in (1/2, 2] and
//     D = sum_j 2^(y_j - m) (m - y_j) = m Z - (Y1 2^-m + t 2^(t-m)) >= 0,
//     H = ln 2 (log2 Z + D / Z).
// D is formed in float64, since it is a difference of nearly equal terms when
// one logit holds most of the mass; log2 Z and D / Z carry only float relative
// error, so they are taken in float.  Few float64 operations: GB300's FP64
// pipe is narrow, and this runs once per row.
__device__ double entropy_nats(float s1, float y1, float t) {
    const bool tok = t != -INFINITY;
    // no other finite logit: the token holds all the mass (its exponent is +inf
    // then, since the reference never left -inf)
    if (!(s1 > 0.f)) return tok ? 0.0 : __longlong_as_double(0x7ff8000000000000ll);
    const float m = ceilf(fmaxf(tok ? t : -INFINITY, log2f(s1)));
    if (!(fabsf(m) < 1000.f))
        return entropy_nats_wide((double)s1, (double)y1, tok ? (double)t : -INFINITY);
    const double sc = __longlong_as_double((long long)(1023 - (int)m) << 52);   // 2^-m
    const double et = tok ? (double)exp2f(t - m) : 0.0;
    const double zs = fma((double)s1, sc, et);
    const double ms = fma((double)y1, sc, tok ? (double)t * et : 0.0);
    const double d = fma((double)m, zs, -ms);
    const float zf = (float)zs;
    return 0.6931471805599453 * ((double)log2f(zf) + (double)((float)d / zf));
}

template <int NP, bool ENT>
__device__ void finalize_row(const RowsParams &p, int64_t r, Acc a, float lt, bool bad) {
    double o0, oq = 0.0, h = 0.0;
    const double qnan = __longlong_as_double(0x7ff8000000000000ll);
    if constexpr (NP == 1) a.st[0] = a.s1;
    bool nonfinite = false;
    if (bad || __float_as_uint(lt) == kAbsent) {
        o0 = oq = h = qnan;
        nonfinite = true;          // already flagged (token or row index)
        if constexpr (multi_tau<NP>())
            for (int k = 0; k < p.n_taus; ++k) p.lq_multi[(int64_t)k * p.n_rows + r] = qnan;
    } else {
        const float t = fmaf(lt, kLog2e, -a.R);
        nonfinite = (lt != lt) || (lt == INFINITY) || (a.R != a.R) || (a.s1 != a.s1) ||
                    (a.st[0] != a.st[0]) || (a.st[n_tau_sums<NP>() - 1] !=
                                             a.st[n_tau_sums<NP>() - 1]) ||
                    (a.R == INFINITY) || (t != t) || (ENT && (a.y1 != a.y1));
        if (nonfinite) {
            set_status(p.status, PS_DEV_NONFINITE);
            o0 = oq = h = qnan;
            if constexpr (multi_tau<NP>())
                for (int k = 0; k < p.n_taus; ++k) p.lq_multi[(int64_t)k * p.n_rows + r] = qnan;
        } else {
            o0 = neg_log1p_exp2(a.s1 > 0.f ? log2f(a.s1) - t : -INFINITY);
            if constexpr (NP == 1) {
                oq = o0;
            } else if constexpr (multi_tau<NP>()) {
                for (int k = 0; k < p.n_taus; ++k) {
                    const int pw = p.tau_pow[k];           // 1/tau: 1, 2, 4 or 8
                    const float sk = pw == 1 ? a.s1 : (pw == 2 ? a.st[0] : (pw == 4 ? a.st[1] : a.st[2]));
                    p.lq_multi[(int64_t)k * p.n_rows + r] =
                        neg_log1p_exp2(sk > 0.f ? log2f(sk) - t * (float)pw : -INFINITY);
                }
            } else {
                const float gt = (NP == 0) ? t * p.g : t * (float)NP;
                oq = neg_log1p_exp2(a.st[0] > 0.f ? log2f(a.st[0]) - gt : -INFINITY);
            }
            if constexpr (ENT) {
                // a token logit of -inf has no mass: t = -inf leaves it out
                h = entropy_nats(a.s1, a.y1, lt == -INFINITY ? -INFINITY : t);
            }
        }
    }
    p.lp0[r] = o0;
    if constexpr (!multi_tau<NP>()) p.lq[r] = oq;
    if constexpr (ENT) p.entropy[r] = h;
}

}  // namespace
}  // namespace ps
