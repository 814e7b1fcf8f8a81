// optstate_device.h -- the FP8 optimizer-state format on the device: log2, exp2
// and powers as fixed sequences of fp32 operations, and the codes of a group
// encoded and decoded by the lanes that hold it.  optstate.hip converts whole
// states with it; adamw.hip decodes, steps and encodes them in one pass, to
// the same bits.  The format itself is described in optstate.hip.
#pragma once
#include <type_traits>

#include "mx_device.h"

namespace mx {

// log2 of the format's dynamic range Fmax / smallest subnormal, rounded to
// fp32: E4M3 448 / 2^-9 = 2^17.807..., E5M2 57344 / 2^-16 = 2^31.807...
template <int FMT> struct Range;
template <> struct Range<E4M3> { static constexpr float log2r = 17.8073549f; };
template <> struct Range<E5M2> { static constexpr float log2r = 31.8073549f; };

// log2 from the bits of a normal x > 0 (or +Inf), less `sub`: x = m * 2^e
// with m in (sqrt(1/2), sqrt(2)), z = m - 1 (exact), log2 x = e + z * P(z),
// P of degree 8 (a least-squares fit of log2(1+z)/z on that range,
// coefficients rounded to fp32), every step one fused multiply-add, in the
// order written.  Subtracting the bits of the smallest fp32 above sqrt(1/2)
// borrows from the exponent field exactly when the mantissa is at most
// sqrt(2), so the arithmetic shift gives e and the low 23 bits, added back,
// give m.
__device__ __forceinline__ float log2_bits(uint32_t bits, int sub)
{
#pragma clang fp contract(off)
    const uint32_t d = bits - 0x3F3504F4u;
    const int ex = ((int32_t)d >> 23) - sub;
    const float z = __uint_as_float((d & 0x007FFFFFu) + 0x3F3504F4u) - 1.0f;   // exact
    float p = 0x1.025a88p-3f;
    p = __builtin_fmaf(p, z, -0x1.a8cd06p-3f);
    p = __builtin_fmaf(p, z, 0x1.b9b144p-3f);
    p = __builtin_fmaf(p, z, -0x1.e94efep-3f);
    p = __builtin_fmaf(p, z, 0x1.26d40cp-2f);
    p = __builtin_fmaf(p, z, -0x1.715c9cp-2f);
    p = __builtin_fmaf(p, z, 0x1.ec73d4p-2f);
    p = __builtin_fmaf(p, z, -0x1.71547p-1f);
    p = __builtin_fmaf(p, z, 0x1.715476p+0f);
    return __builtin_fmaf(z, p, (float)ex);
}

// log2 of x >= 2^-126 (or +Inf)
__device__ __forceinline__ float log2_normal(float x) { return log2_bits(__float_as_uint(x), 0); }

// log2 of x > 0 (finite or +Inf): a subnormal x is first scaled into the
// normal range (exact)
__device__ __forceinline__ float log2_fixed(float x)
{
#pragma clang fp contract(off)
    const bool sub = x < 0x1p-126f;
    return log2_bits(__float_as_uint(sub ? x * 0x1p32f : x), sub ? 32 : 0);
}

// 2^y for y in [-151, 128]: n = floor(y + 1/2), z = y - n (exact, |z| <=
// 1/2), 2^z from a degree-6 fit on [-1/2, 1/2] whose constant term is
// exactly 1, then 2^n
__device__ __forceinline__ float exp2_core(float y)
{
#pragma clang fp contract(off)
    const float n = floorf(y + 0.5f);
    const float z = y - n;
    float s = 0x1.41a7p-13f;
    s = __builtin_fmaf(s, z, 0x1.5f44f4p-10f);
    s = __builtin_fmaf(s, z, 0x1.3b2dfep-7f);
    s = __builtin_fmaf(s, z, 0x1.c6aed6p-5f);
    s = __builtin_fmaf(s, z, 0x1.ebfbdap-3f);
    s = __builtin_fmaf(s, z, 0x1.62e43p-1f);
    s = __builtin_fmaf(s, z, 1.0f);
    return ldexpf(s, (int)n);
}

// 2^y for y <= 0, not NaN: 0 below -150
__device__ __forceinline__ float exp2_nonpos(float y)
{
    const float r = exp2_core(fmaxf(y, -151.0f));
    return y < -150.0f ? 0.0f : r;
}

// 2^y for any y: NaN for NaN, +Inf from 128 up, 0 below -150
__device__ __forceinline__ float exp2_fixed(float y)
{
    const float r = exp2_core(fminf(fmaxf(y, -151.0f), 128.0f));
    const float o = y < -150.0f ? 0.0f : y >= 128.0f ? __builtin_inff() : r;
    return y != y ? y : o;
}

// u^k for u >= 0
__device__ __forceinline__ float pow_fixed(float u, float k)
{
#pragma clang fp contract(off)
    const float p = exp2_fixed(k * log2_fixed(u));
    return u == 0.0f ? 0.0f : p;
}

// exact fp32 value of an FP8 code
template <int FMT>
__device__ __forceinline__ float decode8(uint32_t c)
{
    constexpr int MB = Fmt<FMT>::mbits, EB = 7 - MB, BIAS = FMT == E4M3 ? 7 : 15;
    const uint32_t e = (c >> MB) & ((1u << EB) - 1u), m = c & ((1u << MB) - 1u);
    float v;
    if (FMT == E4M3 && e == 15 && m == 7) v = __builtin_nanf("");
    else if (FMT == E5M2 && e == 31) v = m ? __builtin_nanf("") : __builtin_inff();
    else if (e == 0) v = (float)m * exp2i(1 - BIAS - MB);
    else v = (float)((1u << MB) | m) * exp2i((int)e - BIAS - MB);
    return (c & 0x80u) ? -v : v;
}

// NaN codes: E4M3 0x7F; E5M2 0x7D-0x7F (0x7C is Inf)
template <int FMT>
__device__ __forceinline__ bool is_nan8(uint32_t c7) { return FMT == E4M3 ? c7 == 0x7Fu : c7 > 0x7Cu; }

// log2(|decode(c)| / Fmax) for the 128 magnitudes, in the same fixed
// sequence the per-element form evaluates; -Inf for code 0 (so that its
// power is 0 whenever the exponent 1/k is positive) and 0 for the NaN
// codes, whose output is NaN whatever the power.  Filled by a workgroup of
// 256 threads, which then meets a barrier before it reads.
template <int FMT>
__device__ __forceinline__ void fill_log_table(float (&lg)[128])
{
#pragma clang fp contract(off)
    for (int c = threadIdx.x; c < 128; c += 256)
        lg[c] = c == 0 ? -__builtin_inff()
                       : is_nan8<FMT>((uint32_t)c) ? 0.0f : log2_fixed(fabsf(decode8<FMT>((uint32_t)c)) / Fmt<FMT>::fmax);
}

// whether a word of four codes holds one that is not a finite number
template <int FMT>
__device__ __forceinline__ bool any_nonfinite8(uint32_t w)
{
    constexpr uint32_t up = FMT == E4M3 ? 0x01010101u : 0x04040404u;   // 0x80 less the first such magnitude
    return (((w & 0x7F7F7F7Fu) + up) & 0x80808080u) != 0;
}

// E = 4 NV values of one group from their code words
template <int FMT, int E>
__device__ __forceinline__ void decode_state(const uint32_t (&c4)[E / 4], const float (&lg)[128], float amax, float k,
                                             float (&o)[E])
{
#pragma clang fp contract(off)
    const float kinv = 1.0f / k;
    const bool nan_group = amax != amax || k != k;
    // the table reads first, then arithmetic without branches
    float l[E];
#pragma unroll
    for (int e = 0; e < E; e++) l[e] = lg[(c4[e / 4] >> (8 * (e % 4))) & 0x7Fu];
    bool plain = kinv > 0.0f && kinv < __builtin_inff() && !nan_group;
#pragma unroll
    for (int i = 0; i < E / 4; i++) plain = plain && !any_nonfinite8<FMT>(c4[i]);
    if (plain) {
        // Every lg <= 0, so y <= 0 and not NaN.  The zero below y = -150 of the
        // general form needs no select: 2^y of y < -150 is at most 2^-150,
        // which rounds to zero (a tie, to even), as does 2^-151 for code 0.
#pragma unroll
        for (int e = 0; e < E; e++) {
            const float m = amax * exp2_core(fmaxf(kinv * l[e], -151.0f));
            const uint32_t sign = (c4[e / 4] << (24 - 8 * (e % 4))) & 0x80000000u;
            o[e] = __uint_as_float(__float_as_uint(m) ^ sign);
        }
    } else {
        // a NaN output comes from adding NaN (others add -0, which changes nothing)
#pragma unroll
        for (int e = 0; e < E; e++) {
            const uint32_t c = (c4[e / 4] >> (8 * (e % 4))) & 0xFFu, c7 = c & 0x7Fu;
            const float p = c7 == 0 ? 0.0f : exp2_fixed(kinv * l[e]);
            const float m = amax * p + (is_nan8<FMT>(c7) || nan_group ? __builtin_nanf("") : -0.0f);
            o[e] = (c & 0x80u) ? -m : m;
        }
    }
}

// Code words of E = 4 NV values of a group that T neighbouring lanes hold, and
// the group's largest magnitude and exponent (in every lane).  All lanes of the
// wave take part.  Zeros change neither extremum: lanes past the end of a
// group that is not full pass zeros.
template <int FMT, int T, int E>
__device__ __forceinline__ void encode_state(const float (&xs)[E], uint32_t (&codes)[E / 4], float& gamax, float& gk)
{
#pragma clang fp contract(off)
    static_assert(T >= 1 && T <= 64 && (T & (T - 1)) == 0, "a group's threads lie inside one wave");
    constexpr int NV = E / 4;
    float a[E];
    // group maximum and smallest nonzero magnitude as integer extrema of
    // |x|'s bits (their order is the values' for finite magnitudes; Inf
    // and NaN bits lie above every finite one, so they flag the group by
    // themselves).  The minimum runs over bits - 1, which sends zeros to
    // the top of the unsigned range.
    uint32_t kmax = 0, kmin = ~0u;
#pragma unroll
    for (int e = 0; e < E; e++) {
        const uint32_t b = __float_as_uint(xs[e]) & 0x7FFFFFFFu;
        a[e] = __uint_as_float(b);
        kmax = max(kmax, b);
        kmin = min(kmin, b - 1u);
    }
    // butterflies inside 32-lane halves by swizzle (xor mask in bits 14:10,
    // and mask 0x1F), across halves by a permute
    auto step = [&](auto OFFC) __attribute__((always_inline)) {
        constexpr int off = decltype(OFFC)::value;
        if constexpr (off < T && off < 32) {
            kmax = max(kmax, (uint32_t)__builtin_amdgcn_ds_swizzle((int)kmax, 0x1F | (off << 10)));
            kmin = min(kmin, (uint32_t)__builtin_amdgcn_ds_swizzle((int)kmin, 0x1F | (off << 10)));
        } else if constexpr (off < T) {
            kmax = max(kmax, (uint32_t)__shfl_xor((int)kmax, off));
            kmin = min(kmin, (uint32_t)__shfl_xor((int)kmin, off));
        }
    };
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 4>{});
    step(std::integral_constant<int, 8>{});
    step(std::integral_constant<int, 16>{});
    step(std::integral_constant<int, 32>{});
    const float amin = __uint_as_float(kmin + 1u);  // used only when some |x| > 0
    const bool bad = kmax >= 0x7F800000u;
    const float amax = __uint_as_float(kmax);
    if (bad) {                                   // a NaN or Inf: the NaN code everywhere
#pragma unroll
        for (int i = 0; i < NV; i++) codes[i] = 0x7F7F7F7Fu;
        gamax = __builtin_nanf(""); gk = __builtin_nanf("");
    } else if (amax == 0.0f) {                   // all zero: signed zeros, unit parameters
#pragma unroll
        for (int i = 0; i < NV; i++)
            codes[i] = (__float_as_uint(xs[4 * i]) >> 31) << 7 | (__float_as_uint(xs[4 * i + 1]) >> 31) << 15 |
                       (__float_as_uint(xs[4 * i + 2]) >> 31) << 23 | (__float_as_uint(xs[4 * i + 3]) >> 31) << 31;
        gamax = 1.0f; gk = 1.0f;
    } else {
        const float r = amax / amin;             // >= 1: normal or +Inf
        const float k = r > 1.0f ? Range<FMT>::log2r / log2_normal(r) : 1.0f;
        // k is finite and positive, and every quotient u = |x|/amax lies in
        // [0, 1], so y = k log2 u is finite and at most 0 for u > 0
        const TensorDiv d = make_div(amax);
        if (d.fast && ((kmin + 1u) << 1) - 1u >= d.lo_key) {
            // Every nonzero |x| of the group is at least amin, at or above the
            // division's threshold: the fast form gives the IEEE quotient
            // (+0 for x = 0, a normal number otherwise), and log2 needs no
            // subnormal step.
            auto quotient = [&](int e) __attribute__((always_inline)) {
                const float q0 = a[e] * d.r;
                return __builtin_fmaf(__builtin_fmaf(-q0, d.s, a[e]), d.r, q0);
            };
            // The fixed sequence.  Two steps of the general form are left out
            // because they cannot change a code: 2^y is at most 1 for y <= 0,
            // so |x|'s value stays within Fmax without the clamp; and below
            // y = -150, where the general form returns 0, the power is at most
            // 2^-149 and its product with Fmax far below the format's smallest
            // subnormal, so it rounds to a zero code (of x's sign) just as 0
            // does.
            auto fixed = [&](int e) __attribute__((always_inline)) {
#pragma clang fp contract(off)
                const float u = quotient(e);
                const float p = exp2_core(fmaxf(k * log2_normal(u), -151.0f));
                return __builtin_copysignf((u == 0.0f ? 0.0f : p) * Fmt<FMT>::fmax, xs[e]);
            };
            // Its codes without it, nearly always: the hardware's log2 and exp2
            // give the power within a known factor 1 +- EPS of the fixed
            // sequence's, and where both ends of that interval round to the
            // same code, rounding being monotone, so does what lies between.
            // Against the fixed sequences the hardware's log2 is off by at most
            // 4 units of 2^-24 of the result for arguments from 2^-125 to 1,
            // its exp2 by 2 from -40 to 0 (every argument compared).  Two more
            // units of y = k log2 u are its roundings, so y differs by 6 2^-24
            // |y| with |y| < 17.9 (E4M3) or 31.9 (E5M2), 2^y by ln 2 times that
            // plus 2 units, and the products with Fmax by 2: 79 units, 137.
            // (13 issue slots an element instead of 32; one word of four codes
            // in about 1400 has a value that near a border and takes the fixed
            // sequence.  117M elements: XX us.)
            constexpr float EPS = FMT == E4M3 ? 0x1p-17f : 0x1p-16f;       // 128 and 256 units
#pragma unroll
            for (int i = 0; i < NV; i++) {
                float lo[4], hi[4];
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    const int e = 4 * i + c;
                    // (0 for u = 0: 2^-Inf)
                    const float p = __builtin_copysignf(__builtin_amdgcn_exp2f(k * __builtin_amdgcn_logf(quotient(e))), xs[e]);
                    lo[c] = p * (Fmt<FMT>::fmax * (1.0f - EPS));
                    hi[c] = p * (Fmt<FMT>::fmax * (1.0f + EPS));
                }
                codes[i] = cvt4_fp8<FMT>(lo[0], lo[1], lo[2], lo[3]);
                if (codes[i] != cvt4_fp8<FMT>(hi[0], hi[1], hi[2], hi[3]))
                    codes[i] = cvt4_fp8<FMT>(fixed(4 * i), fixed(4 * i + 1), fixed(4 * i + 2), fixed(4 * i + 3));
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; i++) {
                float y[4];
#pragma unroll
                for (int c = 0; c < 4; c++)
                    y[c] = clamp_fmax<FMT>(__builtin_copysignf(pow_fixed(a[4 * i + c] / amax, k) * Fmt<FMT>::fmax, xs[4 * i + c]));
                codes[i] = cvt4_fp8<FMT>(y[0], y[1], y[2], y[3]);
            }
        }
        gamax = amax; gk = k;
    }
}

}  // namespace mx
