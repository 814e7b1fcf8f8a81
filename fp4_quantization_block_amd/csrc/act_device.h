// act_device.h -- device helpers shared by the activation operators (norm.hip,
// glu.hip): elements loaded and stored in chunks of eight per lane, MX row
// blocks encoded and decoded by the four lanes that hold them, wave and
// workgroup sums in a fixed order, and the gate functions with their slopes.
//
// Chunks.  A lane takes eight consecutive elements at a time, 16 bytes of bf16
// or 32 of fp32; rows may start at any element, since the loads and stores are
// declared with the element's alignment and gfx950 takes 16-byte accesses at
// any of them.  Rows whose length is no multiple of eight end in a chunk that
// overlaps the one before; the few cases that cannot have an element twice
// (an output over an input, rows under eight) take elements one by one.
#pragma once
#include "mx_device.h"

namespace mx {

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

template <int SRC> struct ElemT;
template <> struct ElemT<SRC_BF16> { typedef uint16_t raw; static constexpr int bytes = 2; };
template <> struct ElemT<SRC_F32> { typedef float raw; static constexpr int bytes = 4; };

// two fp32 values rounded to nearest even, as a bf16 pair
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){a, b}, bf16x2_t));
}

// N (eight, or four) consecutive elements as raw dwords
template <int SRC, int N = 8> struct Chunk { uint32_t w[N * ElemT<SRC>::bytes / 4]; };

template <int SRC, int N = 8>
__device__ __forceinline__ Chunk<SRC, N> load_chunk(const void* base, int64_t elem)
{
    Chunk<SRC, N> c;
    const typename ElemT<SRC>::raw* p = (const typename ElemT<SRC>::raw*)base + elem;
    __builtin_memcpy(&c, p, sizeof c);       // 16-byte accesses with the element's alignment
    return c;
}

template <int SRC, int N>
__device__ __forceinline__ float chunk_value(const Chunk<SRC, N>& c, int i)
{
    if constexpr (SRC == SRC_BF16) return (i & 1) ? bf16_hi(c.w[i >> 1]) : bf16_lo(c.w[i >> 1]);
    else return __uint_as_float(c.w[i]);
}

template <int SRC>
__device__ __forceinline__ Chunk<SRC> make_chunk(const float (&v)[8])
{
    Chunk<SRC> c;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        if constexpr (SRC == SRC_F32) c.w[i] = __float_as_uint(v[i]);
        else if ((i & 1) == 0) c.w[i >> 1] = pack_bf16(v[i], v[i + 1]);
    }
    return c;
}

template <int SRC>
__device__ __forceinline__ void store_chunk(void* base, int64_t elem, const Chunk<SRC>& c)
{
    __builtin_memcpy((typename ElemT<SRC>::raw*)base + elem, &c, sizeof c);
}

// one element
template <int SRC>
__device__ __forceinline__ float load_elem(const void* base, int64_t elem)
{
    if constexpr (SRC == SRC_BF16) return __uint_as_float((uint32_t)((const uint16_t*)base)[elem] << 16);
    else return ((const float*)base)[elem];
}

template <int SRC>
__device__ __forceinline__ void store_elem(void* base, int64_t elem, float v)
{
    if constexpr (SRC == SRC_BF16) ((uint16_t*)base)[elem] = (uint16_t)pack_bf16(v, v);
    else ((float*)base)[elem] = v;
}

// a value rounded to the element type
template <int SRC>
__device__ __forceinline__ float rounded(float v)
{
    if constexpr (SRC == SRC_BF16) return bf16_lo(pack_bf16(v, v));
    else return v;
}

// ---------------------------------------------------------------------
// Sums.  The order is fixed by the lane and wave numbers, so a result does
// not change from run to run.  All lanes of the T take part.
// ---------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

enum : int { DPP_XOR1 = 0xB1, DPP_XOR2 = 0x4E, DPP_HALF_MIRROR = 0x141, DPP_MIRROR = 0x140,
             DPP_BCAST15 = 0x142, DPP_BCAST31 = 0x143 };

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) { return v + __uint_as_float(dpp<CTRL>(__float_as_uint(v))); }

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add_rows(float v)
{
    return v + __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, ROWS, 0xF, false));
}

__device__ __forceinline__ float wave_sum(float v)
{
    v = dpp_add<DPP_XOR1>(v);
    v = dpp_add<DPP_XOR2>(v);
    v = dpp_add<DPP_HALF_MIRROR>(v);
    v = dpp_add<DPP_MIRROR>(v);
    v = dpp_add_rows<DPP_BCAST15, 0xA>(v);     // rows 1 and 3 of 16 lanes take rows 0 and 2
    v = dpp_add_rows<DPP_BCAST31, 0xC>(v);     // rows 2 and 3 take lane 31: lane 63 has all
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// the sum over T neighbouring lanes, 8 to 64 of them, in each of them
template <int T>
__device__ __forceinline__ float lanes_sum(float v)
{
    static_assert(T == 8 || T == 16 || T == 32 || T >= 64, "lanes of a row");
    if constexpr (T >= 64) {
        return wave_sum(v);
    } else {
        v = dpp_add<DPP_XOR1>(v);
        v = dpp_add<DPP_XOR2>(v);
        v = dpp_add<DPP_HALF_MIRROR>(v);
        if constexpr (T >= 16) v = dpp_add<DPP_MIRROR>(v);
        if constexpr (T == 32) {
            auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
            v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
        }
        return v;
    }
}

// the sum over T lanes (part of a wave, a wave, or a workgroup of T / 64 waves
// through `red`, T / 64 floats of LDS that no other sum uses before the next
// barrier)
template <int T>
__device__ __forceinline__ float group_sum(float v, float* red)
{
    v = lanes_sum<T>(v);
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int i = 1; i < T / 64; i++) v += red[i];
    }
    return v;
}

// ---------------------------------------------------------------------
// MX row blocks of 32, eight elements in each of four consecutive lanes
// ---------------------------------------------------------------------
// |max| key of three values: their largest magnitude's bits, a NaN's where one
// is NaN (v_maximum3_f32, the maximum of IEEE 754-2019)
__device__ __forceinline__ float abs_max3(float a, float b, float c)
{
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(__builtin_fabsf(a), __builtin_fabsf(b)), __builtin_fabsf(c));
}

template <int N>
__device__ __forceinline__ uint32_t chunk_key(const float (&v)[N])
{
    static_assert(N % 2 == 0, "pairs");
    float k = __builtin_elementwise_maximum(__builtin_fabsf(v[0]), __builtin_fabsf(v[1]));
#pragma unroll
    for (int i = 2; i < N; i += 2) k = abs_max3(k, v[i], v[i + 1]);
    return __float_as_uint(k);
}

__device__ __forceinline__ uint32_t quad_max(uint32_t k)
{
    k = max(k, dpp<DPP_XOR1>(k));
    return max(k, dpp<DPP_XOR2>(k));
}

// Shared exponent of a block from its |max| key, in the forms the converters
// take: the E8M0 byte max(exponent field - emax, 0) (the exponent rule with
// its clamp at -127, which takes zero and subnormal maxima too), 2^e as an
// fp32 whose exponent field is that byte, and Fmax 2^e.
template <int FMT>
struct BlockScale {
    uint32_t byte;
    float scale, top;
    __device__ __forceinline__ explicit BlockScale(uint32_t key)
    {
        constexpr uint32_t TOP = FMT == E4M3 ? (8u << 23) | 0x600000u : (15u << 23) | 0x600000u;   // Fmax = 1.75 2^emax
        byte = __builtin_elementwise_sub_sat(key >> 23, (uint32_t)Fmt<FMT>::emax);
        scale = __uint_as_float(byte << 23);
        top = __uint_as_float((byte << 23) + TOP);
    }
    __device__ __forceinline__ float clamped(float v) const { return __builtin_amdgcn_fmed3f(v, -top, top); }
};

// Four codes of a finite block.  The scaled converters return RNE(x / 2^e),
// the scale's exponent field read as E8M0, and do not saturate: the values are
// clamped to +-Fmax 2^e first, or the kernel has asked the converters to
// (SATURATED: saturate_converters).  (Both were found equal to scaling,
// clamping and converting for every block exponent over 28 binades below it,
// at 1.5 and 0.5 instructions an element instead of 2.5.)
template <int FMT, bool SATURATED = false>
__device__ __forceinline__ uint32_t encode4(const BlockScale<FMT>& b, float v0, float v1, float v2, float v3)
{
    short2v d = {0, 0};
    if constexpr (!SATURATED) v0 = b.clamped(v0), v1 = b.clamped(v1), v2 = b.clamped(v2), v3 = b.clamped(v3);
    if constexpr (FMT == E4M3) {
        d = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(d, v0, v1, b.scale, false);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(d, v2, v3, b.scale, true);
    } else {
        d = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(d, v0, v1, b.scale, false);
        d = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(d, v2, v3, b.scale, true);
    }
    return __builtin_bit_cast(uint32_t, d);
}

// Sets the wave's MODE.FP16_OVFL, with which conversions to FP8 saturate.
// (It clamps fp16 results too: for kernels that have none.)
__device__ __forceinline__ void saturate_converters()
{
    __builtin_amdgcn_s_setreg(1 | 23 << 6, 1);     // register 1 (MODE), bit 23, one bit
}

constexpr uint32_t NONFINITE = 0x7F800000u;      // keys from here on: a block with a NaN or an Inf

struct Codes8 { uint32_t lo, hi, scale; };

// eight values of a block whose |max| key is `key`: codes and scale byte as
// mx_quantize writes them (round to nearest even, saturating; a block with a
// NaN or an Inf: 0x7F everywhere and byte 0xFF)
template <int FMT>
__device__ __forceinline__ Codes8 encode8(const float (&v)[8], uint32_t key)
{
    const BlockScale<FMT> b(key);
    Codes8 c{encode4<FMT>(b, v[0], v[1], v[2], v[3]), encode4<FMT>(b, v[4], v[5], v[6], v[7]), b.byte};
    if (key >= NONFINITE) c = Codes8{0x7F7F7F7Fu, 0x7F7F7F7Fu, 0xFFu};
    return c;
}

__device__ __forceinline__ Codes8 encode8(int fmt, const float (&v)[8], uint32_t key)
{
    return fmt == E4M3 ? encode8<E4M3>(v, key) : encode8<E5M2>(v, key);
}

// the four lanes' part of one block of a row copy: codes of elements elem ..
// elem + 7 (row-major, dense) and the block's scale byte.  `valid` is the
// same for the four lanes.
__device__ __forceinline__ void encode_row_chunk(int fmt, const float (&v)[8], bool valid, int64_t elem, uint8_t* q,
                                                 uint8_t* s)
{
    const Codes8 c = encode8(fmt, v, quad_max(chunk_key(v)));
    if (valid) {
        *(uint2*)(q + elem) = make_uint2(c.lo, c.hi);
        if ((threadIdx.x & 3) == 0) s[elem >> 5] = (uint8_t)c.scale;
    }
}

// Checkpointed values: two codes (the low or high half of c) times 2^(byte -
// 127) by one converter, which reads the scale's exponent field as E8M0, byte
// 0 as 2^-127 and byte 255 as NaN, as mx_dequantize does (equal to it for
// every code and byte).
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t c, uint32_t byte, float* v)
{
    const float s = __uint_as_float(byte << 23);
    f32x2_t a, b;
    if constexpr (FMT == E4M3) {
        a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, s, false);
        b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, s, true);
    } else {
        a = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(c, s, false);
        b = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(c, s, true);
    }
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}

template <int FMT>
__device__ __forceinline__ void decode8(uint2 c, uint32_t byte, float (&v)[8])
{
    decode4<FMT>(c.x, byte, v);
    decode4<FMT>(c.y, byte, v + 4);
}

// Where a backward kernel reads an input: from its tensor, or from a
// checkpoint of one of the formats
enum : int { FROM_TENSOR = -1, FROM_E4M3 = E4M3, FROM_E5M2 = E5M2 };

// ---------------------------------------------------------------------
// Gate functions a = act(x) and their slopes d = act'(x).
//   SILU       a = x s,  s = 1 / (1 + e^-x);  d = s + a (1 - s)
//   GELU       a = x P(x), P the normal distribution function;
//              d = P(x) + x e^(-x^2/2) / sqrt(2 pi)
//   GELU_TANH  x/2 (1 + tanh z) with z = sqrt(2/pi) (x + 0.044715 x^3).
//              (1 + tanh z) / 2 = 1 / (1 + e^-2z) = s, so a = x s and
//              d = s + a (1 - s) z2',  z2' = 2 dz/dx,  1 - s = e^-2z s
// Exponentials are the hardware's base-2 one, divisions its reciprocal, each
// within 1 ulp.  What the exponent's roundings add, relative to the result, for
// an exponent z: |z| 2^-24 for each rounding, of which SILU's product with
// log2 e is one (the rounded constant less than a third of that), GELU's square
// two and GELU_TANH's polynomial three.  e^-x overflows to Inf for x < -88 and
// s becomes 0.
// ---------------------------------------------------------------------
enum : int { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2 };

// The upper tail of the normal distribution at |x|, P(-|x|), from e =
// e^(-x^2/2): e t Q(t) with t = 1 / (1 + 0.37 |x|).  e^(x^2/2) P(-|x|) / t is
// smooth in t on (0, 1] (0.37 / sqrt(2 pi) at t = 0), and Q is its polynomial
// of degree 10, fitted to scipy's erfcx with weights moved to the largest
// relative errors (Lawson's method).  The coefficients as stored are within
// 4.1e-8 of it.  The whole, evaluated in fp32 with correctly rounded
// reciprocals and exponentials, is off by at most 7 units of 2^-24 for |x| < 2,
// 11 below 3 and 33 below 6, where nearly all of it is the exponent's
// roundings; they grow with x^2.  One exponential serves this and the
// density in the slope.  (The forward at 4096 x 14336 bf16: 62 us, bound by
// memory; with the math library's erfcf 92 us, bound by its instructions.)
__device__ __forceinline__ float normal_tail(float x, float e)
{
    constexpr float Q[11] = {0x1.2e4d70p-3f, 0x1.2e4dcap-3f, 0x1.04dffep-3f, 0x1.652b6ep-4f, 0x1.1705bep-5f, -0x1.143360p-6f,
                             -0x1.53f29cp-11f, -0x1.2f7a94p-3f, 0x1.bde68ap-3f, -0x1.ee0992p-4f, 0x1.9506a0p-6f};
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.37f, __builtin_fabsf(x), 1.0f));
    float q = Q[10];
#pragma unroll
    for (int k = 9; k >= 0; k--) q = __builtin_fmaf(q, t, Q[k]);
    return q * t * e;
}

template <int ACT, bool SLOPE>
__device__ __forceinline__ void gate(float x, float& a, float& d)
{
    constexpr float LOG2E = 1.44269504f;
    if constexpr (ACT == ACT_SILU) {
        const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-LOG2E * x));
        a = x * s;
        if constexpr (SLOPE) d = __builtin_fmaf(a, 1.0f - s, s);
    } else if constexpr (ACT == ACT_GELU) {
        const float e = __builtin_amdgcn_exp2f((-0.5f * LOG2E) * x * x);
        const float q = normal_tail(x, e), p = x < 0.0f ? q : 1.0f - q;
        a = x * p;
        if constexpr (SLOPE) d = __builtin_fmaf(0.39894228f * x, e, p);
    } else {
        // x^2 is held below 2^40, where s is 0 or 1 for long: no overflow to
        // Inf, which the vanishing 1 - s would turn into NaN.  1 - s is taken
        // as e s: the rounded difference would be off by 2^-24 absolutely,
        // which a z2' multiplies (the slope off by 33 units of 2^-24 at x = 5,
        // by 4 at most so).  Where e is Inf, s and a are 0: any finite e does.
        constexpr float Z = 1.59576912f, C = 0.044715f;            // 2 sqrt(2/pi)
        const float x2 = fminf(x * x, 0x1p40f);
        const float e = __builtin_amdgcn_exp2f(x * __builtin_fmaf(-LOG2E * Z * C, x2, -LOG2E * Z));
        const float s = __builtin_amdgcn_rcpf(1.0f + e);
        a = x * s;
        if constexpr (SLOPE) d = __builtin_fmaf(a * (fminf(e, 0x1p127f) * s), __builtin_fmaf(3.0f * Z * C, x2, Z), s);
    }
}

}  // namespace mx
