// gemm_glu.hip -- the gate and up projections of a gated MLP block with their
// activation and product in one kernel, for few rows:
//   gate = a_g A Wg^T,  up = a_u A Wu^T,  h = act(gate) * up,
// A [M][K], Wg and Wu [F][K] as MX codes with their scales, as in gemm.hip.
// ([FAF, "格式感知融合的设计思路"]: the producer writes what its consumer reads,
// here h as the down projection's operand and the 8-bit checkpoints of gate
// and up, [COAT, "FP8啟用"].)
//
// Many rows run on k_gemm_w4 (gemm.hip).  k_glu_rows below takes few rows, and
// everything whose K or scale arrays that kernel does not take.  For few rows
// the time goes to reading the weights once.  The matrix instruction gets the
// weights as its first operand and up to 32 tokens as its second, so that one
// wave covers 32 rows of Wg and the same 32 of Wu: a lane then holds gate and
// up of the same elements, 16 of each of a token's 32, and the other 16 lie in
// the lane 32 further on.  A workgroup's waves split K and meet in LDS.
#include "act_device.h"
#include "mx_internal.h"

namespace mx {

namespace {

typedef int int8v __attribute__((ext_vector_type(8)));
typedef int int4v __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));

constexpr int WAVES = 8;            // of a workgroup, which split K
constexpr int UNIT = 128;           // bytes of K a row that a wave takes at a time
constexpr int ROWS = 32;            // rows of each weight, and tokens, of an MFMA tile
constexpr int PITCH = 33;           // of the joined sums: rows of 32 tokens, one float between

template <int FMT> struct MfmaFmt;
template <> struct MfmaFmt<E4M3> { static constexpr int code = 0; };
template <> struct MfmaFmt<E5M2> { static constexpr int code = 1; };
template <> struct MfmaFmt<E2M1> { static constexpr int code = 4; };

// One unit of an operand's tile in the lane layout of the 32x32x64 scaled
// MFMA (gemm.hip): lane l holds row l % 32; of a step's 64 elements, with h =
// l / 32, the 16-byte halves of blocks 0 and 1 that h names (FP8), or block h
// (FP4); the scale byte of block h.
template <bool FP4>
struct Fragment {
    static constexpr int STEPS = FP4 ? 4 : 2;        // MFMA steps of a unit
    int8v q[STEPS];
    uint32_t s[STEPS];
};

struct Row { const uint8_t* q; const uint8_t* s; };

__device__ __forceinline__ int8v put16(int8v v, int half, uint4 w)
{
    v[4 * half] = (int)w.x; v[4 * half + 1] = (int)w.y; v[4 * half + 2] = (int)w.z; v[4 * half + 3] = (int)w.w;
    return v;
}

// unit u of a row: `whole` where all of it lies inside the row, otherwise what
// lies past the end is zero (with the scale 1)
template <bool FP4>
__device__ __forceinline__ void load_unit(Fragment<FP4>& f, const Row& r, int64_t u, int h, bool whole, int64_t kbytes)
{
    constexpr int STEP = FP4 ? 32 : 64, BLOCK = STEP / 2;      // bytes of a step and of a block
#pragma unroll
    for (int s = 0; s < Fragment<FP4>::STEPS; s++) {
        const int64_t at = u * UNIT + s * STEP;
        int8v v = {0, 0, 0, 0, 0, 0, 0, 0};
        uint32_t scale = 127u;
        if constexpr (FP4) {
            if (whole || at + BLOCK * h < kbytes) v = put16(v, 0, *(const uint4*)(r.q + at + BLOCK * h));
        } else {
            if (whole || at < kbytes) v = put16(v, 0, *(const uint4*)(r.q + at + 16 * h));
            if (whole || at + BLOCK < kbytes) v = put16(v, 1, *(const uint4*)(r.q + at + BLOCK + 16 * h));
        }
        if (whole || at + BLOCK * h < kbytes) scale = r.s[at / BLOCK + h];
        f.q[s] = v;
        f.s[s] = scale;
    }
}

// keys of the largest magnitude over 16 neighbouring lanes
__device__ __forceinline__ uint32_t max16(uint32_t k)
{
    k = max(k, dpp<DPP_XOR1>(k));
    k = max(k, dpp<DPP_XOR2>(k));
    k = max(k, dpp<DPP_HALF_MIRROR>(k));
    return max(k, dpp<DPP_MIRROR>(k));
}

// two neighbouring values of one block of a row copy, 16 lanes to the block
__device__ __forceinline__ void emit_codes(int fmt, float a, float b, bool valid, int64_t elem, uint8_t* q, uint8_t* s)
{
    const float v[8] = {a, b, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    const Codes8 c = encode8(fmt, v, max16(chunk_key<2>({a, b})));
    if (valid) {
        *(uint16_t*)(q + elem) = (uint16_t)c.lo;
        if ((threadIdx.x & 15) == 0) s[elem >> 5] = (uint8_t)c.scale;
    }
}

__device__ __forceinline__ void emit_pair(bool f32, void* base, int64_t at, float a, float b, bool first, bool second)
{
    if (f32) {
        if (first) ((float*)base)[at] = a;
        if (second) ((float*)base)[at + 1] = b;
    } else {
        const uint32_t w = pack_bf16(a, b);
        if (first) ((uint16_t*)base)[at] = (uint16_t)w;
        if (second) ((uint16_t*)base)[at + 1] = (uint16_t)(w >> 16);
    }
}

__device__ __forceinline__ float gate_value(int act, float x)
{
    float a, d;
    if (act == ACT_SILU) gate<ACT_SILU, false>(x, a, d);
    else if (act == ACT_GELU) gate<ACT_GELU, false>(x, a, d);
    else gate<ACT_GELU_TANH, false>(x, a, d);
    return a;
}

// NT tiles of 32 tokens each
template <int FA, int FB, int NT>
__global__ __launch_bounds__(64 * WAVES) void k_glu_rows(const GemmGluJob g, int tiles_f, int tiles_m)
{
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr bool FP4 = FA == E2M1;
    constexpr int EPB = FP4 ? 2 : 1;
    __shared__ float red[WAVES][2 * ROWS * PITCH];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = lane >> 5, l32 = lane & 31;
    // the tiles of tokens of one set of weights run one after the other on one XCD
    const int wg = blockIdx.x, tf = wg / (8 * tiles_m) * 8 + wg % 8, tm = wg / 8 % tiles_m;
    if (tf >= tiles_f) return;
    const int64_t f0 = (int64_t)tf * ROWS, m0 = (int64_t)tm * (ROWS * NT);
    const int64_t kbytes = g.K / EPB, kblocks = g.K / 32;
    const int64_t units = (kbytes + UNIT - 1) / UNIT;

    // rows past the end read the last one, and their results are dropped
    const int64_t wrow = min(f0 + l32, g.F - 1);
    const Row rg{g.qg + wrow * kbytes, g.sg + wrow * kblocks}, ru{g.qu + wrow * kbytes, g.su + wrow * kblocks};
    Row rt[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) {
        const int64_t row = min(m0 + 32 * t + l32, g.M - 1);
        rt[t] = Row{g.qa + row * kbytes, g.sa + row * kblocks};
    }

    f16v acc[2][NT];
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int r = 0; r < 16; r++) acc[i][t][r] = 0.0f;

    struct Stage { Fragment<FP4> g, u, t[NT]; };
    auto load = [&](Stage& s, int64_t u) __attribute__((always_inline)) {
        const bool whole = (u + 1) * UNIT <= kbytes;
        load_unit<FP4>(s.g, rg, u, h, whole, kbytes);
        load_unit<FP4>(s.u, ru, u, h, whole, kbytes);
#pragma unroll
        for (int t = 0; t < NT; t++) load_unit<FP4>(s.t[t], rt[t], u, h, whole, kbytes);
    };
    auto multiply = [&](const Stage& s) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < Fragment<FP4>::STEPS; k++)
#pragma unroll
            for (int t = 0; t < NT; t++) {
                acc[0][t] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(s.g.q[k], s.t[t].q[k], acc[0][t], MfmaFmt<FB>::code,
                                                                            MfmaFmt<FA>::code, 0, (int)s.g.s[k], 0, (int)s.t[t].s[k]);
                acc[1][t] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(s.u.q[k], s.t[t].q[k], acc[1][t], MfmaFmt<FB>::code,
                                                                            MfmaFmt<FA>::code, 0, (int)s.u.s[k], 0, (int)s.t[t].s[k]);
            }
    };
    Stage a, b;
    int64_t u = wave;
    if (u < units) load(a, u);
    for (; u < units; u += 2 * WAVES) {
        if (u + WAVES < units) load(b, u + WAVES);
        multiply(a);
        if (u + 2 * WAVES < units) load(a, u + 2 * WAVES);
        if (u + WAVES < units) multiply(b);
    }

    float common = g.alpha;
    if (g.ta) common = common * *g.ta;
    float ag = common, au = common;
    if (g.tg) ag = ag * *g.tg;
    if (g.tu) au = au * *g.tu;
    if (g.hadamard_k) ag = ag * 0.03125f, au = au * 0.03125f;

    // thread t of the join: token t / 16 of the tile, elements 2 (t % 16) and the next
    const int token = threadIdx.x >> 4, pair = 2 * (threadIdx.x & 15);
#pragma unroll
    for (int t = 0; t < NT; t++) {
        if (t > 0) __syncthreads();
#pragma unroll
        for (int r = 0; r < 16; r++) {
            const int row = 8 * (r / 4) + 4 * h + r % 4;
            red[wave][row * PITCH + l32] = acc[0][t][r];
            red[wave][(ROWS + row) * PITCH + l32] = acc[1][t][r];
        }
        __syncthreads();
        float gv[2] = {0.0f, 0.0f}, uv[2] = {0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < WAVES; w++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                gv[e] += red[w][(pair + e) * PITCH + token];
                uv[e] += red[w][(ROWS + pair + e) * PITCH + token];
            }
        float hv[2];
#pragma unroll
        for (int e = 0; e < 2; e++) {
            gv[e] *= ag;
            uv[e] *= au;
            hv[e] = gate_value(g.act, gv[e]) * uv[e];
        }
        const int64_t m = m0 + 32 * t + token, f = f0 + pair;
        const bool row = m < g.M, first = row && f < g.F, second = row && f + 1 < g.F;
        if (g.h) emit_pair(g.out_f32, g.h, m * g.ld_h + f, hv[0], hv[1], first, second);
        if (g.gate) {
            emit_pair(g.out_f32, g.gate, m * g.ld_gate + f, gv[0], gv[1], first, second);
            emit_pair(g.out_f32, g.up, m * g.ld_up + f, uv[0], uv[1], first, second);
        }
        // (F is then a multiple of 32: a block is there whole or not at all)
        if (g.qh) emit_codes(g.h_fmt, hv[0], hv[1], first, m * g.F + f, g.qh, g.sh);
        if (g.qgc) {
            emit_codes(g.ckpt_fmt, gv[0], gv[1], first, m * g.F + f, g.qgc, g.sgc);
            emit_codes(g.ckpt_fmt, uv[0], uv[1], first, m * g.F + f, g.quc, g.suc);
        }
    }
#endif
}

template <int FA, int FB>
hipError_t launch_rows(const GemmGluJob& j, hipStream_t s)
{
    const int tiles_f = (int)((j.F + ROWS - 1) / ROWS);
    const int nt = j.M <= ROWS ? 1 : 2;
    const int tiles_m = (int)((j.M + ROWS * nt - 1) / (ROWS * nt));
    const unsigned grid = (unsigned)((tiles_f + 7) / 8 * 8) * (unsigned)tiles_m;
    if (nt == 1) k_glu_rows<FA, FB, 1><<<grid, 64 * WAVES, 0, s>>>(j, tiles_f, tiles_m);
    else k_glu_rows<FA, FB, 2><<<grid, 64 * WAVES, 0, s>>>(j, tiles_f, tiles_m);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_glu(const GemmGluJob& j, hipStream_t s)
{
    if (j.fa == E2M1) return launch_rows<E2M1, E2M1>(j, s);
    if (j.fa == E4M3) return j.fb == E4M3 ? launch_rows<E4M3, E4M3>(j, s) : launch_rows<E4M3, E5M2>(j, s);
    return j.fb == E4M3 ? launch_rows<E5M2, E4M3>(j, s) : launch_rows<E5M2, E5M2>(j, s);
}

}  // namespace mx
