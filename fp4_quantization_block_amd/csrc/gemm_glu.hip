// gemm_glu.hip -- the gate and up projections of a gated MLP block with their
// activation and product in one kernel, for few rows:
//   gate = a_g A Wg^T,  up = a_u A Wu^T,  h = act(gate) * up,
// A [M][K], Wg and Wu [F][K] as MX codes with their scales, as in gemm.hip.
// ([FAF, "格式感知融合的设计思路"]: the producer writes what its consumer reads,
// here h as the down projection's operand and the 8-bit checkpoints of gate
// and up, [COAT, "FP8啟用"].)
//
// Many rows run on the GEMM kernels (gemm.hip), k_glu_rows below takes few:
// their time goes to reading the weights once.  The matrix instruction gets 32
// rows of Wg, then of Wu, as its first operand and 32 tokens as its second, so
// that a lane holds gate and up of the same elements.  A workgroup covers 32
// elements of F (one block of a row copy) and TM tiles of 32 tokens; its waves
// split K and meet in LDS.
#include "act_device.h"
#include "mx_internal.h"

namespace mx {

namespace {

typedef int int8v __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));

constexpr int WAVES = 4;            // of a workgroup, which split K
constexpr int UNIT = 128;           // bytes of K a row that a wave takes at a time
constexpr int ROWS = 32;            // elements of F of a workgroup, tokens of a tile
constexpr int TILE = ROWS * UNIT;   // bytes of a unit of one operand
constexpr int PITCH = 33;           // of the joined sums: rows of 32 tokens, one float between

template <int FMT> struct MfmaFmt;
template <> struct MfmaFmt<E4M3> { static constexpr int code = 0; };
template <> struct MfmaFmt<E5M2> { static constexpr int code = 1; };
template <> struct MfmaFmt<E2M1> { static constexpr int code = 4; };

// One unit of an operand on its way: global -> registers -> the wave's own LDS
// -> the lanes that multiply it.  A load instruction covers eight whole 128-byte
// lines, eight lanes to a row.  (Loaded straight into the lane layout of the
// matrix instruction, 16 bytes of 32 rows at a time, a line is asked for four
// times: 37 us instead of 31 for one token at 4096 x 14336 E4M3, 63 instead of
// 34 for 32 tokens.)
template <bool FP4>
struct Unit {
    static constexpr int DWORDS = FP4 ? 2 : 1;       // scale dwords of a row
    uint4 q[4];                                      // rows 8 p + lane / 8, chunk lane % 8
    uint32_t s[DWORDS];                              // of row lane % 32
};

// LDS offset of 16-byte chunk `chunk` of row `row`: the key keeps the fragment
// reads (one chunk of 32 rows) off each other's banks
__device__ __forceinline__ int swz(int row, int chunk) { return row * UNIT + ((chunk ^ ((row >> 1) & 7)) << 4); }

// Source of one MFMA step from the unit in LDS.  Lane layout of the 32x32x64
// scaled MFMA (gemm.hip): lane l holds row l % 32; of a step's 64 elements, with
// h = l / 32, the 16-byte halves of blocks 0 and 1 that h names (FP8), or block
// h (FP4).
template <bool FP4>
__device__ __forceinline__ int8v source(const uint8_t* lds, int step, int l32, int h)
{
    if constexpr (FP4) {
        const uint4 a = *(const uint4*)(lds + swz(l32, 2 * step + h));
        return int8v{(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    } else {
        const uint4 a = *(const uint4*)(lds + swz(l32, 4 * step + h)), b = *(const uint4*)(lds + swz(l32, 4 * step + 2 + h));
        return int8v{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
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

template <int FA, int FB, int TM>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(2, 2)))
void k_glu_rows(const GemmGluJob g, int tiles_f, int tiles_m)
{
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr bool FP4 = FA == E2M1;
    constexpr int EPB = FP4 ? 2 : 1, UBLOCKS = UNIT * EPB / 32;      // blocks of a unit
    constexpr int STEPS = UNIT * EPB / 64;                           // MFMA steps of a unit
    typedef Unit<FP4> U;
    __shared__ __align__(16) uint8_t lds[WAVES][(2 + TM) * TILE];
    static_assert(sizeof lds >= WAVES * 2 * ROWS * PITCH * sizeof(float), "the joined sums take the place of the units");

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = lane >> 5, l32 = lane & 31;
    // the tiles of tokens of one set of weights run one after the other on one XCD
    const int wg = blockIdx.x, tf = wg / (8 * tiles_m) * 8 + wg % 8, tm = wg / 8 % tiles_m;
    if (tf >= tiles_f) return;
    const int64_t f0 = (int64_t)tf * ROWS, m0 = (int64_t)tm * (TM * ROWS);
    const int64_t kbytes = g.K / EPB, kblocks = g.K / 32;
    const int units = (int)(kbytes / UNIT), rest = (int)(kbytes % UNIT);   // whole ones, bytes of the last

    // codes: buffer loads over the tile's rows (at most 2^28 bytes), so that
    // rows past the end are zero and not fetched; their scales are the last row's
    auto rsrc = [&](const uint8_t* base, int64_t first, int64_t rows) __attribute__((always_inline)) {
        const int64_t n = max(min(rows - first, (int64_t)ROWS), (int64_t)0) * kbytes;
        return __builtin_amdgcn_make_buffer_rsrc((void*)(base + first * kbytes), (short)0, (int)(uint32_t)n, 0x00020000);
    };
    const auto rg = rsrc(g.qg, f0, g.F), ru = rsrc(g.qu, f0, g.F);
    const int64_t wrow = min(f0 + l32, g.F - 1);
    const uint8_t *sg = g.sg + wrow * kblocks, *su = g.su + wrow * kblocks, *st[TM];
    __amdgpu_buffer_rsrc_t rt[TM];
#pragma unroll
    for (int i = 0; i < TM; i++) {
        rt[i] = rsrc(g.qa, m0 + i * ROWS, g.M);
        st[i] = g.sa + min(m0 + i * ROWS + l32, g.M - 1) * kblocks;
    }
    const uint32_t voff = (uint32_t)((lane >> 3) * kbytes + (lane & 7) * 16), run = (uint32_t)(8 * kbytes);

    f16v acc[TM][2];
#pragma unroll
    for (int t = 0; t < TM; t++)
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int r = 0; r < 16; r++) acc[t][i][r] = 0.0f;

    struct Stage { U g, u, t[TM]; };
    auto load_codes = [&](U& x, __amdgpu_buffer_rsrc_t r, uint32_t at, int u) __attribute__((always_inline)) {
#pragma unroll
        for (int p = 0; p < 4; p++)
            x.q[p] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, at + p * run, u * UNIT, 0));
    };
    constexpr uint32_t OUTSIDE = 0xF0000000u;       // past every tile's rows, whatever run is added
    const int n = (units - wave + WAVES - 1) / WAVES;                 // units wave, wave + WAVES, ... of this wave
    // unit i of the wave; one behind its last is not fetched (and not used), so
    // that no load is conditional
    auto load = [&](Stage& s, int i) __attribute__((always_inline)) {
        const int u = wave + min(i, n - 1) * WAVES;
        const uint32_t off = i < n ? voff : OUTSIDE;
        load_codes(s.g, rg, off, u);
        load_codes(s.u, ru, off, u);
#pragma unroll
        for (int t = 0; t < TM; t++) load_codes(s.t[t], rt[t], off, u);
        const int64_t at = (int64_t)u * UBLOCKS;
        __builtin_memcpy(s.g.s, sg + at, sizeof s.g.s);              // (at any address)
        __builtin_memcpy(s.u.s, su + at, sizeof s.u.s);
#pragma unroll
        for (int t = 0; t < TM; t++) __builtin_memcpy(s.t[t].s, st[t] + at, sizeof s.t[t].s);
    };
    uint8_t* const mine = lds[wave];
    const int wat = swz(lane >> 3, lane & 7);                         // (rows 8 apart: the key's other bits below)
    auto put = [&](const U& x, uint8_t* to) __attribute__((always_inline)) {
#pragma unroll
        for (int p = 0; p < 4; p++) *(uint4*)(to + p * 8 * UNIT + (wat ^ ((p & 1) << 6))) = x.q[p];
    };
    auto multiply = [&](const Stage& s) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < STEPS; k++) {
            const int8v xg = source<FP4>(mine, k, l32, h), xu = source<FP4>(mine + TILE, k, l32, h);
            const int a = (int)(s.g.s[k / 2] >> (8 * h)), b = (int)(s.u.s[k / 2] >> (8 * h));
#pragma unroll
            for (int t = 0; t < TM; t++) {
                const int8v xt = source<FP4>(mine + (2 + t) * TILE, k, l32, h);
                const int c = (int)(s.t[t].s[k / 2] >> (8 * h));
                if (k % 2 == 0) {
                    acc[t][0] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xg, xt, acc[t][0], MfmaFmt<FB>::code, MfmaFmt<FA>::code, 0, a, 0, c);
                    acc[t][1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xu, xt, acc[t][1], MfmaFmt<FB>::code, MfmaFmt<FA>::code, 0, b, 0, c);
                } else {
                    acc[t][0] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xg, xt, acc[t][0], MfmaFmt<FB>::code, MfmaFmt<FA>::code, 2, a, 2, c);
                    acc[t][1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xu, xt, acc[t][1], MfmaFmt<FB>::code, MfmaFmt<FA>::code, 2, b, 2, c);
                }
            }
        }
    };
    // A wave's LDS operations run in order, so its part needs no barrier, only
    // that the compiler keeps the order too.
    auto put_all = [&](const Stage& s) __attribute__((always_inline)) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        put(s.g, mine);
        put(s.u, mine + TILE);
#pragma unroll
        for (int t = 0; t < TM; t++) put(s.t[t], mine + (2 + t) * TILE);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
    // one unit: to LDS, its registers free for unit i, its products
    auto step = [&](Stage& s, int i) __attribute__((always_inline)) {
        put_all(s);
        Stage scales;
        __builtin_memcpy(scales.g.s, s.g.s, sizeof s.g.s);
        __builtin_memcpy(scales.u.s, s.u.s, sizeof s.u.s);
#pragma unroll
        for (int t = 0; t < TM; t++) __builtin_memcpy(scales.t[t].s, s.t[t].s, sizeof s.t[t].s);
        load(s, i);
        multiply(scales);
    };
    // two units in flight
    Stage a, b;
    if (n > 0) {
        load(a, 0);
        load(b, 1);
#pragma unroll 1
        for (int i = 0; i < n; i += 2) {
            step(a, i + 2);
            if (i + 1 < n) step(b, i + 3);
        }
    }
    // what is left of K behind the whole units: chunks past its end are fetched
    // from past every row's end, which gives zeros, with the scale 1
    if (rest != 0 && wave == units % WAVES) {
        const uint32_t at = (lane & 7) * 16 < rest ? voff : OUTSIDE;
        load_codes(a.g, rg, at, units);
        load_codes(a.u, ru, at, units);
#pragma unroll
        for (int t = 0; t < TM; t++) load_codes(a.t[t], rt[t], at, units);
        auto scales = [&](U& x, const uint8_t* from) __attribute__((always_inline)) {
#pragma unroll
            for (int d = 0; d < U::DWORDS; d++) {
                x.s[d] = 0;
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const int64_t block = (int64_t)units * UBLOCKS + 4 * d + k;
                    x.s[d] |= (block < kblocks ? (uint32_t)from[block] : 127u) << (8 * k);
                }
            }
        };
        scales(a.g, sg);
        scales(a.u, su);
#pragma unroll
        for (int t = 0; t < TM; t++) scales(a.t[t], st[t]);
        put_all(a);
        multiply(a);
    }

    float common = g.alpha;
    if (g.ta) common = common * *g.ta;
    float ag = common, au = common;
    if (g.tg) ag = ag * *g.tg;
    if (g.tu) au = au * *g.tu;
    if (g.hadamard_k) ag = ag * 0.03125f, au = au * 0.03125f;

    // join, a tile of tokens at a time: [wave][row of the two MFMA tiles][token],
    // in the units' place
    float* const red = (float*)&lds[0][0];
    constexpr int PART = 2 * ROWS * PITCH;
    const int pair = 2 * (threadIdx.x & 15);
#pragma unroll
    for (int t = 0; t < TM; t++) {
        if (m0 + t * ROWS >= g.M) break;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int r = 0; r < 16; r++)
                red[wave * PART + (ROWS * i + 8 * (r / 4) + 4 * h + r % 4) * PITCH + l32] = acc[t][i][r];
        __syncthreads();
        // thread x: tokens x / 16 and 16 further on, elements 2 (x % 16) and the next
#pragma unroll
        for (int token = threadIdx.x >> 4; token < ROWS; token += 4 * WAVES) {
            float gv[2] = {0.0f, 0.0f}, uv[2] = {0.0f, 0.0f}, hv[2];
#pragma unroll
            for (int w = 0; w < WAVES; w++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    gv[e] += red[w * PART + (pair + e) * PITCH + token];
                    uv[e] += red[w * PART + (ROWS + pair + e) * PITCH + token];
                }
#pragma unroll
            for (int e = 0; e < 2; e++) {
                gv[e] *= ag;
                uv[e] *= au;
                hv[e] = gate_value(g.act, gv[e]) * uv[e];
            }
            const int64_t m = m0 + t * ROWS + token, f = f0 + pair;
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
    }
#endif
}

template <int FA, int FB, int TM>
hipError_t launch_rows(const GemmGluJob& j, hipStream_t s)
{
    const int tiles_f = (int)((j.F + ROWS - 1) / ROWS), tiles_m = (int)((j.M + TM * ROWS - 1) / (TM * ROWS));
    const unsigned grid = (unsigned)((tiles_f + 7) / 8 * 8) * (unsigned)tiles_m;
    k_glu_rows<FA, FB, TM><<<grid, 64 * WAVES, 0, s>>>(j, tiles_f, tiles_m);
    return hipGetLastError();
}

template <int TM>
hipError_t launch_rows(const GemmGluJob& j, hipStream_t s)
{
    if (j.fa == E2M1) return launch_rows<E2M1, E2M1, TM>(j, s);
    if (j.fa == E4M3) return j.fb == E4M3 ? launch_rows<E4M3, E4M3, TM>(j, s) : launch_rows<E4M3, E5M2, TM>(j, s);
    return j.fb == E4M3 ? launch_rows<E5M2, E4M3, TM>(j, s) : launch_rows<E5M2, E5M2, TM>(j, s);
}

}  // namespace

hipError_t launch_gemm_glu(const GemmGluJob& j, hipStream_t s)
{
    // Workgroups of 32 tokens that all run at once (one on each CU) are left
    // narrow, more of them take two tiles of tokens (n: how many there are then).
    // At F = 4096, K = 2048 E4M3, 32 and 64 tokens a workgroup: M = 64 8.1 and
    // 10.5 us, M = 128 12.7 and 10.8, M = 256 22 and 17; at F = 14336, K = 4096:
    // M = 64 48 and 41 (E2M1 22.5 and 18.9).  Four tiles were no better: M = 128
    // 61 us, two 60.
    const int64_t tiles_f = (j.F + ROWS - 1) / ROWS, n = (j.M + 2 * ROWS - 1) / (2 * ROWS) * tiles_f;
    const bool narrow = j.M <= ROWS || (j.M + ROWS - 1) / ROWS * tiles_f <= 256;
    // These take a time in proportion to n, the GEMM kernels one in proportion to
    // their rounds, all in proportion to K.  Rows and tiles: where one round of
    // half tiles is enough (F = 2048, K = 4096 E4M3) n = 512 25 and 33 us, n =
    // 1024 46 and 34 (E2M1 17 and 20, 28 and 21); F = 14336 n = 448 41 and 43, n =
    // 896 54 and 44; else, a round (F = 28672 and 65536) n = 896 74.5 and 74.7 (E2M1
    // 41-44 and 44), n = 1024 74-77 and 78 (47 and 56), n = 1792 103 and 77; K not a
    // multiple of 128 bytes n = 896 69 and 82, n = 1792 100 and 98.
    bool half;
    const int64_t rounds = gemm_glu_rounds(j, half);
    // (The launch counts its threads with 32 bits, and pads tiles_f to eight.)
    if (n > (half ? 640 : 1024 * rounds) || n > 1 << 20) return launch_gemm_glu_tiles(j, s);
    return narrow ? launch_rows<1>(j, s) : launch_rows<2>(j, s);
}

}  // namespace mx
