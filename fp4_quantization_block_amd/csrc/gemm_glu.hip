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
// rows of Wg, then of Wu, as its first operand and up to 32 tokens as its
// second, so that a lane holds gate and up of the same elements.  A workgroup
// covers 32 elements of F (one block of a row copy); its waves split K and meet
// in LDS.
#include "act_device.h"
#include "mx_internal.h"

namespace mx {

namespace {

typedef int int8v __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));

constexpr int WAVES = 4;            // of a workgroup, which split K
constexpr int UNIT = 128;           // bytes of K a row that a wave takes at a time
constexpr int ROWS = 32;            // elements of F of a workgroup, and tokens of a tile
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

template <int FA, int FB>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(2, 2)))
void k_glu_rows(const GemmGluJob g, int tiles_f, int tiles_m)
{
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr bool FP4 = FA == E2M1;
    constexpr int EPB = FP4 ? 2 : 1, UBLOCKS = UNIT * EPB / 32;      // blocks of a unit
    constexpr int STEPS = UNIT * EPB / 64;                           // MFMA steps of a unit
    typedef Unit<FP4> U;
    __shared__ __align__(16) uint8_t lds[WAVES][3 * TILE];
    static_assert(sizeof lds >= WAVES * 2 * ROWS * PITCH * sizeof(float), "the joined sums take the place of the units");

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = lane >> 5, l32 = lane & 31;
    // the tiles of tokens of one set of weights run one after the other on one XCD
    const int wg = blockIdx.x, tf = wg / (8 * tiles_m) * 8 + wg % 8, tm = wg / 8 % tiles_m;
    if (tf >= tiles_f) return;
    const int64_t f0 = (int64_t)tf * ROWS, m0 = (int64_t)tm * ROWS;
    const int64_t kbytes = g.K / EPB, kblocks = g.K / 32;
    const int units = (int)(kbytes / UNIT), rest = (int)(kbytes % UNIT);   // whole ones, bytes of the last

    // codes: buffer loads over the tile's rows (at most 2^28 bytes), so that
    // rows past the end are zero and not fetched; their scales are the last row's
    auto rsrc = [&](const uint8_t* base, int64_t first, int64_t rows) __attribute__((always_inline)) {
        const int64_t n = min(rows - first, (int64_t)ROWS) * kbytes;
        return __builtin_amdgcn_make_buffer_rsrc((void*)(base + first * kbytes), (short)0, (int)(uint32_t)n, 0x00020000);
    };
    const auto rg = rsrc(g.qg, f0, g.F), ru = rsrc(g.qu, f0, g.F), rt = rsrc(g.qa, m0, g.M);
    const int64_t wrow = min(f0 + l32, g.F - 1), trow = min(m0 + l32, g.M - 1);
    const uint8_t *sg = g.sg + wrow * kblocks, *su = g.su + wrow * kblocks, *st = g.sa + trow * kblocks;
    const uint32_t voff = (uint32_t)((lane >> 3) * kbytes + (lane & 7) * 16), run = (uint32_t)(8 * kbytes);

    f16v acc[2];
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int r = 0; r < 16; r++) acc[i][r] = 0.0f;

    struct Stage { U g, u, t; };
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
        load_codes(s.t, rt, off, u);
        const int64_t at = (int64_t)u * UBLOCKS;
        __builtin_memcpy(s.g.s, sg + at, sizeof s.g.s);              // (at any address)
        __builtin_memcpy(s.u.s, su + at, sizeof s.u.s);
        __builtin_memcpy(s.t.s, st + at, sizeof s.t.s);
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
            const int8v xt = source<FP4>(mine + 2 * TILE, k, l32, h);
            const int a = (int)(s.g.s[k / 2] >> (8 * h)), b = (int)(s.u.s[k / 2] >> (8 * h)), c = (int)(s.t.s[k / 2] >> (8 * h));
            if (k % 2 == 0) {
                acc[0] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xg, xt, acc[0], MfmaFmt<FB>::code, MfmaFmt<FA>::code, 0, a, 0, c);
                acc[1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xu, xt, acc[1], MfmaFmt<FB>::code, MfmaFmt<FA>::code, 0, b, 0, c);
            } else {
                acc[0] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xg, xt, acc[0], MfmaFmt<FB>::code, MfmaFmt<FA>::code, 2, a, 2, c);
                acc[1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xu, xt, acc[1], MfmaFmt<FB>::code, MfmaFmt<FA>::code, 2, b, 2, c);
            }
        }
    };
    // A wave's LDS operations run in order, so its part needs no barrier, only
    // that the compiler keeps the order too.
    auto put_all = [&](const Stage& s) __attribute__((always_inline)) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        put(s.g, mine);
        put(s.u, mine + TILE);
        put(s.t, mine + 2 * TILE);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
    // one unit: to LDS, its registers free for unit i, its products
    auto step = [&](Stage& s, int i) __attribute__((always_inline)) {
        put_all(s);
        Stage scales;
        __builtin_memcpy(scales.g.s, s.g.s, sizeof s.g.s);
        __builtin_memcpy(scales.u.s, s.u.s, sizeof s.u.s);
        __builtin_memcpy(scales.t.s, s.t.s, sizeof s.t.s);
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
        load_codes(a.t, rt, at, units);
#pragma unroll
        for (int d = 0; d < U::DWORDS; d++) {
            a.g.s[d] = a.u.s[d] = a.t.s[d] = 0;
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const int64_t block = (int64_t)units * UBLOCKS + 4 * d + k;
                const bool in = block < kblocks;
                a.g.s[d] |= (in ? (uint32_t)sg[block] : 127u) << (8 * k);
                a.u.s[d] |= (in ? (uint32_t)su[block] : 127u) << (8 * k);
                a.t.s[d] |= (in ? (uint32_t)st[block] : 127u) << (8 * k);
            }
        }
        put_all(a);
        multiply(a);
    }

    // join: [wave][row of the two MFMA tiles][token], in the units' place
    float* const red = (float*)&lds[0][0];
    constexpr int PART = 2 * ROWS * PITCH;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int r = 0; r < 16; r++) red[wave * PART + (ROWS * i + 8 * (r / 4) + 4 * h + r % 4) * PITCH + l32] = acc[i][r];

    float common = g.alpha;
    if (g.ta) common = common * *g.ta;
    float ag = common, au = common;
    if (g.tg) ag = ag * *g.tg;
    if (g.tu) au = au * *g.tu;
    if (g.hadamard_k) ag = ag * 0.03125f, au = au * 0.03125f;
    __syncthreads();

    // thread t: tokens t / 16 and 16 further on, elements 2 (t % 16) and the next
    const int pair = 2 * (threadIdx.x & 15);
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
        const int64_t m = m0 + token, f = f0 + pair;
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
    const int tiles_f = (int)((j.F + ROWS - 1) / ROWS), tiles_m = (int)((j.M + ROWS - 1) / ROWS);
    const unsigned grid = (unsigned)((tiles_f + 7) / 8 * 8) * (unsigned)tiles_m;
    k_glu_rows<FA, FB><<<grid, 64 * WAVES, 0, s>>>(j, tiles_f, tiles_m);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_glu(const GemmGluJob& j, hipStream_t s)
{
    // k_glu_rows takes a time in proportion to its workgroups (32 rows x 32
    // elements), the GEMM kernels one in proportion to their rounds of a 256 x
    // 128 tile on each CU, both in proportion to K.  At F = 14336, K = 4096, by
    // rows and by tiles: M = 64 (896 workgroups) E4M3 37-48 and 51-65 us, E2M1
    // 24 and 36; M = 96 (1344) 64 and 66, 32 and 38; M = 128 (1792) 58-73 and
    // 51-70, 37 and 36; M = 256 127 and 51-76, 65 and 36.
    const int64_t wgs = ((j.M + ROWS - 1) / ROWS) * ((j.F + ROWS - 1) / ROWS);
    const int64_t rounds = (((j.M + 255) / 256) * ((j.F + 127) / 128) + 255) / 256;
    if (wgs > 6 * 256 * rounds) return launch_gemm_glu_tiles(j, s);
    if (j.fa == E2M1) return launch_rows<E2M1, E2M1>(j, s);
    if (j.fa == E4M3) return j.fb == E4M3 ? launch_rows<E4M3, E4M3>(j, s) : launch_rows<E4M3, E5M2>(j, s);
    return j.fb == E4M3 ? launch_rows<E5M2, E4M3>(j, s) : launch_rows<E5M2, E5M2>(j, s);
}

}  // namespace mx
