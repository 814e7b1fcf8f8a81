// glu.hip -- the gated activation h = act(g) u and its gradients for gfx950:
//   dg = dh u act'(g),   du = dh act(g)
// with g and u read from tensors or from their 8-bit checkpoints (MX row
// copies, [COAT, "FP8啟用"]).  The forward can write h as the row copy that
// the next GEMM reads, and the checkpoints; the dual-layout backward writes
// the operands of the backward GEMMs ([FAF, "格式感知融合的设计思路"]).
//
// Sources:
//   [COAT] write-up of "COAT: Compressing Optimizer States and Activation for
//          memory efficient FP8 Training"
//   [FAF]  "格式感知融合:让FP4预训练提速两倍的工程实践"
//
// Kernels (times at 8192 x 14336 bf16, SiLU, on one MI355X, where a 1 GiB copy
// runs at 5.1 TB/s)
//   k_glu_fwd, k_glu_bwd   one chunk of eight elements per thread, in order
//                    over rows and columns: each byte read and written once,
//                    and bound by that.  The forward with h as E4M3 codes and
//                    both checkpoints, 833 MB: 145 us, 5.7 TB/s.  The
//                    backward from the checkpoints, 947 MB: 163 us, 5.8 TB/s.
//   k_glu_bwd_dual   tiles whose gradients never leave registers before they
//                    are codes, in both layouts.  From the checkpoints, with
//                    h, 1083 MB: 239 us, 4.5 TB/s (counters: 493 MB read, 622
//                    MB written).  The same by k_glu_bwd and the dual-layout
//                    quantizer moves 2.1 GB.
#include "act_device.h"
#include "mx_internal.h"

namespace mx {

namespace {

// n / d for 32-bit n and a divisor known to the host, by the round-up method
// (T. Granlund and P. Montgomery, "Division by Invariant Integers using
// Multiplication", PLDI 1994, figure 4.1): floor((2^32 + m) n / 2^(32 + l)), 2^l
// the power of two at or above d and m = floor(2^32 (2^l - d) / d) + 1
struct FastDiv { uint32_t d, m, s1, s2; };

FastDiv fast_div(uint32_t d)
{
    uint32_t l = 0;
    while (l < 32 && (1ull << l) < d) l++;
    const uint32_t m = (uint32_t)(((1ull << 32) * ((1ull << l) - d)) / d + 1);
    return FastDiv{d, m, l < 1 ? l : 1u, l > 0 ? l - 1 : 0u};
}

__device__ __forceinline__ uint32_t quotient(const FastDiv& f, uint32_t n)
{
    const uint32_t t = __umulhi(f.m, n);
    return (t + ((n - t) >> f.s1)) >> f.s2;
}

// Places of a thread:
//   WHOLE    the eight consecutive elements of chunk `id`; rows are multiples
//            of eight
//   OVERLAP  the same for any row of at least eight: a row's last chunk is
//            its last eight elements, some of which the chunk before has too,
//            with the same results
//   STRIDED  elements id * 2048 + i * 256 + thread: any row, no element twice
//            (an output may be written over an input)
// `units` counts chunks (WHOLE, OVERLAP) or elements.
enum : int { WHOLE, OVERLAP, STRIDED };

template <int MODE>
struct Place {
    static constexpr int NP = MODE == STRIDED ? 8 : 1;
    uint32_t row[NP], col[NP];
    bool ok[NP];
    __device__ __forceinline__ Place(const FastDiv& per_row, uint32_t units, uint32_t cols)
    {
#pragma unroll
        for (int i = 0; i < NP; i++) {
            uint32_t u = MODE == STRIDED ? blockIdx.x * 2048u + 256u * i + threadIdx.x : blockIdx.x * 256u + threadIdx.x;
            ok[i] = u < units;
            u = ok[i] ? u : 0u;
            row[i] = quotient(per_row, u);
            col[i] = (u - row[i] * per_row.d) * (MODE == STRIDED ? 1u : 8u);
            if (MODE == OVERLAP) col[i] = min(col[i], cols - 8u);
        }
    }
    template <int SRC>
    __device__ __forceinline__ void load(const void* p, int64_t ld, float (&v)[8]) const
    {
        if constexpr (MODE != STRIDED) {
            const Chunk<SRC> c = load_chunk<SRC>(p, row[0] * ld + col[0]);
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = chunk_value<SRC>(c, i);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = load_elem<SRC>(p, row[i] * ld + col[i]);
        }
    }
    template <int SRC>
    __device__ __forceinline__ void store(void* p, int64_t ld, const float (&v)[8]) const
    {
        if constexpr (MODE != STRIDED) {
            if (ok[0]) store_chunk<SRC>(p, row[0] * ld + col[0], make_chunk<SRC>(v));
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (ok[i]) store_elem<SRC>(p, row[i] * ld + col[i], v[i]);
        }
    }
    // place in a dense row copy (WHOLE)
    __device__ __forceinline__ int64_t dense(int64_t cols) const { return row[0] * cols + col[0]; }
};

template <int SRC, int ACT, int MODE>
__global__ __launch_bounds__(256) void k_glu_fwd(GluFwdJob a, FastDiv per_row, uint32_t units)
{
    const Place<MODE> at(per_row, units, (uint32_t)a.cols);
    float g[8], u[8], h[8];
    at.template load<SRC>(a.gate, a.ld_gate, g);
    at.template load<SRC>(a.up, a.ld_up, u);
#pragma unroll
    for (int i = 0; i < 8; i++) {
        float act, slope;
        gate<ACT, false>(g[i], act, slope);
        h[i] = act * u[i];
    }
    if (a.h) {
        if (a.out_f32) at.template store<SRC_F32>(a.h, a.ld_h, h);
        else at.template store<SRC_BF16>(a.h, a.ld_h, h);
    }
    if constexpr (MODE == WHOLE) {
        const int64_t e = at.dense(a.cols);
        if (a.qh) encode_row_chunk(a.h_fmt, h, at.ok[0], e, a.qh, a.sh);
        if (a.qg) {
            encode_row_chunk(a.ckpt_fmt, g, at.ok[0], e, a.qg, a.sg);
            encode_row_chunk(a.ckpt_fmt, u, at.ok[0], e, a.qu, a.su);
        }
    }
}

template <int SRC, int ACT, int FROM, int MODE>
__global__ __launch_bounds__(256) void k_glu_bwd(GluBwdJob a, FastDiv per_row, uint32_t units)
{
    const Place<MODE> at(per_row, units, (uint32_t)a.cols);
    float d[8], g[8], u[8], h[8];
    at.template load<SRC>(a.dh, a.ld_dh, d);
    if constexpr (FROM != FROM_TENSOR) {
        const int64_t e = at.dense(a.cols);
        const uint2 cg = *(const uint2*)(a.qg + e), cu = *(const uint2*)(a.qu + e);
        const uint32_t bg = a.sg[e >> 5], bu = a.su[e >> 5];
        decode8<FROM>(cg, bg, g);
        decode8<FROM>(cu, bu, u);
    } else {
        at.template load<SRC>(a.gate, a.ld_gate, g);
        at.template load<SRC>(a.up, a.ld_up, u);
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
        float act, slope;
        gate<ACT, true>(g[i], act, slope);
        h[i] = act * u[i];
        g[i] = d[i] * u[i] * slope;
        u[i] = d[i] * act;
    }
    at.template store<SRC>(a.dgate, a.ld_dgate, g);
    at.template store<SRC>(a.dup, a.ld_dup, u);
    if (a.h) at.template store<SRC>(a.h, a.ld_h, h);
}

// Launches of at most 2^31 elements: the rows of a larger tensor are taken in
// slices, since the kernels count places in 32 bits.
template <int MODE, class F>
hipError_t sliced(int64_t rows, int64_t cols, F&& f)
{
    const int64_t per_row = MODE == STRIDED ? cols : (cols + 7) / 8, most = ((int64_t)1 << 31) / per_row;
    const FastDiv d = fast_div((uint32_t)per_row);
    for (int64_t r = 0; r < rows; r += most) {
        const int64_t n = rows - r < most ? rows - r : most, units = n * per_row;
        const int64_t per_group = MODE == STRIDED ? 2048 : 256;
        f(r, n, d, (uint32_t)units, dim3((unsigned)((units + per_group - 1) / per_group)));
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

// f(how the rows are taken): `in_place` where an output is written over an input
template <class F>
hipError_t by_mode(int64_t cols, bool in_place, F&& f)
{
    if (cols % 8 == 0) return f(std::integral_constant<int, WHOLE>());
    if (cols > 8 && !in_place) return f(std::integral_constant<int, OVERLAP>());
    return f(std::integral_constant<int, STRIDED>());
}

template <class T>
void advance(T*& p, int64_t bytes)
{
    if (p) p = (T*)((uint8_t*)p + bytes);
}

template <int SRC, int ACT, int MODE>
hipError_t run_fwd(const GluFwdJob& job, hipStream_t s)
{
    return sliced<MODE>(job.rows, job.cols, [&](int64_t r, int64_t n, FastDiv d, uint32_t units, dim3 grid) {
        GluFwdJob j = job;
        constexpr int64_t B = ElemT<SRC>::bytes;
        j.rows = n;
        advance(j.gate, r * j.ld_gate * B);
        advance(j.up, r * j.ld_up * B);
        advance(j.h, r * j.ld_h * (j.out_f32 ? 4 : 2));
        for (uint8_t** q : {&j.qh, &j.qg, &j.qu}) advance(*q, r * j.cols);
        for (uint8_t** q : {&j.sh, &j.sg, &j.su}) advance(*q, r * (j.cols / 32));
        k_glu_fwd<SRC, ACT, MODE><<<grid, dim3(256), 0, s>>>(j, d, units);
    });
}

template <int SRC, int ACT, int FROM, int MODE>
hipError_t run_bwd(const GluBwdJob& job, hipStream_t s)
{
    return sliced<MODE>(job.rows, job.cols, [&](int64_t r, int64_t n, FastDiv d, uint32_t units, dim3 grid) {
        GluBwdJob j = job;
        constexpr int64_t B = ElemT<SRC>::bytes;
        j.rows = n;
        advance(j.dh, r * j.ld_dh * B);
        advance(j.gate, r * j.ld_gate * B);
        advance(j.up, r * j.ld_up * B);
        advance(j.dgate, r * j.ld_dgate * B);
        advance(j.dup, r * j.ld_dup * B);
        advance(j.h, r * j.ld_h * B);
        for (const uint8_t** q : {&j.qg, &j.qu}) advance(*q, r * j.cols);
        for (const uint8_t** q : {&j.sg, &j.su}) advance(*q, r * (j.cols / 32));
        k_glu_bwd<SRC, ACT, FROM, MODE><<<grid, dim3(256), 0, s>>>(j, d, units);
    });
}

template <class F>
hipError_t by_act(int act, F&& f)
{
    if (act == ACT_SILU) return f(std::integral_constant<int, ACT_SILU>());
    if (act == ACT_GELU) return f(std::integral_constant<int, ACT_GELU>());
    return f(std::integral_constant<int, ACT_GELU_TANH>());
}

// ---------------------------------------------------------------------------
// k_glu_bwd_dual: workgroups of WR x WC waves walk tiles of 32 WR rows by
// 64 WC columns of h; a wave takes 32 x 64 of them.  Lane 8 k + m holds rows
// 4 m .. 4 m + 3 and columns 8 k .. 8 k + 7, so that a wave's loads of bf16
// rows are whole 128-byte lines: a column block is spread over eight
// neighbouring lanes, a row block over four lanes 8 apart, and both maxima
// are two or three cross-lane steps on registers.  A lane's codes of a row
// (eight columns) or of a column (four rows) are two dwords or one, and go
// through LDS to leave as whole runs of a row or a column.  The next tile's
// inputs are loaded into registers before the current tile is worked on.
//
// Tiles are 128 x 128, so that every input and output line of codes is a
// whole 128-byte line of one tile: an L2 (4 MiB for 32 CUs) keeps a line for
// some microseconds at this kernel's rate, too short to wait for the tile
// that has the other half.  A row's scale bytes are 4 per tile; a workgroup
// takes its tiles along the rows, and reads and writes the scale bytes of up
// to 16 tiles at a time through LDS.
//
// What it waits for, timed with parts of it left out (8192 x 14336, 263 us
// then): no loads and no stores 179 us, no loads 193, no stores 223.  So the
// arithmetic (five encodings of 1 1/2 steps an element, the gate, the block
// maxima; vector units busy 47% of the time at two waves a SIMD) and the
// memory traffic overlap in part; one workgroup a CU, held by 256 registers a
// lane and 129 KiB of LDS, meets at two barriers a tile.  Measured slower: 16
// waves with 4 x 4 values a lane (275 us: half-line loads), 64-row tiles two
// to a CU (289: 64-byte runs), 256 x 64 tiles (303), stores that bypass the
// cache (290 against 275 then), double row buffers (294 against 286 then).
// ---------------------------------------------------------------------------

// Block maxima from the lanes' own, for several blocks a step at a time (a
// cross-lane step has to wait for the one before on the same register).

// over the four lanes 8 apart that hold a row block: l ^ 8 (in the 16-lane
// row) and l ^ 16
template <int B>
__device__ __forceinline__ void row_block_max(uint32_t (&k)[B])
{
#pragma unroll
    for (int j = 0; j < B; j++) k[j] = max(k[j], dpp<0x128>(k[j]));        // rotate by 8 in a row of 16
#pragma unroll
    for (int j = 0; j < B; j++) {
        auto p = __builtin_amdgcn_permlane16_swap(k[j], k[j], false, false);
        k[j] = max((uint32_t)p[0], (uint32_t)p[1]);
    }
}

// over eight neighbouring lanes
template <int B>
__device__ __forceinline__ void oct_max(uint32_t (&k)[B])
{
#pragma unroll
    for (int j = 0; j < B; j++) k[j] = max(k[j], dpp<DPP_XOR1>(k[j]));
#pragma unroll
    for (int j = 0; j < B; j++) k[j] = max(k[j], dpp<DPP_XOR2>(k[j]));
#pragma unroll
    for (int j = 0; j < B; j++) k[j] = max(k[j], dpp<DPP_HALF_MIRROR>(k[j]));
}

// Waits for this wave's LDS traffic only (its global loads and stores stay in
// flight), then meets the workgroup.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// the inputs of one lane's 4 x 8 values, as they are in memory
template <int SRC, bool TENSOR> struct DualRaw;
template <int SRC> struct DualRaw<SRC, true> { Chunk<SRC> d[4], g[4], u[4]; };
template <int SRC> struct DualRaw<SRC, false> { Chunk<SRC> d[4]; uint2 g[4], u[4]; };

// Accesses at base + offset, base the same for the whole wave and offset a
// lane's, in the form of one scalar address and a 32-bit vector offset.  (The
// compiler would otherwise add a loop-invariant offset to the tensor's base
// first, and hold a 64-bit address in vector registers for every access.)
// V: an integer, or a vector of 32-bit ones, at any alignment.
#define MX_GLOBAL __attribute__((address_space(1)))
typedef uint32_t dwords2 __attribute__((ext_vector_type(2)));
typedef uint32_t dwords4 __attribute__((ext_vector_type(4)));
template <class V> struct __attribute__((packed)) Unaligned { V v; };

template <class V>
__device__ __forceinline__ MX_GLOBAL Unaligned<V>* lane_at(const void* base, uint32_t offset)
{
    MX_GLOBAL uint8_t* b = (MX_GLOBAL uint8_t*)base;
    asm("" : "+s"(b));
    asm("" : "+v"(offset));
    return (MX_GLOBAL Unaligned<V>*)(b + offset);
}

template <int SRC>
__device__ __forceinline__ Chunk<SRC> lane_chunk(const void* base, uint32_t offset)
{
    if constexpr (SRC == SRC_BF16) {
        return __builtin_bit_cast(Chunk<SRC>, dwords4(lane_at<dwords4>(base, offset)->v));
    } else {
        struct { dwords4 lo, hi; } w = {lane_at<dwords4>(base, offset)->v, lane_at<dwords4>(base, offset + 16)->v};
        return __builtin_bit_cast(Chunk<SRC>, w);
    }
}

// Places of a lane in the tiles' inputs: byte offsets from a tile's first
// element, 32 bits of them (row strides are at most 2^23), so that the loads
// share one address register a tensor, with the row added to the scalar base
struct DualAt { uint32_t d, g, u, q; };

template <int SRC, bool TENSOR>
__device__ __forceinline__ void dual_load_dh(const GluBwdJob& a, int64_t row, int64_t col, const DualAt& at,
                                             DualRaw<SRC, TENSOR>& r)
{
#pragma unroll
    for (int i = 0; i < 4; i++)
        r.d[i] = lane_chunk<SRC>((const uint8_t*)a.dh + ((row + i) * a.ld_dh + col) * ElemT<SRC>::bytes, at.d);
}

template <int SRC, bool TENSOR>
__device__ __forceinline__ void dual_load_gate(const GluBwdJob& a, int64_t row, int64_t col, const DualAt& at,
                                               DualRaw<SRC, TENSOR>& r)
{
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if constexpr (TENSOR) r.g[i] = lane_chunk<SRC>((const uint8_t*)a.gate + ((row + i) * a.ld_gate + col) * ElemT<SRC>::bytes, at.g);
        else r.g[i] = __builtin_bit_cast(uint2, dwords2(lane_at<dwords2>(a.qg + (row + i) * a.cols + col, at.q)->v));
    }
}

template <int SRC, bool TENSOR>
__device__ __forceinline__ void dual_load_up(const GluBwdJob& a, int64_t row, int64_t col, const DualAt& at,
                                             DualRaw<SRC, TENSOR>& r)
{
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if constexpr (TENSOR) r.u[i] = lane_chunk<SRC>((const uint8_t*)a.up + ((row + i) * a.ld_up + col) * ElemT<SRC>::bytes, at.u);
        else r.u[i] = __builtin_bit_cast(uint2, dwords2(lane_at<dwords2>(a.qu + (row + i) * a.cols + col, at.q)->v));
    }
}

// Staged lines of LB code bytes are LB + 8 bytes apart: the eight lines that
// a wave writes row codes of at once are four lines apart, and start in eight
// different groups of eight banks.  Column codes are written eight lines
// apart, two lines to a group of sixteen banks; another order of the bytes
// there, one line to each eight banks, changed neither the time (236.7 us at
// 8192 x 14336 both ways) nor the count of conflicts.
template <int LB> constexpr int line_bytes() { return LB + 8; }

// Codes and scale bytes of B blocks, N values of each in this lane; a block
// with a NaN or an Inf, in any lane, is put right in a step of its own
template <int FMT, int B, int N>
__device__ __forceinline__ void encode_blocks(const float (&v)[B][N], const uint32_t (&key)[B], uint32_t (&code)[B][N / 4],
                                              uint32_t (&byte)[B])
{
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < B; j++) {
        const BlockScale<FMT> b(key[j]);
#pragma unroll
        for (int i = 0; i < N / 4; i++)
            code[j][i] = encode4<FMT, true>(b, v[j][4 * i], v[j][4 * i + 1], v[j][4 * i + 2], v[j][4 * i + 3]);
        byte[j] = b.byte;
        most = max(most, key[j]);
    }
    if (__builtin_expect(most >= NONFINITE, 0)) {
#pragma unroll
        for (int j = 0; j < B; j++) {
            if (key[j] < NONFINITE) continue;
#pragma unroll
            for (int i = 0; i < N / 4; i++) code[j][i] = 0x7F7F7F7Fu;
            byte[j] = 0xFFu;
        }
    }
}

// Row codes of one tensor's 4 x 8 values per lane to `stage`, eight bytes from
// `at` in lines line0 .. line0 + 3, and the blocks' scale bytes
template <int FMT, int LB, int SPL>
__device__ __forceinline__ void stage_rows(const float (&v)[4][8], uint8_t* stage, uint8_t* scales, int line0, int at,
                                           int block, bool writes)
{
    uint32_t key[4], code[4][2], byte[4];
#pragma unroll
    for (int i = 0; i < 4; i++) key[i] = chunk_key(v[i]);
    row_block_max(key);
    encode_blocks<FMT>(v, key, code, byte);
#pragma unroll
    for (int i = 0; i < 4; i++) *(uint2*)(stage + (line0 + i) * line_bytes<LB>() + at) = make_uint2(code[i][0], code[i][1]);
    if (writes) {
#pragma unroll
        for (int i = 0; i < 4; i++) scales[(line0 + i) * SPL + block] = (uint8_t)byte[i];
    }
}

// Column codes: four bytes from `at` in lines line0 .. line0 + 7
template <int FMT, int LB, int SPL>
__device__ __forceinline__ void stage_columns(const float (&v)[4][8], uint8_t* stage, uint8_t* scales, int line0, int at,
                                              int block, bool writes)
{
    float w[8][4];
    uint32_t key[8], code[8][1], byte[8];
#pragma unroll
    for (int c = 0; c < 8; c++) {
#pragma unroll
        for (int r = 0; r < 4; r++) w[c][r] = v[r][c];
        key[c] = chunk_key(w[c]);
    }
    oct_max(key);
    encode_blocks<FMT>(w, key, code, byte);
#pragma unroll
    for (int c = 0; c < 8; c++) *(uint32_t*)(stage + (line0 + c) * line_bytes<LB>() + at) = code[c][0];
    if (writes) {
#pragma unroll
        for (int c = 0; c < 8; c++) scales[(line0 + c) * SPL + block] = (uint8_t)byte[c];
    }
}

// n scale bytes, 1 <= n <= N, staged at src, to base + offset
template <int N>
__device__ __forceinline__ void store_scale_bytes(uint8_t* base, uint32_t offset, const uint8_t* src, int n)
{
    if (N == 4 && n == 4) {
        lane_at<uint32_t>(base, offset)->v = *(const uint32_t*)src;
    } else {
#pragma unroll
        for (int i = 0; i < N; i++)
            if (i < n) lane_at<uint8_t>(base, offset + i)->v = src[i];
    }
}

// A thread's number, in a form that the compiler computes with where it is
// used: what a tile's stores derive from it is cheap, and would otherwise be
// held in registers all through the loop over tiles (and spilled).
__device__ __forceinline__ int thread_here()
{
    int t = (int)threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

// One staged tensor to its copy: `lines` of LB bytes, of which `bytes` are in
// the tensor, to stored rows q, q + stride, ...
template <int LB, int LINES, int NT>
__device__ __forceinline__ void store_lines(int tid, const uint8_t* stage, uint8_t* q, uint32_t stride, int lines, int bytes)
{
    constexpr int CH = LB / 16;
#pragma unroll
    for (int k = 0; k < (LINES * CH + NT - 1) / NT; k++) {
        const int id = tid + k * NT, line = id / CH, ch = id % CH;
        if (line < lines && ch * 16 < bytes) {
            const dwords2* p = (const dwords2*)(stage + line * line_bytes<LB>() + ch * 16);
            lane_at<dwords4>(q, (uint32_t)line * stride + ch * 16)->v = __builtin_shufflevector(p[0], p[1], 0, 1, 2, 3);
        }
    }
}

// Scale bytes of the rows of a window of tiles: WB bytes a line in LDS, of
// which n are in the tensor, from or to rows g, g + stride, ...  at any
// alignment; 16 bytes a thread.  The lines are 16 bytes more apart, so that
// lanes four lines apart use different banks.
constexpr int WINDOW = 16;              // tiles

template <int WB, int LINES, int NT, bool STORE>
__device__ __forceinline__ void move_row_scales(int tid, uint8_t* lds, uint8_t* g, uint32_t stride, int lines, int n)
{
    constexpr int CH = WB / 16;
#pragma unroll
    for (int k = 0; k < (LINES * CH + NT - 1) / NT; k++) {
        const int id = tid + k * NT, line = id / CH, at = id % CH * 16;
        const uint32_t to = (uint32_t)line * stride + at;
        uint8_t* l = lds + line * (WB + 16) + at;
        if (line < lines && at + 16 <= n) {
            if constexpr (STORE) lane_at<dwords4>(g, to)->v = *(const dwords4*)l;
            else *(dwords4*)l = lane_at<dwords4>(g, to)->v;
        } else if (line < lines) {
            for (int i = 0; at + i < n; i++) {
                if constexpr (STORE) lane_at<uint8_t>(g, to + i)->v = l[i];
                else l[i] = lane_at<uint8_t>(g, to + i)->v;
            }
        }
    }
}

struct DualTiles { uint32_t nx, ny; };

constexpr int WAIT_VMEM = 0x0F70;       // s_waitcnt vmcnt(0): expcnt and lgkmcnt at their largest

template <int SRC, int ACT, int FROM, int FMT, int WR, int WC>
__global__ __launch_bounds__(64 * WR * WC) void k_glu_bwd_dual(GluBwdJob a, DualTiles tiles)
{
    constexpr int TR = 32 * WR, TC = 64 * WC, NT = 64 * WR * WC, WB = WINDOW * 2 * WC, WS = WB + 16;
    constexpr bool TENSOR = FROM == FROM_TENSOR;
    static_assert(NT >= TC, "a thread per column for its scale bytes");
    constexpr bool EARLY = !(TENSOR && SRC == SRC_F32);    // two tiles' inputs fit the registers
    __shared__ __align__(16) uint8_t cols[3][TC * line_bytes<TR>()], rows[2][TR * line_bytes<TC>()];
    __shared__ __align__(16) uint8_t col_scales[3][TC * WR], row_scales[2][TR * WS], in_scales[2][TENSOR ? 16 : TR * WS];
    saturate_converters();
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6, band = wave % WR, part = wave / WR;
    const int m = lane & 7, k8 = lane >> 3, lr = band * 32 + m * 4, lc = part * 64 + k8 * 8;
    const uint32_t sr = (uint32_t)(a.rows / 32), sc = (uint32_t)(a.cols / 32);
    // this workgroup's run of tiles, along the rows of tiles
    const uint64_t all = (uint64_t)tiles.nx * tiles.ny;
    uint32_t tile = (uint32_t)(all * blockIdx.x / gridDim.x);
    const uint32_t end = (uint32_t)(all * (blockIdx.x + 1) / gridDim.x);
    uint32_t ty = tile / tiles.nx, tx = tile - ty * tiles.nx;
    constexpr uint32_t B = ElemT<SRC>::bytes;
    const DualAt place{(uint32_t)(lr * a.ld_dh + lc) * B, (uint32_t)(lr * a.ld_gate + lc) * B, (uint32_t)(lr * a.ld_up + lc) * B,
                       (uint32_t)(lr * a.cols + lc)};
    DualRaw<SRC, TENSOR> raw;
    // a lane past the tensor's end reads the tile's first places instead (its
    // whole blocks lie outside: rows and cols are multiples of 32)
    // `more` false: the run has ended.  The registers are cleared then, rather
    // than left: what they hold need not be kept through the iteration.
    enum { DH = 1, GATE = 2, UP = 4 };
    auto fetch = [&](bool more, uint32_t y, uint32_t x, int which) {
        if (!more) {
            const DualRaw<SRC, TENSOR> none{};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                if (which & DH) raw.d[i] = none.d[i];
                if (which & GATE) raw.g[i] = none.g[i];
                if (which & UP) raw.u[i] = none.u[i];
            }
            return;
        }
        const int64_t r = (int64_t)y * TR, c = (int64_t)x * TC;
        const bool in = r + lr < a.rows && c + lc < a.cols;
        const DualAt at = in ? place : DualAt{};
        if (which & DH) dual_load_dh(a, r, c, at, raw);
        if (which & GATE) dual_load_gate(a, r, c, at, raw);
        if (which & UP) dual_load_up(a, r, c, at, raw);
    };
    fetch(tile < end, ty, tx, DH | GATE | UP);
    __builtin_amdgcn_s_waitcnt(WAIT_VMEM);     // as inside the loop: no load is in flight where it begins again
    uint32_t first = tx, left = 0;             // the window's first tile column, its tiles still to do
    while (tile < end) {
        const int64_t r0 = (int64_t)ty * TR, c0 = (int64_t)tx * TC;
        const int nr = (int)min((int64_t)TR, a.rows - r0), nc = (int)min((int64_t)TC, a.cols - c0);
        if (left == 0) {
            first = tx;
            left = min(min((uint32_t)WINDOW, tiles.nx - tx), end - tile);
            if constexpr (!TENSOR) {
                const int tid = thread_here();
                const int64_t at = r0 * sc + c0 / 32;
                const int n = (int)min((int64_t)left * 2 * WC, (int64_t)sc - c0 / 32);
                move_row_scales<WB, TR, NT, false>(tid, in_scales[0], (uint8_t*)a.sg + at, sc, nr, n);
                move_row_scales<WB, TR, NT, false>(tid, in_scales[1], (uint8_t*)a.su + at, sc, nr, n);
                lds_barrier();
            }
        }
        const int block = ((int)(tx - first) * WC + part) * 2 + (k8 >> 2);     // the lane's block of the window's rows
        const DualRaw<SRC, TENSOR> now = raw;
        uint32_t y1 = ty, x1 = tx + 1;
        if (x1 == tiles.nx) x1 = 0, y1++;
        const bool more = tile + 1 < end;
        if constexpr (EARLY) fetch(more, y1, x1, DH | GATE | UP);
        float g[4][8], u[4][8], h[4][8];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if constexpr (!TENSOR) {
                decode8<FROM>(now.g[i], in_scales[0][(lr + i) * WS + block], g[i]);
                decode8<FROM>(now.u[i], in_scales[1][(lr + i) * WS + block], u[i]);
            } else {
#pragma unroll
                for (int c = 0; c < 8; c++) g[i][c] = chunk_value(now.g[i], c), u[i][c] = chunk_value(now.u[i], c);
            }
#pragma unroll
            for (int c = 0; c < 8; c++) {
                const float dh = chunk_value(now.d[i], c);
                float act, slope;
                gate<ACT, true>(g[i][c], act, slope);
                h[i][c] = act * u[i][c];
                g[i][c] = dh * u[i][c] * slope;
                u[i][c] = dh * act;
                // fp32 tensors fill the registers: one element at a time, its
                // results computed here and not where they are used (178
                // registers; with the order left to the compiler GELU and
                // GELU_TANH take 256 and keep more in scratch, 262 and 352 us
                // at 4096 x 14336 against 217 and 214)
                if constexpr (!EARLY) asm volatile("" : "+v"(g[i][c]), "+v"(u[i][c]), "+v"(h[i][c]));
            }
        }
        const bool row_writer = (k8 & 3) == 0, col_writer = m == 0;
        auto stage_h = [&] {
            if (!a.qh) return;
            if (a.h_fmt == E4M3) stage_columns<E4M3, TR, WR>(h, cols[2], col_scales[2], lc, lr, band, col_writer);
            else stage_columns<E5M2, TR, WR>(h, cols[2], col_scales[2], lc, lr, band, col_writer);
        };
        // fp32 tensors: each of the next tile's inputs is asked for when a
        // staged tensor has given its registers back
        if constexpr (!EARLY) {
            stage_h();
            fetch(more, y1, x1, DH);
        }
        stage_rows<FMT, TC, WS>(g, rows[0], row_scales[0], lr, lc, block, row_writer);
        if constexpr (EARLY) stage_rows<FMT, TC, WS>(u, rows[1], row_scales[1], lr, lc, block, row_writer);
        stage_columns<FMT, TR, WR>(g, cols[0], col_scales[0], lc, lr, band, col_writer);
        if constexpr (!EARLY) fetch(more, y1, x1, GATE | UP);
        if constexpr (!EARLY) stage_rows<FMT, TC, WS>(u, rows[1], row_scales[1], lr, lc, block, row_writer);
        stage_columns<FMT, TR, WR>(u, cols[1], col_scales[1], lc, lr, band, col_writer);
        if constexpr (EARLY) stage_h();
        // The next tile's inputs have landed, most of a tile's work after they
        // were asked for: waited for here, ahead of this tile's stores, since
        // loads and stores complete in one count and a wait for the loads
        // behind the stores would be one for the stores too.
        __builtin_amdgcn_s_waitcnt(WAIT_VMEM);
        lds_barrier();                         // the tile is staged
        const int tid = thread_here();
        // row copy: dgate in columns 0 .. cols - 1, dup after them
#pragma unroll
        for (int w = 0; w < 2; w++) {
            store_lines<TC, TR, NT>(tid, rows[w], a.q_row + (2 * r0 + w) * a.cols + c0, 2 * (uint32_t)a.cols, nr, nc);
            store_lines<TR, TC, NT>(tid, cols[w], a.q_col + (w * a.cols + c0) * a.rows + r0, (uint32_t)a.rows, nc, nr);
        }
        if (a.qh) store_lines<TR, TC, NT>(tid, cols[2], a.qh + c0 * a.rows + r0, (uint32_t)a.rows, nc, nr);
        if (const int line = tid; line < nc) {
            const int64_t at = c0 * sr + r0 / 32;
            store_scale_bytes<WR>(a.s_col + at, (uint32_t)line * sr, &col_scales[0][line * WR], nr / 32);
            store_scale_bytes<WR>(a.s_col + a.cols * sr + at, (uint32_t)line * sr, &col_scales[1][line * WR], nr / 32);
            if (a.qh) store_scale_bytes<WR>(a.sh + at, (uint32_t)line * sr, &col_scales[2][line * WR], nr / 32);
        }
        if (--left == 0) {
            const int64_t at = 2 * r0 * sc + (int64_t)first * 2 * WC;
            const int n = (int)min((int64_t)(tx - first + 1) * 2 * WC, (int64_t)sc - (int64_t)first * 2 * WC);
            move_row_scales<WB, TR, NT, true>(tid, row_scales[0], a.s_row + at, 2 * sc, nr, n);
            move_row_scales<WB, TR, NT, true>(tid, row_scales[1], a.s_row + at + sc, 2 * sc, nr, n);
        }
        lds_barrier();                         // the staged tile has been read
        tile++;
        ty = y1;
        tx = x1;
    }
}

template <int SRC, int ACT, int FROM, int FMT, int WR, int WC>
hipError_t run_dual(const GluBwdJob& j, DualTiles n, int cus, hipStream_t s)
{
    const int64_t all = (int64_t)n.nx * n.ny, most = (int64_t)cus * (8 / (WR * WC)), grid = all < most ? all : most;
    k_glu_bwd_dual<SRC, ACT, FROM, FMT, WR, WC><<<dim3((unsigned)grid), dim3(64 * WR * WC), 0, s>>>(j, n);
    return hipGetLastError();
}

// Tiles of 128 x 128, or, where no wave then has more than one of them, of 32
// x 64 (288 x 4096: 10.2 us against 13.8; 32 x 14336: 8.3 and 11.4; 288 x
// 14336 15.8 and 22.5; 1024 x 4096 16.1 and 16.7).  With more, the large ones:
// 1536 x 4096 25.1 us against 28.8, 2048 x 7168 40 and 60.
template <int SRC, int ACT, int FROM, int FMT>
hipError_t run_dual(const GluBwdJob& j, hipStream_t s)
{
    auto tiles = [&](int64_t r, int64_t c) { return DualTiles{(uint32_t)((j.cols + c - 1) / c), (uint32_t)((j.rows + r - 1) / r)}; };
    int dev = 0, cus = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return e;
    const DualTiles small = tiles(32, 64);
    if ((int64_t)small.nx * small.ny <= 8 * (int64_t)cus) return run_dual<SRC, ACT, FROM, FMT, 1, 1>(j, small, cus, s);
    return run_dual<SRC, ACT, FROM, FMT, 4, 2>(j, tiles(128, 128), cus, s);
}

// f(where gate and up come from)
template <class F>
hipError_t by_source(const GluBwdJob& j, F&& f)
{
    if (!j.qg) return f(std::integral_constant<int, FROM_TENSOR>());
    if (j.ckpt_fmt == E4M3) return f(std::integral_constant<int, FROM_E4M3>());
    return f(std::integral_constant<int, FROM_E5M2>());
}

}  // namespace

hipError_t launch_glu_fwd(const GluFwdJob& j, hipStream_t s)
{
    // (checkpoints and row copies of odd rows are refused: what the overlapping
    // chunks can write over is h)
    const bool in_place = j.h && (j.h == j.gate || j.h == j.up);
    return by_act(j.act, [&](auto A) {
        return by_mode(j.cols, in_place, [&](auto mode) {
            return j.src == SRC_F32 ? run_fwd<SRC_F32, A, mode>(j, s) : run_fwd<SRC_BF16, A, mode>(j, s);
        });
    });
}

hipError_t launch_glu_bwd(const GluBwdJob& j, hipStream_t s)
{
    bool in_place = false;
    for (const void* out : {(const void*)j.dgate, (const void*)j.dup, (const void*)j.h})
        in_place |= out && (out == j.dh || out == j.gate || out == j.up);
    return by_act(j.act, [&](auto A) {
        return by_source(j, [&](auto from) {
            auto run = [&](auto mode) {
                return j.src == SRC_F32 ? run_bwd<SRC_F32, A, from, mode>(j, s) : run_bwd<SRC_BF16, A, from, mode>(j, s);
            };
            if constexpr (from == FROM_TENSOR) return by_mode(j.cols, in_place, run);
            else return run(std::integral_constant<int, WHOLE>());
        });
    });
}

hipError_t launch_glu_bwd_dual(const GluBwdJob& j, hipStream_t s)
{
    return by_act(j.act, [&](auto A) {
        return by_source(j, [&](auto from) {
            auto fmt = [&](auto F) {
                return j.src == SRC_F32 ? run_dual<SRC_F32, A, from, F>(j, s) : run_dual<SRC_BF16, A, from, F>(j, s);
            };
            return j.fmt == E4M3 ? fmt(std::integral_constant<int, E4M3>()) : fmt(std::integral_constant<int, E5M2>());
        });
    });
}

}  // namespace mx
