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
// Kernels
//   k_glu_fwd, k_glu_bwd   one chunk of eight elements per thread, in order
//                    over rows and columns: each byte read and written once.
//   k_glu_bwd_dual   a wave takes 32 rows by 64 columns, a lane four rows by
//                    eight columns, so that row blocks end inside four lanes
//                    and column blocks inside eight; the gradients never
//                    leave registers before they are codes.
#include "act_device.h"
#include "mx_internal.h"

namespace mx {

namespace {

// n / d for 32-bit n and a divisor known to the host: d = 2^l' - ... by the
// round-up method (T. Granlund and P. Montgomery, "Division by Invariant
// Integers using Multiplication", PLDI 1994, figure 4.1)
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

// Places of a thread: VEC: eight consecutive elements of chunk `id`; else the
// elements id * 2048 + i * 256 + thread.  `units` counts chunks or elements.
template <bool VEC>
struct Place {
    uint32_t row[VEC ? 1 : 8], col[VEC ? 1 : 8];
    bool ok[VEC ? 1 : 8];
    __device__ __forceinline__ Place(const FastDiv& per_row, uint32_t units)
    {
#pragma unroll
        for (int i = 0; i < (VEC ? 1 : 8); i++) {
            uint32_t u = VEC ? blockIdx.x * 256u + threadIdx.x : blockIdx.x * 2048u + 256u * i + threadIdx.x;
            ok[i] = u < units;
            u = ok[i] ? u : 0u;
            row[i] = quotient(per_row, u);
            col[i] = (u - row[i] * per_row.d) * (VEC ? 8u : 1u);
        }
    }
    template <int SRC>
    __device__ __forceinline__ void load(const void* p, int64_t ld, float (&v)[8]) const
    {
        if constexpr (VEC) {
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
        if constexpr (VEC) {
            if (ok[0]) store_chunk<SRC>(p, row[0] * ld + col[0], make_chunk<SRC>(v));
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (ok[i]) store_elem<SRC>(p, row[i] * ld + col[i], v[i]);
        }
    }
    // place in a dense row copy (VEC)
    __device__ __forceinline__ int64_t dense(int64_t cols) const { return row[0] * cols + col[0]; }
};

template <int SRC, int ACT, bool VEC>
__global__ __launch_bounds__(256) void k_glu_fwd(GluFwdJob a, FastDiv per_row, uint32_t units)
{
    const Place<VEC> at(per_row, units);
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
    if constexpr (VEC) {
        const int64_t e = at.dense(a.cols);
        if (a.qh) encode_row_chunk(a.h_fmt, h, at.ok[0], e, a.qh, a.sh);
        if (a.qg) {
            encode_row_chunk(a.ckpt_fmt, g, at.ok[0], e, a.qg, a.sg);
            encode_row_chunk(a.ckpt_fmt, u, at.ok[0], e, a.qu, a.su);
        }
    }
}

template <int SRC, int ACT, bool CKPT, bool VEC>
__global__ __launch_bounds__(256) void k_glu_bwd(GluBwdJob a, FastDiv per_row, uint32_t units)
{
    const Place<VEC> at(per_row, units);
    float d[8], g[8], u[8], h[8];
    at.template load<SRC>(a.dh, a.ld_dh, d);
    if constexpr (CKPT) {
        const int64_t e = at.dense(a.cols);
        const uint2 cg = *(const uint2*)(a.qg + e), cu = *(const uint2*)(a.qu + e);
        const uint32_t bg = a.sg[e >> 5], bu = a.su[e >> 5];
        decode8(a.ckpt_fmt, cg, bg, g);
        decode8(a.ckpt_fmt, cu, bu, u);
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
template <bool VEC, class F>
hipError_t sliced(int64_t rows, int64_t cols, F&& f)
{
    const int64_t per_row = VEC ? cols / 8 : cols;
    const int64_t most = ((int64_t)1 << 31) / per_row < rows ? ((int64_t)1 << 31) / per_row : rows;
    const FastDiv d = fast_div((uint32_t)per_row);
    for (int64_t r = 0; r < rows; r += most) {
        const int64_t n = rows - r < most ? rows - r : most, units = n * per_row;
        const int64_t per_group = VEC ? 256 : 2048;
        f(r, n, d, (uint32_t)units, dim3((unsigned)((units + per_group - 1) / per_group)));
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class T>
void advance(T*& p, int64_t bytes)
{
    if (p) p = (T*)((uint8_t*)p + bytes);
}

template <int SRC, int ACT, bool VEC>
hipError_t run_fwd(const GluFwdJob& job, hipStream_t s)
{
    return sliced<VEC>(job.rows, job.cols, [&](int64_t r, int64_t n, FastDiv d, uint32_t units, dim3 grid) {
        GluFwdJob j = job;
        constexpr int64_t B = ElemT<SRC>::bytes;
        j.rows = n;
        advance(j.gate, r * j.ld_gate * B);
        advance(j.up, r * j.ld_up * B);
        advance(j.h, r * j.ld_h * (j.out_f32 ? 4 : 2));
        for (uint8_t** q : {&j.qh, &j.qg, &j.qu}) advance(*q, r * j.cols);
        for (uint8_t** q : {&j.sh, &j.sg, &j.su}) advance(*q, r * (j.cols / 32));
        k_glu_fwd<SRC, ACT, VEC><<<grid, dim3(256), 0, s>>>(j, d, units);
    });
}

template <int SRC, int ACT, bool CKPT, bool VEC>
hipError_t run_bwd(const GluBwdJob& job, hipStream_t s)
{
    return sliced<VEC>(job.rows, job.cols, [&](int64_t r, int64_t n, FastDiv d, uint32_t units, dim3 grid) {
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
        k_glu_bwd<SRC, ACT, CKPT, VEC><<<grid, dim3(256), 0, s>>>(j, d, units);
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
// k_glu_bwd_dual: workgroups of four waves take tiles of 128 rows by 64
// columns of h, wave w the rows 32 w .. 32 w + 31.  Lane 8 k + m holds rows
// 4 m .. 4 m + 3 and columns 8 k .. 8 k + 7: a column block is spread over the
// eight lanes 8 k .. 8 k + 7, a row block over four lanes 8 apart.  Row codes
// are stored at once, eight bytes a lane; a lane's column codes are four rows
// of a column, one dword, and go through LDS to leave as whole runs of 128
// bytes a column.
// ---------------------------------------------------------------------------
constexpr int DR = 128, DC = 64;

// LDS byte of (column, 16-byte chunk of its 128 rows): chunks are permuted by
// the column's lane, so that a wave's writes spread over the banks
__device__ __forceinline__ int dual_at(int col, int chunk) { return col * DR + ((chunk ^ (col >> 3)) << 4); }

// the largest key of the four lanes 8 apart that hold a row block's chunks:
// lanes l, l ^ 8 (in the 16-lane row) and l ^ 16
__device__ __forceinline__ uint32_t row_block_max(uint32_t k)
{
    k = max(k, dpp<0x128>(k));                 // rotate by 8 in a row of 16
    return max(k, (uint32_t)__shfl_xor((int)k, 16));
}

__device__ __forceinline__ uint32_t oct_max(uint32_t k)
{
    k = max(k, dpp<DPP_XOR1>(k));
    k = max(k, dpp<DPP_XOR2>(k));
    return max(k, dpp<DPP_HALF_MIRROR>(k));
}

// Column codes of one tensor's 4 x 8 values per lane into `stage` and scale
// bytes (packed by column, one byte per wave) into `scales`
template <int FMT>
__device__ __forceinline__ void stage_columns(const float (&v)[4][8], uint8_t* stage, uint8_t* scales, int wave, int lane)
{
    const int m = lane & 7, k = lane >> 3;
#pragma unroll
    for (int c = 0; c < 8; c++) {
        uint32_t key = 0;
#pragma unroll
        for (int r = 0; r < 4; r++) key = max(key, abs_key(v[r][c]));
        key = oct_max(key);
        const int e = block_exponent<FMT>(key);
        float y[4];
#pragma unroll
        for (int r = 0; r < 4; r++) y[r] = clamp_fmax<FMT>(scale_by(v[r][c], e));
        const bool bad = key >= 0x7F800000u;
        const int col = 8 * k + c;
        *(uint32_t*)(stage + dual_at(col, wave * 2 + (m >> 2)) + (m & 3) * 4) =
            bad ? 0x7F7F7F7Fu : cvt4_fp8<FMT>(y[0], y[1], y[2], y[3]);
        if (m == c) scales[col * 4 + wave] = bad ? 0xFF : (uint8_t)(e + 127);
    }
}

__device__ __forceinline__ void stage_columns(int fmt, const float (&v)[4][8], uint8_t* stage, uint8_t* scales, int wave,
                                              int lane)
{
    if (fmt == E4M3) stage_columns<E4M3>(v, stage, scales, wave, lane);
    else stage_columns<E5M2>(v, stage, scales, wave, lane);
}

// the runs of one staged tensor: nc columns of nr rows to the column copy
// whose stored row 0 is the tile's first column
__device__ __forceinline__ void store_columns(const uint8_t* stage, const uint8_t* scales, uint8_t* q, uint8_t* s,
                                              int64_t rows, int64_t r0, int nr, int nc)
{
    for (int id = (int)threadIdx.x; id < DC * (DR / 16); id += 256) {
        const int col = id / (DR / 16), ch = id % (DR / 16);
        if (col < nc && ch * 16 < nr) *(uint4*)(q + col * rows + r0 + ch * 16) = *(const uint4*)(stage + dual_at(col, ch));
    }
    const int col = (int)threadIdx.x / 4, blk = (int)threadIdx.x % 4;
    if (col < nc && blk * 32 < nr) s[col * (rows / 32) + r0 / 32 + blk] = scales[col * 4 + blk];
}

template <int SRC, int ACT, bool CKPT>
__global__ __launch_bounds__(256) void k_glu_bwd_dual(GluBwdJob a, uint32_t col_tiles)
{
    __shared__ __align__(16) uint8_t stage[3][DC * DR];
    __shared__ uint8_t scales[3][DC * 4];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int64_t r0 = (int64_t)(blockIdx.x / col_tiles) * DR, c0 = (int64_t)(blockIdx.x % col_tiles) * DC;
    const int nr = (int)min((int64_t)DR, a.rows - r0), nc = (int)min((int64_t)DC, a.cols - c0);
    const int lr = wave * 32 + (lane & 7) * 4, lc = (lane >> 3) * 8;
    const bool ok = lr < nr && lc < nc;        // the same for the lanes of a block: rows and columns end at multiples of 32
    float g[4][8], u[4][8], h[4][8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int64_t row = r0 + (ok ? lr : 0) + i, col = c0 + (ok ? lc : 0);
        const Chunk<SRC> d = load_chunk<SRC>(a.dh, row * a.ld_dh + col);
        if constexpr (CKPT) {
            const int64_t e = row * a.cols + col;
            decode8(a.ckpt_fmt, *(const uint2*)(a.qg + e), a.sg[e >> 5], g[i]);
            decode8(a.ckpt_fmt, *(const uint2*)(a.qu + e), a.su[e >> 5], u[i]);
        } else {
            const Chunk<SRC> cg = load_chunk<SRC>(a.gate, row * a.ld_gate + col);
            const Chunk<SRC> cu = load_chunk<SRC>(a.up, row * a.ld_up + col);
#pragma unroll
            for (int k = 0; k < 8; k++) g[i][k] = chunk_value<SRC>(cg, k), u[i][k] = chunk_value<SRC>(cu, k);
        }
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const float dh = chunk_value<SRC>(d, k);
            float act, slope;
            gate<ACT, true>(g[i][k], act, slope);
            h[i][k] = act * u[i][k];
            g[i][k] = dh * u[i][k] * slope;
            u[i][k] = dh * act;
        }
        // row copies: dgate in columns 0 .. cols - 1, dup after them
        const Codes8 cg = encode8(a.fmt, g[i], row_block_max(chunk_key(g[i])));
        const Codes8 cu = encode8(a.fmt, u[i], row_block_max(chunk_key(u[i])));
        if (ok) {
            const int64_t e = row * 2 * a.cols + col;
            *(uint2*)(a.q_row + e) = make_uint2(cg.lo, cg.hi);
            *(uint2*)(a.q_row + e + a.cols) = make_uint2(cu.lo, cu.hi);
            if ((lane >> 3 & 3) == 0) {
                a.s_row[e >> 5] = (uint8_t)cg.scale;
                a.s_row[(e + a.cols) >> 5] = (uint8_t)cu.scale;
            }
        }
    }
    stage_columns(a.fmt, g, stage[0], scales[0], wave, lane);
    stage_columns(a.fmt, u, stage[1], scales[1], wave, lane);
    if (a.qh) stage_columns(a.h_fmt, h, stage[2], scales[2], wave, lane);
    __syncthreads();
    const int64_t sr = a.rows / 32;
    store_columns(stage[0], scales[0], a.q_col + c0 * a.rows, a.s_col + c0 * sr, a.rows, r0, nr, nc);
    store_columns(stage[1], scales[1], a.q_col + (a.cols + c0) * a.rows, a.s_col + (a.cols + c0) * sr, a.rows, r0, nr, nc);
    if (a.qh) store_columns(stage[2], scales[2], a.qh + c0 * a.rows, a.sh + c0 * sr, a.rows, r0, nr, nc);
}

}  // namespace

hipError_t launch_glu_fwd(const GluFwdJob& j, hipStream_t s)
{
    const bool vec = j.cols % 8 == 0;
    return by_act(j.act, [&](auto A) {
        if (j.src == SRC_F32) return vec ? run_fwd<SRC_F32, A, true>(j, s) : run_fwd<SRC_F32, A, false>(j, s);
        return vec ? run_fwd<SRC_BF16, A, true>(j, s) : run_fwd<SRC_BF16, A, false>(j, s);
    });
}

hipError_t launch_glu_bwd(const GluBwdJob& j, hipStream_t s)
{
    const bool vec = j.cols % 8 == 0;
    return by_act(j.act, [&](auto A) {
        if (j.src == SRC_F32) {
            if (j.qg) return run_bwd<SRC_F32, A, true, true>(j, s);
            return vec ? run_bwd<SRC_F32, A, false, true>(j, s) : run_bwd<SRC_F32, A, false, false>(j, s);
        }
        if (j.qg) return run_bwd<SRC_BF16, A, true, true>(j, s);
        return vec ? run_bwd<SRC_BF16, A, false, true>(j, s) : run_bwd<SRC_BF16, A, false, false>(j, s);
    });
}

hipError_t launch_glu_bwd_dual(const GluBwdJob& j, hipStream_t s)
{
    const int64_t ct = (j.cols + DC - 1) / DC, rt = (j.rows + DR - 1) / DR;
    return by_act(j.act, [&](auto A) {
        const dim3 grid((unsigned)(ct * rt)), block(256);
        const uint32_t c = (uint32_t)ct;
        if (j.src == SRC_F32) {
            if (j.qg) k_glu_bwd_dual<SRC_F32, A, true><<<grid, block, 0, s>>>(j, c);
            else k_glu_bwd_dual<SRC_F32, A, false><<<grid, block, 0, s>>>(j, c);
        } else {
            if (j.qg) k_glu_bwd_dual<SRC_BF16, A, true><<<grid, block, 0, s>>>(j, c);
            else k_glu_bwd_dual<SRC_BF16, A, false><<<grid, block, 0, s>>>(j, c);
        }
        return hipGetLastError();
    });
}

}  // namespace mx
