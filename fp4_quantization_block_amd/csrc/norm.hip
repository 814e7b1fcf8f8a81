// norm.hip -- layer norm and RMS norm, forward and backward, for gfx950.
//
//   forward   s = x, or x + residual rounded to the source type;
//             m = mean(s) (0 for the RMS norm),
//             r = 1 / sqrt(mean((s - m)^2) + eps),  y = (s - m) r w + b
//   backward  h = (s - m) r,  g = dy w,
//             dx = r (g - mean(g) - h mean(g h)) + dsum  (no mean(g) for RMS),
//             dw = sum over rows of dy h,  db = sum over rows of dy
// with s in the backward read from the tensor or from its 8-bit checkpoint
// (an MX row copy, [COAT, "FP8啟用"]).  All arithmetic is fp32; the variance
// is taken of the centred values, in a second pass over registers, so a large
// mean costs no digits.
//
// Sources:
//   [COAT] write-up of "COAT: Compressing Optimizer States and Activation for
//          memory efficient FP8 Training"
//
// Kernels
//   k_norm_fwd       T threads hold a row in registers (N chunks of eight
//                    elements each): read once, written once.
//   k_norm_fwd_wide  rows beyond 16384: a workgroup walks the row, and reads
//                    it again for each of the statistics and the output.
//   k_norm_bwd       T threads hold a row; a workgroup walks rows and keeps
//                    its share of the dw and db sums in registers, written
//                    as one row of partial sums each at the end.
//   k_norm_bwd_wide / k_norm_cols   the same in two kernels for rows beyond
//                    16384: dx by rows, then partial sums by column strips.
//   k_norm_colsum    adds the partial rows up, in a fixed order.
#include "act_device.h"
#include "mx_internal.h"

namespace mx {

namespace {

// A row spread over T lanes: element i of lane t's chunk j
template <bool VEC, int T>
__device__ __forceinline__ int64_t col_of(int64_t j, int t, int i)
{
    return VEC ? (j * T + t) * 8 + i : (j * 8 + i) * T + t;
}

// chunk j of a row as fp32.  Places past the row read the row's first
// elements (VEC) or element (else): the caller leaves them out.
template <int SRC, bool VEC, int T>
__device__ __forceinline__ void load_row(const void* row, int64_t j, int t, int64_t cols, float (&v)[8])
{
    if constexpr (VEC) {
        const int64_t c = col_of<VEC, T>(j, t, 0);
        const Chunk<SRC> w = load_chunk<SRC>(row, c < cols ? c : 0);
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = chunk_value<SRC>(w, i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int64_t c = col_of<VEC, T>(j, t, i);
            v[i] = load_elem<SRC>(row, c < cols ? c : 0);
        }
    }
}

template <int SRC, bool VEC, int T>
__device__ __forceinline__ void store_row(void* row, int64_t j, int t, int64_t cols, const float (&v)[8])
{
    if constexpr (VEC) {
        const int64_t c = col_of<VEC, T>(j, t, 0);
        if (c < cols) store_chunk<SRC>(row, c, make_chunk<SRC>(v));
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int64_t c = col_of<VEC, T>(j, t, i);
            if (c < cols) store_elem<SRC>(row, c, v[i]);
        }
    }
}

template <bool VEC, int T>
__device__ __forceinline__ void load_param(const void* p, int f32, int64_t j, int t, int64_t cols, float (&v)[8])
{
    if (f32) load_row<SRC_F32, VEC, T>(p, j, t, cols, v);
    else load_row<SRC_BF16, VEC, T>(p, j, t, cols, v);
}

// the sum of f(i) over the chunk's elements that are in the row
template <bool VEC, int T, class F>
__device__ __forceinline__ float chunk_sum(int64_t j, int t, int64_t cols, F&& f)
{
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float x = f(i);
        s += VEC || col_of<VEC, T>(j, t, i) < cols ? x : 0.0f;
    }
    return !VEC || col_of<VEC, T>(j, t, 0) < cols ? s : 0.0f;
}

template <int SRC>
__device__ __forceinline__ const void* row_of(const void* p, int64_t row, int64_t ld)
{
    return (const uint8_t*)p + row * ld * ElemT<SRC>::bytes;
}

// y of one chunk, and its outputs
template <int SRC, bool VEC, int T>
__device__ __forceinline__ void finish_chunk(const NormFwdJob& a, int64_t row, int64_t j, int t, const float (&s)[8],
                                             float mean, float rstd)
{
    if (!a.y && !a.qy) return;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; i++) y[i] = (s[i] - mean) * rstd;
    if (a.weight) {
        float w[8];
        load_param<VEC, T>(a.weight, a.param_f32, j, t, a.cols, w);
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] *= w[i];
    }
    if (a.bias) {
        float b[8];
        load_param<VEC, T>(a.bias, a.param_f32, j, t, a.cols, b);
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] += b[i];
    }
    if (a.y) {
        if (a.out_f32) store_row<SRC_F32, VEC, T>((float*)a.y + row * a.ld_y, j, t, a.cols, y);
        else store_row<SRC_BF16, VEC, T>((uint16_t*)a.y + row * a.ld_y, j, t, a.cols, y);
    }
    if constexpr (VEC) {
        const int64_t c = col_of<VEC, T>(j, t, 0);
        if (a.qy) encode_row_chunk(a.y_fmt, y, c < a.cols, row * a.cols + c, a.qy, a.sy);
    }
}

// s = x (+ residual) of one chunk, with the sum and the checkpoint written
template <int SRC, bool VEC, int T>
__device__ __forceinline__ void residual_and_checkpoint(const NormFwdJob& a, int64_t row, int64_t j, int t,
                                                        float (&s)[8])
{
    if (a.residual) {
        float r[8];
        load_row<SRC, VEC, T>(row_of<SRC>(a.residual, row, a.ld_res), j, t, a.cols, r);
#pragma unroll
        for (int i = 0; i < 8; i++) s[i] = rounded<SRC>(s[i] + r[i]);
        store_row<SRC, VEC, T>((void*)row_of<SRC>(a.sum, row, a.ld_sum), j, t, a.cols, s);
    }
    if constexpr (VEC) {
        const int64_t c = col_of<VEC, T>(j, t, 0);
        if (a.qx) encode_row_chunk(a.ckpt_fmt, s, c < a.cols, row * a.cols + c, a.qx, a.sx);
    }
}

__device__ __forceinline__ float inv_sqrt(float v) { return 1.0f / __builtin_sqrtf(v); }

template <int SRC, bool VEC, int T, int N>
__global__ __launch_bounds__(T < 256 ? 256 : T) void k_norm_fwd(NormFwdJob a)
{
    constexpr int RPB = T < 256 ? 256 / T : 1;
    __shared__ float red[2][T < 256 ? 1 : T / 64];
    const int t = (int)threadIdx.x % T;
    const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / T;
    if (row >= a.rows) return;               // whole waves, and only where no barrier follows (T = 64)
    float s[N][8];
#pragma unroll
    for (int j = 0; j < N; j++) load_row<SRC, VEC, T>(row_of<SRC>(a.x, row, a.ld_x), j, t, a.cols, s[j]);
#pragma unroll
    for (int j = 0; j < N; j++) residual_and_checkpoint<SRC, VEC, T>(a, row, j, t, s[j]);
    const float n = (float)a.cols;
    float mean = 0.0f;
    if (a.layer) {
        float p = 0.0f;
#pragma unroll
        for (int j = 0; j < N; j++) p += chunk_sum<VEC, T>(j, t, a.cols, [&](int i) { return s[j][i]; });
        mean = group_sum<T>(p, red[0]) / n;
    }
    float p = 0.0f;
#pragma unroll
    for (int j = 0; j < N; j++)
        p += chunk_sum<VEC, T>(j, t, a.cols, [&](int i) { const float c = s[j][i] - mean; return c * c; });
    const float rstd = inv_sqrt(group_sum<T>(p, red[1]) / n + a.eps);
    if (t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int j = 0; j < N; j++) finish_chunk<SRC, VEC, T>(a, row, j, t, s[j], mean, rstd);
}

template <int SRC, bool VEC>
__global__ __launch_bounds__(1024) void k_norm_fwd_wide(NormFwdJob a)
{
    constexpr int T = 1024;
    __shared__ float red[2][T / 64];
    const int t = (int)threadIdx.x;
    const int64_t row = blockIdx.x, steps = (a.cols + T * 8 - 1) / (T * 8);
    // after the first pass s is in the sum, written by the same thread
    const void* xr = row_of<SRC>(a.x, row, a.ld_x);
    const void* sr = a.residual ? row_of<SRC>(a.sum, row, a.ld_sum) : xr;
    float p = 0.0f;
    for (int64_t j = 0; j < steps; j++) {
        float s[8];
        load_row<SRC, VEC, T>(xr, j, t, a.cols, s);
        residual_and_checkpoint<SRC, VEC, T>(a, row, j, t, s);
        p += chunk_sum<VEC, T>(j, t, a.cols, [&](int i) { return a.layer ? s[i] : s[i] * s[i]; });
    }
    const float n = (float)a.cols;
    p = group_sum<T>(p, red[0]) / n;
    float mean = 0.0f, var = p;
    if (a.layer) {
        mean = p;
        p = 0.0f;
        for (int64_t j = 0; j < steps; j++) {
            float s[8];
            load_row<SRC, VEC, T>(sr, j, t, a.cols, s);
            p += chunk_sum<VEC, T>(j, t, a.cols, [&](int i) { const float c = s[i] - mean; return c * c; });
        }
        var = group_sum<T>(p, red[1]) / n;
    }
    const float rstd = inv_sqrt(var + a.eps);
    if (t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
    for (int64_t j = 0; j < steps; j++) {
        float s[8];
        load_row<SRC, VEC, T>(sr, j, t, a.cols, s);
        finish_chunk<SRC, VEC, T>(a, row, j, t, s, mean, rstd);
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// chunk j of the normalised input (s - m) r, from the tensor or the checkpoint
template <int SRC, int FROM, bool VEC, int T>
__device__ __forceinline__ void load_unit(const NormBwdJob& a, int64_t row, int64_t j, int t, float mean, float rstd,
                                          float (&h)[8])
{
    if constexpr (FROM != FROM_TENSOR) {
        const int64_t c = col_of<VEC, T>(j, t, 0), e = row * a.cols + (c < a.cols ? c : 0);
        decode8<FROM>(*(const uint2*)(a.qx + e), a.sx[e >> 5], h);
    } else {
        load_row<SRC, VEC, T>(row_of<SRC>(a.x, row, a.ld_x), j, t, a.cols, h);
    }
#pragma unroll
    for (int i = 0; i < 8; i++) h[i] = (h[i] - mean) * rstd;
}

// dx of one chunk from g, h and the two means
template <int SRC, bool VEC, int T>
__device__ __forceinline__ void store_dx(const NormBwdJob& a, int64_t row, int64_t j, int t, const float (&g)[8],
                                         const float (&h)[8], float rstd, float mg, float mgh)
{
    float d[8];
#pragma unroll
    for (int i = 0; i < 8; i++) d[i] = rstd * (g[i] - mg - h[i] * mgh);
    if (a.dsum) {
        float r[8];
        load_row<SRC, VEC, T>(row_of<SRC>(a.dsum, row, a.ld_dsum), j, t, a.cols, r);
#pragma unroll
        for (int i = 0; i < 8; i++) d[i] += r[i];
    }
    store_row<SRC, VEC, T>((void*)row_of<SRC>(a.dx, row, a.ld_dx), j, t, a.cols, d);
}

template <int SRC, int FROM, bool VEC, int T, int N>
__global__ __launch_bounds__(T < 256 ? 256 : T) void k_norm_bwd(NormBwdJob a)
{
    constexpr int RPB = T < 256 ? 256 / T : 1;
    __shared__ float red[2][2][T < 256 ? 1 : T / 64];
    const int t = (int)threadIdx.x % T;
    const int64_t part = (int64_t)blockIdx.x * RPB + threadIdx.x / T, parts = (int64_t)gridDim.x * RPB;
    float w[N][8], dw[N][8], db[N][8];
#pragma unroll
    for (int j = 0; j < N; j++) {
#pragma unroll
        for (int i = 0; i < 8; i++) w[j][i] = 1.0f, dw[j][i] = 0.0f, db[j][i] = 0.0f;
        if (a.weight) load_param<VEC, T>(a.weight, a.param_f32, j, t, a.cols, w[j]);
    }
    const float n = (float)a.cols;
    // the two sums alternate between two halves of `red`: a wave writes one
    // half again only after the barrier of the row between, which every wave
    // reaches after reading it
    int half = 0;
    for (int64_t row = part; row < a.rows; row += parts, half ^= 1) {
        const float mean = a.layer ? a.mean[row] : 0.0f, rstd = a.rstd[row];
        float g[N][8], h[N][8], pg = 0.0f, pgh = 0.0f;
#pragma unroll
        for (int j = 0; j < N; j++) load_row<SRC, VEC, T>(row_of<SRC>(a.dy, row, a.ld_dy), j, t, a.cols, g[j]);
#pragma unroll
        for (int j = 0; j < N; j++) load_unit<SRC, FROM, VEC, T>(a, row, j, t, mean, rstd, h[j]);
#pragma unroll
        for (int j = 0; j < N; j++) {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                dw[j][i] += g[j][i] * h[j][i];
                db[j][i] += g[j][i];
                g[j][i] *= w[j][i];
            }
            pgh += chunk_sum<VEC, T>(j, t, a.cols, [&](int i) { return g[j][i] * h[j][i]; });
            pg += chunk_sum<VEC, T>(j, t, a.cols, [&](int i) { return g[j][i]; });
        }
        const float mgh = group_sum<T>(pgh, red[half][0]) / n;
        const float mg = a.layer ? group_sum<T>(pg, red[half][1]) / n : 0.0f;
#pragma unroll
        for (int j = 0; j < N; j++) store_dx<SRC, VEC, T>(a, row, j, t, g[j], h[j], rstd, mg, mgh);
    }
#pragma unroll
    for (int j = 0; j < N; j++) {
        if (a.dweight) store_row<SRC_F32, VEC, T>(a.work + part * a.cols, j, t, a.cols, dw[j]);
        if (a.dbias) store_row<SRC_F32, VEC, T>(a.work + ((a.dweight ? parts : 0) + part) * a.cols, j, t, a.cols, db[j]);
    }
}

template <int SRC, int FROM, bool VEC>
__global__ __launch_bounds__(1024) void k_norm_bwd_wide(NormBwdJob a)
{
    constexpr int T = 1024;
    __shared__ float red[2][T / 64];
    const int t = (int)threadIdx.x;
    const int64_t row = blockIdx.x, steps = (a.cols + T * 8 - 1) / (T * 8);
    const float mean = a.layer ? a.mean[row] : 0.0f, rstd = a.rstd[row], n = (float)a.cols;
    const void* dyr = row_of<SRC>(a.dy, row, a.ld_dy);
    float pg = 0.0f, pgh = 0.0f;
    auto gradient = [&](int64_t j, float (&g)[8]) {
        load_row<SRC, VEC, T>(dyr, j, t, a.cols, g);
        if (a.weight) {
            float w[8];
            load_param<VEC, T>(a.weight, a.param_f32, j, t, a.cols, w);
#pragma unroll
            for (int i = 0; i < 8; i++) g[i] *= w[i];
        }
    };
    for (int64_t j = 0; j < steps; j++) {
        float g[8], h[8];
        gradient(j, g);
        load_unit<SRC, FROM, VEC, T>(a, row, j, t, mean, rstd, h);
        pgh += chunk_sum<VEC, T>(j, t, a.cols, [&](int i) { return g[i] * h[i]; });
        pg += chunk_sum<VEC, T>(j, t, a.cols, [&](int i) { return g[i]; });
    }
    const float mgh = group_sum<T>(pgh, red[0]) / n;
    const float mg = a.layer ? group_sum<T>(pg, red[1]) / n : 0.0f;
    for (int64_t j = 0; j < steps; j++) {
        float g[8], h[8];
        gradient(j, g);
        load_unit<SRC, FROM, VEC, T>(a, row, j, t, mean, rstd, h);
        store_dx<SRC, VEC, T>(a, row, j, t, g, h, rstd, mg, mgh);
    }
}

// Partial sums of dw and db over the rows of one part, a strip of 512
// columns per wave: grid (strips / 4, parts)
template <int SRC, int FROM, bool VEC>
__global__ __launch_bounds__(256) void k_norm_cols(NormBwdJob a, int64_t rows_per_part)
{
    constexpr int T = 64;
    const int t = (int)threadIdx.x & 63;
    const int64_t j = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), part = blockIdx.y, parts = gridDim.y;
    if (j * T * 8 >= a.cols) return;
    float dw[8] = {}, db[8] = {};
    const int64_t end = min((part + 1) * rows_per_part, a.rows);
    for (int64_t row = part * rows_per_part; row < end; row++) {
        float dy[8], h[8];
        load_row<SRC, VEC, T>(row_of<SRC>(a.dy, row, a.ld_dy), j, t, a.cols, dy);
        load_unit<SRC, FROM, VEC, T>(a, row, j, t, a.layer ? a.mean[row] : 0.0f, a.rstd[row], h);
#pragma unroll
        for (int i = 0; i < 8; i++) dw[i] += dy[i] * h[i], db[i] += dy[i];
    }
    if (a.dweight) store_row<SRC_F32, VEC, T>(a.work + part * a.cols, j, t, a.cols, dw);
    if (a.dbias) store_row<SRC_F32, VEC, T>(a.work + ((a.dweight ? parts : 0) + part) * a.cols, j, t, a.cols, db);
}

// dw (blockIdx.y 0) and db (1, or 0 without dw): 32 columns per workgroup, 32
// threads down the partial rows of each column, added by halves at the end
__global__ __launch_bounds__(1024) void k_norm_colsum(const float* work, int64_t parts, int64_t cols, float* out0,
                                                      float* out1)
{
    __shared__ float sum[32][33];
    const int x = (int)threadIdx.x & 31, y = (int)threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + x;
    const float* p = work + (int64_t)blockIdx.y * parts * cols;
    float s = 0.0f;
    if (c < cols)
        for (int64_t r = y; r < parts; r += 32) s += p[r * cols + c];
    sum[y][x] = s;
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
        __syncthreads();
        if (y < m) sum[y][x] += sum[y + m][x];
    }
    if (y == 0 && c < cols) (blockIdx.y ? out1 : out0)[c] = sum[0][x];
}

// Threads and chunks per row: the fewest threads that hold it in registers.
template <class F>
hipError_t by_width(int64_t cols, F&& f)
{
    if (cols <= 512) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
    if (cols <= 2048) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 1>());
    if (cols <= 4096) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 2>());
    if (cols <= 8192) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 2>());
    return f(std::integral_constant<int, 1024>(), std::integral_constant<int, 2>());
}

constexpr int64_t WIDE = 16384;        // rows beyond this do not stay in registers

template <int SRC, bool VEC>
hipError_t launch_fwd(const NormFwdJob& j, hipStream_t s)
{
    if (j.cols > WIDE) {
        k_norm_fwd_wide<SRC, VEC><<<dim3((unsigned)j.rows), dim3(1024), 0, s>>>(j);
        return hipGetLastError();
    }
    return by_width(j.cols, [&](auto T, auto N) {
        constexpr int B = T < 256 ? 256 : (int)T, RPB = B / T;
        k_norm_fwd<SRC, VEC, T, N><<<dim3((unsigned)((j.rows + RPB - 1) / RPB)), dim3(B), 0, s>>>(j);
        return hipGetLastError();
    });
}

// workgroups of the backward kernel, and the rows each of its workgroups takes at a time
int64_t bwd_groups(int64_t rows, int64_t cols)
{
    const int64_t rpb = cols <= 512 ? 4 : 1, want = (rows + rpb - 1) / rpb;
    return want < 512 ? want : 512;
}

int64_t wide_parts(int64_t rows) { return rows < 64 ? rows : 64; }

template <int SRC, int FROM, bool VEC>
hipError_t launch_bwd(const NormBwdJob& j, hipStream_t s)
{
    int64_t parts = 0;
    if (j.cols > WIDE) {
        k_norm_bwd_wide<SRC, FROM, VEC><<<dim3((unsigned)j.rows), dim3(1024), 0, s>>>(j);
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
        if (j.dweight || j.dbias) {
            parts = wide_parts(j.rows);
            const int64_t per = (j.rows + parts - 1) / parts;
            parts = (j.rows + per - 1) / per;
            k_norm_cols<SRC, FROM, VEC><<<dim3((unsigned)((j.cols + 2047) / 2048), (unsigned)parts), dim3(256), 0, s>>>(j, per);
        }
    } else {
        const int64_t groups = bwd_groups(j.rows, j.cols);
        const hipError_t e = by_width(j.cols, [&](auto T, auto N) {
            constexpr int B = T < 256 ? 256 : (int)T;
            k_norm_bwd<SRC, FROM, VEC, T, N><<<dim3((unsigned)groups), dim3(B), 0, s>>>(j);
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
        parts = groups * (j.cols <= 512 ? 4 : 1);
    }
    if (j.dweight || j.dbias) {
        const bool both = j.dweight && j.dbias;
        k_norm_colsum<<<dim3((unsigned)((j.cols + 31) / 32), both ? 2u : 1u), dim3(1024), 0, s>>>(
            j.work, parts, j.cols, j.dweight ? j.dweight : j.dbias, j.dbias);
    }
    return hipGetLastError();
}

}  // namespace

int64_t norm_bwd_partials(int64_t rows, int64_t cols)
{
    if (cols > WIDE) return wide_parts(rows);
    return bwd_groups(rows, cols) * (cols <= 512 ? 4 : 1);
}

hipError_t launch_norm_fwd(const NormFwdJob& j, hipStream_t s)
{
    const bool vec = j.cols % 8 == 0;
    if (j.src == SRC_F32) return vec ? launch_fwd<SRC_F32, true>(j, s) : launch_fwd<SRC_F32, false>(j, s);
    return vec ? launch_fwd<SRC_BF16, true>(j, s) : launch_fwd<SRC_BF16, false>(j, s);
}

hipError_t launch_norm_bwd(const NormBwdJob& j, hipStream_t s)
{
    auto run = [&](auto src) {
        if (j.qx) return j.ckpt_fmt == E4M3 ? launch_bwd<src, FROM_E4M3, true>(j, s) : launch_bwd<src, FROM_E5M2, true>(j, s);
        return j.cols % 8 == 0 ? launch_bwd<src, FROM_TENSOR, true>(j, s) : launch_bwd<src, FROM_TENSOR, false>(j, s);
    };
    return j.src == SRC_F32 ? run(std::integral_constant<int, SRC_F32>()) : run(std::integral_constant<int, SRC_BF16>());
}

}  // namespace mx
