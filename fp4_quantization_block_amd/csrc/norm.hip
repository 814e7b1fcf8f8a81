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
// What is rounded: the sum to the source type, since it is the residual stream
// that the next block reads, and what is normalised is what was stored; y, dx
// and the codes once each, from fp32.  Statistics and the parameters'
// gradients stay fp32.
//
// All of it is bound by memory: a few operations an element, so that the one
// aim is to read and write each byte once.
//
// Kernels (times at 8192 x 4096 bf16 on one MI355X, where a 1 GiB copy runs at
// 5.1 TB/s)
//   k_norm_fwd       T threads hold a row in registers (N chunks of eight
//                    elements each): read once, written once.  RMS norm with
//                    residual, sum, y and checkpoint, 303 MB: 53 us, 5.7 TB/s
//                    (counters: 134 MB read, 169 MB written).
//   k_norm_fwd_wide  rows beyond 16384: a workgroup walks the row, and reads
//                    it again for each of the statistics and the output.
//   k_norm_bwd       T threads hold a row; a workgroup walks rows, the next
//                    one's inputs loaded ahead, and keeps its share of the dw
//                    and db sums in registers, written as one row of partial
//                    sums each at the end.  From the checkpoint, with dsum,
//                    236 MB: 40.5 us.
//   k_norm_bwd_wide / k_norm_cols   the same in two kernels for rows beyond
//                    16384: dx by rows, then partial sums by column strips.
//   k_norm_colsum    adds the partial rows up, in a fixed order: 4.7 us for
//                    256 rows of 4096, most of it the launch and one pass of
//                    latency (both backward kernels 5.2 TB/s).
#include "act_device.h"
#include "mx_internal.h"

namespace mx {

namespace {

// How a row is spread over T lanes (chunk j of lane t):
//   WHOLE    eight consecutive elements; the row is a multiple of eight
//   OVERLAP  the same for any row of at least eight: the last chunk is the
//            row's last eight elements, so that some of them are held twice.
//            They come out the same twice, and are left out of one lane's
//            part of a sum.
//   STRIDED  elements t, t + T, ... t + 7 T of a run of 8 T: any row, and
//            no element twice (an output may be written over an input)
enum : int { WHOLE, OVERLAP, STRIDED };

template <int MODE, int T>
struct Cols {
    int64_t c0, c;          // where chunk j would begin, and where it is read
    bool in;                // whether any of it is in the row (else it reads the row's beginning)
    int64_t cols;
    __device__ __forceinline__ Cols(int64_t j, int t, int64_t n) : cols(n)
    {
        c0 = MODE == STRIDED ? j * 8 * T + t : (j * T + t) * 8;
        in = c0 < n;
        c = !in ? 0 : MODE == OVERLAP && c0 + 8 > n ? n - 8 : c0;
    }
    __device__ __forceinline__ int64_t at(int i) const          // column of element i, clamped into the row
    {
        if constexpr (MODE == STRIDED) return c0 + i * T < cols ? c0 + i * T : 0;
        else return c + i;
    }
    __device__ __forceinline__ bool counts(int i) const          // whether element i is this lane's in a sum
    {
        if constexpr (MODE == STRIDED) return c0 + i * T < cols;
        else if constexpr (MODE == OVERLAP) return in && c + i >= c0;
        else return in;
    }
};

// a chunk as it is in memory
template <int SRC, int MODE> struct RowRaw { uint32_t w[MODE == STRIDED ? 8 : 2 * ElemT<SRC>::bytes]; };

template <int SRC, int MODE, int T>
__device__ __forceinline__ RowRaw<SRC, MODE> load_raw(const void* row, const Cols<MODE, T>& p)
{
    RowRaw<SRC, MODE> r;
    if constexpr (MODE == STRIDED) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            if constexpr (SRC == SRC_BF16) r.w[i] = ((const uint16_t*)row)[p.at(i)];
            else r.w[i] = ((const uint32_t*)row)[p.at(i)];
        }
    } else {
        r = __builtin_bit_cast(decltype(r), load_chunk<SRC>(row, p.c));
    }
    return r;
}

template <int SRC, int MODE>
__device__ __forceinline__ void raw_values(const RowRaw<SRC, MODE>& r, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; i++) {
        if constexpr (SRC == SRC_F32) v[i] = __uint_as_float(r.w[i]);
        else if constexpr (MODE == STRIDED) v[i] = bf16_lo(r.w[i]);
        else v[i] = (i & 1) ? bf16_hi(r.w[i >> 1]) : bf16_lo(r.w[i >> 1]);
    }
}

template <int SRC, int MODE, int T>
__device__ __forceinline__ void load_row(const void* row, const Cols<MODE, T>& p, float (&v)[8])
{
    raw_values(load_raw<SRC>(row, p), v);
}

template <int SRC, int MODE, int T>
__device__ __forceinline__ void store_row(void* row, const Cols<MODE, T>& p, const float (&v)[8])
{
    if constexpr (MODE == STRIDED) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (p.counts(i)) store_elem<SRC>(row, p.at(i), v[i]);
    } else {
        if (p.in) store_chunk<SRC>(row, p.c, make_chunk<SRC>(v));
    }
}

template <int MODE, int T>
__device__ __forceinline__ void load_param(const void* q, int f32, const Cols<MODE, T>& p, float (&v)[8])
{
    if (f32) load_row<SRC_F32>(q, p, v);
    else load_row<SRC_BF16>(q, p, v);
}

// the sum of f(i) over the elements of the chunk that count
template <int MODE, int T, class F>
__device__ __forceinline__ float chunk_sum(const Cols<MODE, T>& p, F&& f)
{
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float x = f(i);
        s += MODE == WHOLE || p.counts(i) ? x : 0.0f;
    }
    return MODE != WHOLE || p.in ? s : 0.0f;
}

template <int SRC>
__device__ __forceinline__ const void* row_of(const void* p, int64_t row, int64_t ld)
{
    return (const uint8_t*)p + row * ld * ElemT<SRC>::bytes;
}

// y of one chunk, and its outputs
template <int SRC, int MODE, int T>
__device__ __forceinline__ void finish_chunk(const NormFwdJob& a, int64_t row, const Cols<MODE, T>& p, const float (&s)[8],
                                             float mean, float rstd)
{
    if (!a.y && !a.qy) return;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; i++) y[i] = (s[i] - mean) * rstd;
    if (a.weight) {
        float w[8];
        load_param(a.weight, a.param_f32, p, w);
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] *= w[i];
    }
    if (a.bias) {
        float b[8];
        load_param(a.bias, a.param_f32, p, b);
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] += b[i];
    }
    if (a.y) {
        if (a.out_f32) store_row<SRC_F32>((float*)a.y + row * a.ld_y, p, y);
        else store_row<SRC_BF16>((uint16_t*)a.y + row * a.ld_y, p, y);
    }
    if constexpr (MODE == WHOLE)
        if (a.qy) encode_row_chunk(a.y_fmt, y, p.in, row * a.cols + p.c0, a.qy, a.sy);
}

// s = x (+ residual) of one chunk, with the sum and the checkpoint written
template <int SRC, int MODE, int T>
__device__ __forceinline__ void residual_and_checkpoint(const NormFwdJob& a, int64_t row, const Cols<MODE, T>& p,
                                                        float (&s)[8])
{
    if (a.residual) {
        float r[8];
        load_row<SRC>(row_of<SRC>(a.residual, row, a.ld_res), p, r);
#pragma unroll
        for (int i = 0; i < 8; i++) s[i] = rounded<SRC>(s[i] + r[i]);
        store_row<SRC>((void*)row_of<SRC>(a.sum, row, a.ld_sum), p, s);
    }
    if constexpr (MODE == WHOLE)
        if (a.qx) encode_row_chunk(a.ckpt_fmt, s, p.in, row * a.cols + p.c0, a.qx, a.sx);
}

__device__ __forceinline__ float inv_sqrt(float v) { return 1.0f / __builtin_sqrtf(v); }

template <int SRC, int MODE, int T, int N>
__global__ __launch_bounds__(T < 128 ? 256 : T) void k_norm_fwd(NormFwdJob a)
{
    constexpr int RPB = T < 128 ? 256 / T : 1;
    __shared__ float red[2][T < 64 ? 1 : T / 64];
    const int t = (int)threadIdx.x % T;
    const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / T;
    if (row >= a.rows) return;               // whole rows' lanes, and only where no barrier follows (T <= 64)
    typedef Cols<MODE, T> P;
    float s[N][8];
#pragma unroll
    for (int j = 0; j < N; j++) load_row<SRC>(row_of<SRC>(a.x, row, a.ld_x), P(j, t, a.cols), s[j]);
#pragma unroll
    for (int j = 0; j < N; j++) residual_and_checkpoint<SRC>(a, row, P(j, t, a.cols), s[j]);
    const float n = (float)a.cols;
    float mean = 0.0f;
    if (a.layer) {
        float p = 0.0f;
#pragma unroll
        for (int j = 0; j < N; j++) p += chunk_sum(P(j, t, a.cols), [&](int i) { return s[j][i]; });
        mean = group_sum<T>(p, red[0]) / n;
    }
    float p = 0.0f;
#pragma unroll
    for (int j = 0; j < N; j++)
        p += chunk_sum(P(j, t, a.cols), [&](int i) { const float c = s[j][i] - mean; return c * c; });
    const float rstd = inv_sqrt(group_sum<T>(p, red[1]) / n + a.eps);
    if (t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int j = 0; j < N; j++) finish_chunk<SRC>(a, row, P(j, t, a.cols), s[j], mean, rstd);
}

template <int SRC, int MODE>
__global__ __launch_bounds__(1024) void k_norm_fwd_wide(NormFwdJob a)
{
    constexpr int T = 1024;
    typedef Cols<MODE, T> P;
    __shared__ float red[2][T / 64];
    const int t = (int)threadIdx.x;
    const int64_t row = blockIdx.x, steps = (a.cols + T * 8 - 1) / (T * 8);
    // after the first pass s is in the sum, written by the same thread (and
    // by a second one, in OVERLAP, with the same values)
    const void* xr = row_of<SRC>(a.x, row, a.ld_x);
    const void* sr = a.residual ? row_of<SRC>(a.sum, row, a.ld_sum) : xr;
    float p = 0.0f;
    for (int64_t j = 0; j < steps; j++) {
        float s[8];
        const P at(j, t, a.cols);
        load_row<SRC>(xr, at, s);
        residual_and_checkpoint<SRC>(a, row, at, s);
        p += chunk_sum(at, [&](int i) { return a.layer ? s[i] : s[i] * s[i]; });
    }
    const float n = (float)a.cols;
    p = group_sum<T>(p, red[0]) / n;
    float mean = 0.0f, var = p;
    if (a.layer) {
        mean = p;
        p = 0.0f;
        for (int64_t j = 0; j < steps; j++) {
            float s[8];
            const P at(j, t, a.cols);
            load_row<SRC>(sr, at, s);
            p += chunk_sum(at, [&](int i) { const float c = s[i] - mean; return c * c; });
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
        const P at(j, t, a.cols);
        load_row<SRC>(sr, at, s);
        finish_chunk<SRC>(a, row, at, s, mean, rstd);
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// the inputs of one chunk of a row, as they are in memory
template <int SRC, int FROM, int MODE>
struct BwdRaw {
    RowRaw<SRC, MODE> dy, x, dsum;
    uint2 q;
    uint8_t s;
};

template <int SRC, int FROM, int MODE, int T>
__device__ __forceinline__ void load_bwd(const NormBwdJob& a, int64_t row, const Cols<MODE, T>& p, bool dsum,
                                         BwdRaw<SRC, FROM, MODE>& r)
{
    r.dy = load_raw<SRC>(row_of<SRC>(a.dy, row, a.ld_dy), p);
    if constexpr (FROM != FROM_TENSOR) {
        const int64_t e = row * a.cols + p.c;
        r.q = *(const uint2*)(a.qx + e);
        r.s = a.sx[e >> 5];
    } else {
        r.x = load_raw<SRC>(row_of<SRC>(a.x, row, a.ld_x), p);
    }
    if (dsum) r.dsum = load_raw<SRC>(row_of<SRC>(a.dsum, row, a.ld_dsum), p);
}

// h = (s - m) r of one chunk
template <int SRC, int FROM, int MODE>
__device__ __forceinline__ void unit_values(const BwdRaw<SRC, FROM, MODE>& r, float mean, float rstd, float (&h)[8])
{
    if constexpr (FROM != FROM_TENSOR) decode8<FROM>(r.q, r.s, h);
    else raw_values<SRC, MODE>(r.x, h);
#pragma unroll
    for (int i = 0; i < 8; i++) h[i] = (h[i] - mean) * rstd;
}

// dx of one chunk from g, h and the two means
template <int SRC, int FROM, int MODE, int T>
__device__ __forceinline__ void store_dx(const NormBwdJob& a, int64_t row, const Cols<MODE, T>& p,
                                         const BwdRaw<SRC, FROM, MODE>& r, const float (&g)[8], const float (&h)[8],
                                         float rstd, float mg, float mgh)
{
    float d[8];
#pragma unroll
    for (int i = 0; i < 8; i++) d[i] = rstd * (g[i] - mg - h[i] * mgh);
    if (a.dsum) {
        float e[8];
        raw_values<SRC, MODE>(r.dsum, e);
#pragma unroll
        for (int i = 0; i < 8; i++) d[i] += e[i];
    }
    store_row<SRC>((void*)row_of<SRC>(a.dx, row, a.ld_dx), p, d);
}

// Workgroups of RPB groups of T threads, a row per group at a time.  The next
// row's inputs are loaded before the current row is worked on, except where
// 1024 threads (128 registers each) hold two chunks, and the weight stays in
// registers where a thread has one chunk.  Two groups of 384 threads for bf16, four of 192: one row ahead of
// one group is too little in flight for a CU (8192 x 2304 bf16 with a
// checkpoint 33.6 us against 44.7, 16384 x 2656 59.9 and 71.3, 500 x 2656 9.0
// and 8.5).  fp32 rows have the bytes with one group of 384 (16384 x 3000
// 146.7 us, with two 151.7), as have those of 512 threads (8192 x 4096 46.2
// and 47.7).
template <int SRC, int T>
constexpr int bwd_block() { return T == 192 ? 768 : T <= 256 ? 512 : T == 384 && SRC == SRC_BF16 ? 768 : T; }

template <int SRC, int FROM, int MODE, int T, int N>
__global__ __launch_bounds__((bwd_block<SRC, T>())) void k_norm_bwd(NormBwdJob a)
{
    constexpr int RPB = bwd_block<SRC, T>() / T, W = T < 64 ? 1 : T / 64;
    typedef Cols<MODE, T> P;
    __shared__ float red[2][2][RPB][W];
    __shared__ float part[RPB > 1 ? RPB - 1 : 1][RPB > 1 ? N * T * 8 : 1];
    const int t = (int)threadIdx.x % T, sub = (int)threadIdx.x / T;
    constexpr bool AHEAD = N == 1 || T == 512, KEEP = N == 1;
    float w[N][8], dw[N][8], db[N][8];
    auto weight = [&](int j) {
#pragma unroll
        for (int i = 0; i < 8; i++) w[j][i] = 1.0f;
        if (a.weight) load_param(a.weight, a.param_f32, P(j, t, a.cols), w[j]);
    };
#pragma unroll
    for (int j = 0; j < N; j++) {
#pragma unroll
        for (int i = 0; i < 8; i++) dw[j][i] = 0.0f, db[j][i] = 0.0f;
        if (KEEP) weight(j);
    }
    const float n = (float)a.cols;
    BwdRaw<SRC, FROM, MODE> raw[N];
    float mean = 0.0f, rstd = 0.0f;
    auto fetch = [&](int64_t row) {
        rstd = a.rstd[row];
        mean = a.layer ? a.mean[row] : 0.0f;
#pragma unroll
        for (int j = 0; j < N; j++) load_bwd(a, row, P(j, t, a.cols), a.dsum != nullptr, raw[j]);
    };
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + sub;
    if (AHEAD && row < a.rows) fetch(row);
    // The sums alternate between two halves of `red`: a wave writes one half
    // again only after the barrier of the step between, which every wave
    // reaches after reading it.  A group whose rows have ended keeps meeting
    // the others' barriers.
    for (int half = 0; row - sub < a.rows; row += step, half ^= 1) {
        const bool live = row < a.rows;
        if (!AHEAD && live) fetch(row);
        const float m = mean, r = rstd;
        BwdRaw<SRC, FROM, MODE> now[N];
#pragma unroll
        for (int j = 0; j < N; j++) now[j] = raw[j];
        if (AHEAD && row + step < a.rows) fetch(row + step);
        float g[N][8], h[N][8], pg = 0.0f, pgh = 0.0f;
        if (live) {
#pragma unroll
            for (int j = 0; j < N; j++) {
                const P p(j, t, a.cols);
                if (!KEEP) weight(j);
                raw_values<SRC, MODE>(now[j].dy, g[j]);
                unit_values(now[j], m, r, h[j]);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    dw[j][i] += g[j][i] * h[j][i];
                    db[j][i] += g[j][i];
                    g[j][i] *= w[j][i];
                }
                pgh += chunk_sum(p, [&](int i) { return g[j][i] * h[j][i]; });
                pg += chunk_sum(p, [&](int i) { return g[j][i]; });
            }
            pgh = lanes_sum<T>(pgh);
            if (a.layer) pg = lanes_sum<T>(pg);
        }
        if constexpr (W > 1) {
            if ((threadIdx.x & 63) == 0) {
                red[half][0][sub][t >> 6] = pgh;
                red[half][1][sub][t >> 6] = pg;
            }
            __syncthreads();
            pgh = red[half][0][sub][0];
            pg = red[half][1][sub][0];
#pragma unroll
            for (int i = 1; i < W; i++) {
                pgh += red[half][0][sub][i];
                pg += red[half][1][sub][i];
            }
        }
        if (live) {
            const float mgh = pgh / n, mg = a.layer ? pg / n : 0.0f;
#pragma unroll
            for (int j = 0; j < N; j++) store_dx(a, row, P(j, t, a.cols), now[j], g[j], h[j], r, mg, mgh);
        }
    }
    // the groups' sums added in their order, and this workgroup's partial row
    auto finish = [&](float (&v)[N][8], float* out) {
        if constexpr (RPB > 1) {
            __syncthreads();
            if (sub > 0) {
#pragma unroll
                for (int j = 0; j < N; j++)
#pragma unroll
                    for (int i = 0; i < 8; i++) part[sub - 1][(j * 8 + i) * T + t] = v[j][i];
            }
            __syncthreads();
            if (sub > 0) return;
#pragma unroll 4
            for (int k = 0; k < RPB - 1; k++)
#pragma unroll
                for (int j = 0; j < N; j++)
#pragma unroll
                    for (int i = 0; i < 8; i++) v[j][i] += part[k][(j * 8 + i) * T + t];
        }
#pragma unroll
        for (int j = 0; j < N; j++) store_row<SRC_F32>(out, P(j, t, a.cols), v[j]);
    };
    if (a.dweight) finish(dw, a.work + blockIdx.x * a.cols);
    if (a.dbias) finish(db, a.work + ((a.dweight ? gridDim.x : 0) + blockIdx.x) * a.cols);
}

template <int SRC, int FROM, int MODE>
__global__ __launch_bounds__(1024) void k_norm_bwd_wide(NormBwdJob a, int64_t row0)
{
    constexpr int T = 1024;
    typedef Cols<MODE, T> P;
    __shared__ float red[2][T / 64];
    const int t = (int)threadIdx.x;
    const int64_t row = row0 + blockIdx.x, steps = (a.cols + T * 8 - 1) / (T * 8);
    const float mean = a.layer ? a.mean[row] : 0.0f, rstd = a.rstd[row], n = (float)a.cols;
    float pg = 0.0f, pgh = 0.0f;
    auto values = [&](const P& p, const BwdRaw<SRC, FROM, MODE>& r, float (&g)[8], float (&h)[8]) {
        raw_values<SRC, MODE>(r.dy, g);
        if (a.weight) {
            float w[8];
            load_param(a.weight, a.param_f32, p, w);
#pragma unroll
            for (int i = 0; i < 8; i++) g[i] *= w[i];
        }
        unit_values(r, mean, rstd, h);
    };
    for (int64_t j = 0; j < steps; j++) {
        float g[8], h[8];
        const P p(j, t, a.cols);
        BwdRaw<SRC, FROM, MODE> r;
        load_bwd(a, row, p, false, r);
        values(p, r, g, h);
        pgh += chunk_sum(p, [&](int i) { return g[i] * h[i]; });
        pg += chunk_sum(p, [&](int i) { return g[i]; });
    }
    const float mgh = group_sum<T>(pgh, red[0]) / n;
    const float mg = a.layer ? group_sum<T>(pg, red[1]) / n : 0.0f;
    for (int64_t j = 0; j < steps; j++) {
        float g[8], h[8];
        const P p(j, t, a.cols);
        BwdRaw<SRC, FROM, MODE> r;
        load_bwd(a, row, p, a.dsum != nullptr, r);
        values(p, r, g, h);
        store_dx(a, row, p, r, g, h, rstd, mg, mgh);
    }
}

// Partial sums of dw and db over the rows of one part, a strip of 512
// columns per wave: grid (strips / 4, parts)
template <int SRC, int FROM, int MODE>
__global__ __launch_bounds__(256) void k_norm_cols(NormBwdJob a, int64_t rows_per_part)
{
    constexpr int T = 64;
    const int t = (int)threadIdx.x & 63;
    const int64_t j = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), part = blockIdx.y, parts = gridDim.y;
    if (j * T * 8 >= a.cols) return;
    const Cols<MODE, T> p(j, t, a.cols);
    float dw[8] = {}, db[8] = {};
    const int64_t end = min((part + 1) * rows_per_part, a.rows);
    for (int64_t row = part * rows_per_part; row < end; row++) {
        float dy[8], h[8];
        BwdRaw<SRC, FROM, MODE> r;
        load_bwd(a, row, p, false, r);
        raw_values<SRC, MODE>(r.dy, dy);
        unit_values(r, a.layer ? a.mean[row] : 0.0f, a.rstd[row], h);
#pragma unroll
        for (int i = 0; i < 8; i++) dw[i] += dy[i] * h[i], db[i] += dy[i];
    }
    if (a.dweight) store_row<SRC_F32>(a.work + part * a.cols, p, dw);
    if (a.dbias) store_row<SRC_F32>(a.work + ((a.dweight ? parts : 0) + part) * a.cols, p, db);
}

// dw (blockIdx.y 0) and db (1, or 0 without dw): 32 columns per workgroup, from
// column c0 on, 32 threads down the partial rows of each column, added by
// halves at the end
__global__ __launch_bounds__(1024) void k_norm_colsum(const float* work, int64_t parts, int64_t cols, int64_t c0,
                                                      float* out0, float* out1)
{
    __shared__ float sum[32][33];
    const int x = (int)threadIdx.x & 31, y = (int)threadIdx.x >> 5;
    const int64_t c = c0 + (int64_t)blockIdx.x * 32 + x;
    const float* p = work + (int64_t)blockIdx.y * parts * cols;
    float s = 0.0f;
    if (c < cols) {
        // four partial rows in flight a thread
        float v[4] = {};
        int64_t r = y;
        for (; r + 96 < parts; r += 128)
#pragma unroll
            for (int k = 0; k < 4; k++) v[k] += p[(r + 32 * k) * cols + c];
        for (; r < parts; r += 32) v[0] += p[r * cols + c];
        s = (v[0] + v[1]) + (v[2] + v[3]);
    }
    sum[y][x] = s;
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
        __syncthreads();
        if (y < m) sum[y][x] += sum[y + m][x];
    }
    if (y == 0 && c < cols) (blockIdx.y ? out1 : out0)[c] = sum[0][x];
}

// Threads per row, one chunk each where 1024 threads hold the row so.  Against
// 256 threads with 2 to 4 chunks each (64 and 512 threads in the backward),
// bf16 with a checkpoint: the forward 32768 x 1024 50.5 us against 52.8, 8192 x
// 4096 50.4 against 52.9, 8192 x 8192 105.7 against 114.4; the backward 44.1
// against 65.9, 44.8 against 46.9, 94.4 against 95.0.  Rows of up to 256 share
// a wave (the norms of single heads).
// 640 threads are for the forward alone (8192 x 5120: 71.5 us against 72.5 with
// 768; the backward 63.4 against 60.2), 192 for the backward, four rows at a
// time (16384 x 1536 bf16 37.9 us against 49.8 with 256 threads two at a time
// and 39.2 four at a time, which is slower for 8192 x 2048, 27.9 against 27.2).
// Rows of 8193 to 12288 bf16 elements in the backward: 512 threads with three
// chunks, which have the registers to load a row ahead (4096 x 8224 with a
// checkpoint 65.8 us against 75.6 with two chunks of 1024 threads, 4096 x 12288
// 82.9 and 90.1).  In fp32 three chunks spill (146 us against 124 at 4096 x
// 8224), as do four chunks, and three in the STRIDED form.
template <bool BACKWARD, int SRC, int MODE, class F>
hipError_t by_width(int64_t cols, F&& f)
{
    constexpr std::integral_constant<int, 1> one;
    constexpr std::integral_constant<int, 2> two;
    if (cols <= 8 * 8) return f(std::integral_constant<int, 8>(), one);
    if (cols <= 16 * 8) return f(std::integral_constant<int, 16>(), one);
    if (cols <= 32 * 8) return f(std::integral_constant<int, 32>(), one);
    if (cols <= 64 * 8) return f(std::integral_constant<int, 64>(), one);
    if (cols <= 128 * 8) return f(std::integral_constant<int, 128>(), one);
    if constexpr (BACKWARD)
        if (cols <= 192 * 8) return f(std::integral_constant<int, 192>(), one);
    if (cols <= 256 * 8) return f(std::integral_constant<int, 256>(), one);
    if (cols <= 384 * 8) return f(std::integral_constant<int, 384>(), one);
    if (cols <= 512 * 8) return f(std::integral_constant<int, 512>(), one);
    if constexpr (!BACKWARD)
        if (cols <= 640 * 8) return f(std::integral_constant<int, 640>(), one);
    if (cols <= 768 * 8) return f(std::integral_constant<int, 768>(), one);
    if (cols <= 1024 * 8) return f(std::integral_constant<int, 1024>(), one);
    if constexpr (BACKWARD && SRC == SRC_BF16 && MODE != STRIDED)
        if (cols <= 3 * 512 * 8) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 3>());
    return f(std::integral_constant<int, 1024>(), two);
}

// A launch counts its threads in 32 bits: f(first row, rows) for slices of
// rows (or of columns) that need at most 2^31, at T threads each.
template <class F>
hipError_t sliced(int64_t rows, int64_t T, F&& f)
{
    const int64_t most = ((int64_t)1 << 31) / T;
    for (int64_t r = 0; r < rows; r += most) {
        f(r, rows - r < most ? rows - r : most);
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class T>
void advance(T*& p, int64_t bytes)
{
    if (p) p = (T*)((uint8_t*)p + bytes);
}

template <int SRC>
NormFwdJob rows_of(NormFwdJob j, int64_t r, int64_t n)
{
    constexpr int64_t B = ElemT<SRC>::bytes;
    j.rows = n;
    advance(j.x, r * j.ld_x * B);
    advance(j.residual, r * j.ld_res * B);
    advance(j.sum, r * j.ld_sum * B);
    advance(j.y, r * j.ld_y * (j.out_f32 ? 4 : 2));
    for (uint8_t** q : {&j.qy, &j.qx}) advance(*q, r * j.cols);
    for (uint8_t** q : {&j.sy, &j.sx}) advance(*q, r * (j.cols / 32));
    for (float** v : {&j.mean, &j.rstd}) advance(*v, r * 4);
    return j;
}

template <int SRC, int MODE>
hipError_t launch_fwd(const NormFwdJob& job, hipStream_t s)
{
    if (job.cols > NORM_WIDE) {
        return sliced(job.rows, 1024, [&](int64_t r, int64_t n) {
            k_norm_fwd_wide<SRC, MODE><<<dim3((unsigned)n), dim3(1024), 0, s>>>(rows_of<SRC>(job, r, n));
        });
    }
    return by_width<false, SRC, MODE>(job.cols, [&](auto T, auto N) {
        constexpr int B = T < 128 ? 256 : (int)T, RPB = B / T;
        return sliced(job.rows, T, [&](int64_t r, int64_t n) {
            k_norm_fwd<SRC, MODE, T, N><<<dim3((unsigned)((n + RPB - 1) / RPB)), dim3(B), 0, s>>>(rows_of<SRC>(job, r, n));
        });
    });
}

// Workgroups, and so partial rows, of the backward at most: one for each CU,
// two for rows that few threads hold.  (32768 x 1024 43.9 us with 512, 45.9
// with 256; 8192 x 4096 layer norm 54.3 and 48.7; 2047 x 4097 fp32 37.7 and
// 30.9: there the partial sums' traffic counts.)
int64_t most_parts(int64_t cols) { return cols <= 1024 ? 512 : 256; }

int64_t wide_parts(int64_t rows) { return rows < 64 ? rows : 64; }

template <int SRC, int FROM, int MODE>
hipError_t launch_bwd(const NormBwdJob& j, hipStream_t s)
{
    int64_t parts = 0;
    if (j.cols > NORM_WIDE) {
        const hipError_t e = sliced(j.rows, 1024, [&](int64_t r, int64_t n) {
            k_norm_bwd_wide<SRC, FROM, MODE><<<dim3((unsigned)n), dim3(1024), 0, s>>>(j, r);
        });
        if (e != hipSuccess) return e;
        if (j.dweight || j.dbias) {
            parts = wide_parts(j.rows);
            const int64_t per = (j.rows + parts - 1) / parts;
            parts = (j.rows + per - 1) / per;
            k_norm_cols<SRC, FROM, MODE><<<dim3((unsigned)((j.cols + 2047) / 2048), (unsigned)parts), dim3(256), 0, s>>>(j, per);
        }
    } else {
        const hipError_t e = by_width<true, SRC, MODE>(j.cols, [&](auto T, auto N) {
            constexpr int RPB = bwd_block<SRC, T>() / T;
            parts = (j.rows + RPB - 1) / RPB;
            parts = parts < most_parts(j.cols) ? parts : most_parts(j.cols);
            k_norm_bwd<SRC, FROM, MODE, T, N><<<dim3((unsigned)parts), dim3(bwd_block<SRC, T>()), 0, s>>>(j);
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
    }
    if (j.dweight || j.dbias) {
        const bool both = j.dweight && j.dbias;
        return sliced(j.cols, 32, [&](int64_t c0, int64_t n) {
            k_norm_colsum<<<dim3((unsigned)((n + 31) / 32), both ? 2u : 1u), dim3(1024), 0, s>>>(
                j.work, parts, j.cols, c0, j.dweight ? j.dweight : j.dbias, j.dbias);
        });
    }
    return hipSuccess;
}

// f(how the rows are spread): `in_place` where an output is written over an input
template <class F>
hipError_t by_mode(int64_t cols, bool in_place, F&& f)
{
    if (cols % 8 == 0) return f(std::integral_constant<int, WHOLE>());
    if (cols > 8 && !in_place) return f(std::integral_constant<int, OVERLAP>());
    return f(std::integral_constant<int, STRIDED>());
}

}  // namespace

int64_t norm_bwd_partials(int64_t rows, int64_t cols)
{
    if (cols > NORM_WIDE) return wide_parts(rows);
    return rows < most_parts(cols) ? rows : most_parts(cols);
}

hipError_t launch_norm_fwd(const NormFwdJob& j, hipStream_t s)
{
    // a wide row's y is written while what was normalised is read again
    const bool in_place = (j.residual && (j.sum == j.x || j.sum == j.residual)) ||
                          (j.cols > NORM_WIDE && j.y && (j.y == j.x || j.y == j.sum));
    return by_mode(j.cols, in_place, [&](auto mode) {
        return j.src == SRC_F32 ? launch_fwd<SRC_F32, mode>(j, s) : launch_fwd<SRC_BF16, mode>(j, s);
    });
}

hipError_t launch_norm_bwd(const NormBwdJob& j, hipStream_t s)
{
    auto run = [&](auto src) {
        if (j.qx) return j.ckpt_fmt == E4M3 ? launch_bwd<src, FROM_E4M3, WHOLE>(j, s) : launch_bwd<src, FROM_E5M2, WHOLE>(j, s);
        return by_mode(j.cols, j.dx == j.dy || j.dx == j.dsum || j.dx == j.x, [&](auto mode) { return launch_bwd<src, FROM_TENSOR, mode>(j, s); });
    };
    return j.src == SRC_F32 ? run(std::integral_constant<int, SRC_F32>()) : run(std::integral_constant<int, SRC_BF16>());
}

}  // namespace mx
