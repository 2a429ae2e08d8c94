// norm_act.cu -- RMSNorm and SwiGLU whose input is kept in 8 bits for the
// backward pass (sm_103a).
//
// The forward kernels write, beside their BF16 result, the input as 1x128
// codes and scales (the layout and rule of fp8_quant_1x128: s = fp32(amax /
// fmax), q = RNE_satfinite(x / s)); the backward kernels read those 1.03 bytes
// an element instead of the BF16 tensor.
//
// All four stream their operands once and are bound by HBM: 16-byte loads,
// every row (RMSNorm) or run of chunks (SwiGLU) held in registers from its
// load to its stores, so nothing is read twice.
#include <algorithm>

#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace fp8fg {

namespace {

// 8 codes of a tensor kept in 8 bits, times their chunk's scale.
template <int FMT>
__device__ __forceinline__ void kept8(uint2 q, float s, float (&x)[8])
{
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint16_t c = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
        uint32_t h;
        if (FMT == FP8_E4M3)
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
        else
            asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(c));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        x[2 * k] = f.x * s;
        x[2 * k + 1] = f.y * s;
    }
}

__device__ __forceinline__ void widen8(uint4 v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[2 * k] = bf16_lo(w[k]);
        x[2 * k + 1] = bf16_hi(w[k]);
    }
}

__device__ __forceinline__ uint4 round8(const float (&x)[8])
{
    return make_uint4(bf16x2_rn(x[0], x[1]), bf16x2_rn(x[2], x[3]), bf16x2_rn(x[4], x[5]), bf16x2_rn(x[6], x[7]));
}

// A load of data that this kernel may overwrite in place afterwards (so not
// through the read-only path), not kept in L1.
__device__ __forceinline__ uint4 load_once(const uint16_t *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The sum of v over the NT threads of a row (a warp, or the whole CTA through
// `part`, which no thread may still be reading).
template <int NT>
__device__ __forceinline__ float row_sum(float v, float *part)
{
    v = warp_sum(v);
    if (NT == 32) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) v += part[w];
    return v;
}

}  // namespace

// ---------------------------------------------------------------------------
// RMSNorm forward: h = x (+ res, rounded to BF16), rstd = (mean h^2 +
// eps)^-1/2, y = h rstd w.  NT threads hold a row, VPT 16-byte vectors each
// (norm_shape: a warp for the shortest rows, so that CTAs of 8 rows need no
// barrier, up to 512 threads for the longest); 16 neighbouring lanes hold one
// 128-column chunk, whose scale they reduce by shuffles.
// ---------------------------------------------------------------------------
struct NormFwdArgs {
    const uint16_t *x, *res, *w;
    uint16_t *y, *sum;
    uint8_t *c;
    float *cs, *rstd;
    int64_t rows, ldx, ldres, ldy, ldsum;
    int cols;
    float eps;
    int *status;
};

// A CTA's threads and rows: NT threads to one row, or 8 rows of a warp each.
template <int NT> constexpr int norm_threads() { return NT == 32 ? 256 : NT; }
template <int NT> constexpr int norm_rows() { return NT == 32 ? 8 : 1; }
// Backward: CTAs an SM of its persistent grid, and most rows of a ring.
template <int NT, int VPT> constexpr int norm_ctas() { return NT == 512 ? (VPT == 2 ? 2 : 1) : VPT <= 2 ? 3 : 2; }
constexpr int kNormStages = 4;

template <int FMT, int NT, int VPT>
__global__ void __launch_bounds__(norm_threads<NT>(), NT == 512 ? 2 : NT == 256 ? 5 : 1) k_rmsnorm_fwd(NormFwdArgs g)
{
    __shared__ float part[32];
    dependents_launch();
    dependency_wait();
    constexpr int kRows = norm_rows<NT>();
    const int t = threadIdx.x % NT;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / NT;
    if (row >= g.rows) return;   // a whole warp: only NT = 32 has rows to spare
    const int nv = g.cols / 8;
    uint4 v[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int at = t + NT * i;
        v[i] = at < nv ? load_once(g.x + row * g.ldx + at * 8) : make_uint4(0, 0, 0, 0);
    }
    if (g.res) {
        uint4 r[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int at = t + NT * i;
            r[i] = at < nv ? load_once(g.res + row * g.ldres + at * 8) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int at = t + NT * i;
            float a[8], b[8];
            widen8(v[i], a);
            widen8(r[i], b);
#pragma unroll
            for (int k = 0; k < 8; ++k) a[k] += b[k];
            v[i] = round8(a);
            if (at < nv && dbg_span(row * g.ldsum + at * 8, 8, (g.rows - 1) * g.ldsum + g.cols, g.status))
                *reinterpret_cast<uint4 *>(g.sum + row * g.ldsum + at * 8) = v[i];
        }
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        float a[8];
        widen8(v[i], a);
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fmaf(a[k], a[k], ss);
    }
    // the chunks' codes need no sum over the row: they are stored while it is formed
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int at = t + NT * i;
        uint32_t m = absmax8(v[i]);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (at < nv) {
            const float s = scale_from_amax_bits(m, FMT);
            const int64_t q = row * g.cols + at * 8;
            const uint2 code = quant8p<FMT>(v[i], Divider2(s));
            if (dbg_span(q, 8, g.rows * g.cols, g.status)) *reinterpret_cast<uint2 *>(g.c + q) = code;
            if ((at & 15) == 0) {
                if (m >= 0x7F80u) set_status(g.status, FP8_ERR_NONFINITE);
                if (dbg_cell(at >> 4, row, 1, g.cols / 128, g.rows, g.status)) g.cs[(int64_t)(at >> 4) * g.rows + row] = s;
            }
        }
    }
    ss = row_sum<NT>(ss, part);
    const float rstd = rsqrtf(ss / (float)g.cols + g.eps);
    if (t == 0 && dbg_span(row, 1, g.rows, g.status)) g.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int at = t + NT * i;
        if (at >= nv) continue;
        float a[8], w[8];
        widen8(v[i], a);
        widen8(*reinterpret_cast<const uint4 *>(g.w + at * 8), w);
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] = a[k] * rstd * w[k];
        if (dbg_span(row * g.ldy + at * 8, 8, (g.rows - 1) * g.ldy + g.cols, g.status))
            *reinterpret_cast<uint4 *>(g.y + row * g.ldy + at * 8) = round8(a);
    }
}

// ---------------------------------------------------------------------------
// RMSNorm backward.  With n = h rstd (h the values the codes stand for),
//   dh = (dy w - n mean(dy w n)) rstd (+ dsum),   dw = sum_rows dy n.
// A persistent grid walks the rows, NT threads one.  A row's codes, dy and dsum
// are fetched by bulk copies into a ring of up to 4 rows (short rows: one for each
// warp), so that the next rows are on their way while the current one is reduced
// (rows prefetched into registers, one ahead, kept half as many bytes in flight:
// 46 us at 8192 x 4096).  Every thread sees
// the same columns of all its rows and sums their dw in registers; the CTAs' sums
// go to the workspace and are added in a fixed order by k_column_sums.
// ---------------------------------------------------------------------------
struct NormBwdArgs {
    const uint8_t *c;
    const float *cs, *rstd;
    const uint16_t *w, *dy, *dsum;
    uint16_t *dx;
    float *part;        // [gridDim.x][cols]
    int64_t rows, lddy, lddsum, lddx;
    int cols, stages;
    int *status;
};

template <int FMT, int NT, int VPT>
__global__ void __launch_bounds__(norm_threads<NT>(), norm_ctas<NT, VPT>()) k_rmsnorm_bwd(NormBwdArgs g)
{
    constexpr int kRows = norm_rows<NT>();
    extern __shared__ __align__(128) uint8_t rings[];   // [rows of the CTA][stages][codes | dy | dsum]
    __shared__ __align__(8) uint64_t bars[kRows][kNormStages];
    __shared__ float part[2][32];
    __shared__ int abort_flag;
    const int t = threadIdx.x % NT, sub = threadIdx.x / NT, nv = g.cols / 8, S = g.stages;
    const uint32_t bytes = (uint32_t)g.cols * (g.dsum ? 5 : 3);
    uint8_t *ring = rings + (size_t)sub * S * bytes;
    uint64_t *full = bars[sub];
    if (threadIdx.x == 0) {
        for (int i = 0; i < kRows; ++i)
            for (int s = 0; s < S; ++s) mbar_init(&bars[i][s], 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    dependency_wait();
    const int64_t row0 = (int64_t)blockIdx.x * kRows + sub, step = (int64_t)gridDim.x * kRows;
    auto fetch = [&](int64_t row, int s) {      // thread 0 of the row
        uint8_t *to = ring + (size_t)s * bytes;
        mbar_arrive_expect_tx(&full[s], bytes);
        bulk_load(to, g.c + row * g.cols, (uint32_t)g.cols, &full[s]);
        bulk_load(to + g.cols, g.dy + row * g.lddy, (uint32_t)g.cols * 2, &full[s]);
        if (g.dsum) bulk_load(to + 3 * g.cols, g.dsum + row * g.lddsum, (uint32_t)g.cols * 2, &full[s]);
    };
    // a row's scales (4 bytes apart from the next row's: no copy fetches them) and rstd
    float scale[VPT], rstd = 0.0f;
    auto scales = [&](int64_t row) {
        if (row >= g.rows) return;
        rstd = __ldg(g.rstd + row);
#pragma unroll
        for (int i = 0; i < VPT; ++i) scale[i] = t + NT * i < nv ? __ldg(g.cs + (int64_t)((t + NT * i) >> 4) * g.rows + row) : 0.0f;
    };
    if (t == 0)
        for (int s = 0; s < S && row0 + s * step < g.rows; ++s) fetch(row0 + s * step, s);
    scales(row0);

    uint4 w[VPT];
    uint64_t acc[VPT][4];       // packed pairs
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        w[i] = t + NT * i < nv ? __ldg(reinterpret_cast<const uint4 *>(g.w) + t + NT * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][k] = 0;
    }
    int s = 0;
    uint32_t phase = 0;
    int it = 0;
    for (int64_t row = row0; row < g.rows; row += step, ++it) {
        float use[VPT];
        const float r = rstd;
#pragma unroll
        for (int i = 0; i < VPT; ++i) use[i] = scale[i] * r;
        scales(row + step);
        thread_wait(smem_u32(&full[s]), phase, &abort_flag, g.status);
        const uint8_t *at = ring + (size_t)s * bytes;
        uint64_t n[VPT][4], dot2 = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = t + NT * i;
            if (v >= nv) continue;
            const uint2 q = reinterpret_cast<const uint2 *>(at)[v];
            const uint4 d4 = reinterpret_cast<const uint4 *>(at + g.cols)[v];
            const uint32_t d[4] = {d4.x, d4.y, d4.z, d4.w}, ww[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            const uint64_t u2 = p2(use[i], use[i]);
            float f[8];
            kept8<FMT>(q, 1.0f, f);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                n[i][k] = p2_mul(p2(f[2 * k], f[2 * k + 1]), u2);
                const uint64_t p = p2_mul(p2_bf16x2(d[k]), n[i][k]);
                acc[i][k] = f2_add(acc[i][k], p);
                dot2 = p2_fma(p, p2_bf16x2(ww[k]), dot2);
            }
        }
        float lo, hi;
        f2_unpack(dot2, lo, hi);
        const float mean = row_sum<NT>(lo + hi, part[it & 1]) / (float)g.cols;
        // all threads are past the row before this one: its place takes the next to come
        if (NT == 32) __syncwarp();
        if (t == 0 && it > 0 && row + (S - 1) * step < g.rows) fetch(row + (S - 1) * step, s == 0 ? S - 1 : s - 1);
        const uint64_t m2 = p2(-mean, -mean), r2 = p2(r, r);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = t + NT * i;
            if (v >= nv) continue;
            const uint4 d4 = reinterpret_cast<const uint4 *>(at + g.cols)[v];
            const uint4 e4 = g.dsum ? reinterpret_cast<const uint4 *>(at + 3 * g.cols)[v] : make_uint4(0, 0, 0, 0);
            const uint32_t d[4] = {d4.x, d4.y, d4.z, d4.w}, e[4] = {e4.x, e4.y, e4.z, e4.w}, ww[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                o[k] = p2_bf16(p2_fma(p2_fma(n[i][k], m2, p2_mul(p2_bf16x2(d[k]), p2_bf16x2(ww[k]))), r2, p2_bf16x2(e[k])));
            if (dbg_span(row * g.lddx + v * 8, 8, (g.rows - 1) * g.lddx + g.cols, g.status))
                *reinterpret_cast<uint4 *>(g.dx + row * g.lddx + v * 8) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if (++s == S) {
            s = 0;
            phase ^= 1;
        }
    }
    dependents_launch();
    if (abort_flag && t == 0)       // copies that were given up on land before the CTA leaves
        for (int i = 0; i < S; ++i) mbar_wait_bounded(&full[i], i < s ? phase ^ 1 : phase, nullptr);
    float a[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) f2_unpack(acc[i][k], a[i][2 * k], a[i][2 * k + 1]);
    if (NT == 32) {     // the CTA's 8 warps' sums, one after another, through the rings
        float *sums = reinterpret_cast<float *>(rings);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = t + NT * i;
            if (v >= nv) continue;
            float4 *p = reinterpret_cast<float4 *>(sums + sub * g.cols + v * 8);
            p[0] = make_float4(a[i][0], a[i][1], a[i][2], a[i][3]);
            p[1] = make_float4(a[i][4], a[i][5], a[i][6], a[i][7]);
        }
        __syncthreads();
        for (int c = threadIdx.x; c < g.cols; c += 256) {
            float x = sums[c];
#pragma unroll
            for (int w = 1; w < 8; ++w) x += sums[w * g.cols + c];
            if (dbg_cell(blockIdx.x, c, 1, gridDim.x, g.cols, g.status)) g.part[(int64_t)blockIdx.x * g.cols + c] = x;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = t + NT * i;
        if (v >= nv || !dbg_cell(blockIdx.x, v * 8, 8, gridDim.x, g.cols, g.status)) continue;
        float4 *p = reinterpret_cast<float4 *>(g.part + (int64_t)blockIdx.x * g.cols + v * 8);
        p[0] = make_float4(a[i][0], a[i][1], a[i][2], a[i][3]);
        p[1] = make_float4(a[i][4], a[i][5], a[i][6], a[i][7]);
    }
}

// dw[c] (+)= sum over n rows of part[.][c]: 32 columns a CTA, its 32 warps
// take every 32nd row, then their sums are added in order.
__global__ void __launch_bounds__(1024) k_column_sums(const float *part, int n, int cols, float *dw, int accumulate, int *status)
{
    __shared__ float sums[32][33];
    dependents_launch();
    dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v = 0.0f;
#pragma unroll 4
    for (int r = warp; r < n; r += 32) v += part[(int64_t)r * cols + c];
    sums[warp][lane] = v;
    __syncthreads();
    if (warp == 0) {
        for (int w = 1; w < 32; ++w) v += sums[w][lane];
        if (dbg_span(c, 1, cols, status)) dw[c] = accumulate ? dw[c] + v : v;
    }
}

// ---------------------------------------------------------------------------
// SwiGLU forward from gu [rows][2F]: h = silu(g) u in BF16, gu's codes and
// scales.  A half-warp takes a run of U 128-column chunks of one row's gate
// half and the same chunks of its up half.
// ---------------------------------------------------------------------------
template <int FMT>
__global__ void __launch_bounds__(256, 4) k_swiglu_fwd_ckpt(const uint16_t *__restrict__ gu, int64_t rows, int nc, uint16_t *__restrict__ h,
                                                         uint8_t *__restrict__ c, float *__restrict__ cs, int *status)
{
    constexpr int U = 4;
    dependents_launch();
    dependency_wait();
    const int l16 = threadIdx.x & 15, hbase = threadIdx.x & 16;
    const int runs = (nc + U - 1) / U;
    const int64_t items = rows * runs, nhw = ((int64_t)gridDim.x * blockDim.x) >> 4, F = (int64_t)nc * 128;
    for (int64_t it = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 4; (it & ~(int64_t)1) < items; it += nhw) {
        const bool valid = it < items;
        const int64_t r = valid ? it / runs : 0;
        const int c0 = valid ? (int)(it - r * runs) * U : nc;
        const uint16_t *src = gu + r * 2 * F + l16 * 8;
        uint4 v[2 * U];     // gate chunks, then up chunks
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = c0 + u < nc;
            v[u] = in ? ldg_stream(src + (int64_t)(c0 + u) * 128) : make_uint4(0, 0, 0, 0);
            v[U + u] = in ? ldg_stream(src + F + (int64_t)(c0 + u) * 128) : make_uint4(0, 0, 0, 0);
        }
        uint32_t m[2 * U];
#pragma unroll
        for (int u = 0; u < 2 * U; ++u) m[u] = absmax8(v[u]);
        const GroupScale gs = half_warp_scales8<FMT>(m, l16);
        const int mine = c0 + gs.u % U;
        if (!(l16 & 2) && mine < nc) {
            if (gs.amax >= 0x7F80u) set_status(status, FP8_ERR_NONFINITE);
            const int64_t chunk = (gs.u < U ? 0 : nc) + mine;
            if (dbg_cell(chunk, r, 1, 2 * nc, rows, status)) cs[chunk * rows + r] = gs.s;
        }
#pragma unroll
        for (int u = 0; u < 2 * U; ++u) {
            const float su = __shfl_sync(0xffffffffu, gs.s, hbase + half_group_lane(u));
            const float ru = __shfl_sync(0xffffffffu, gs.r, hbase + half_group_lane(u));
            const int cb = c0 + u % U;
            if (cb >= nc) continue;
            const uint2 code = quant8p<FMT>(v[u], Divider2(su, ru));
            const int64_t at = r * 2 * F + (u < U ? 0 : F) + (int64_t)cb * 128 + l16 * 8;
            if (dbg_span(at, 8, rows * 2 * F, status)) *reinterpret_cast<uint2 *>(c + at) = code;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = r * F + (int64_t)(c0 + u) * 128 + l16 * 8;
            if (c0 + u < nc && dbg_span(at, 8, rows * F, status)) *reinterpret_cast<uint4 *>(h + at) = swiglu8(v[u], v[U + u]);
        }
    }
}

// ---------------------------------------------------------------------------
// SwiGLU backward from gu's codes: dgate = dh u sig (1 + g (1 - sig)), dup =
// dh g sig.  A warp takes 512 columns of one row (16 a lane, 16-byte loads of
// codes); a CTA's 8 warps take as much of one row as it has, then further rows
// (8192 x 14336: 151 us, 6.28 TB/s; with 8 rows of 512 columns each, whose scales
// would share sectors, 156 us).
// ---------------------------------------------------------------------------
template <bool LEFT>
__device__ __forceinline__ void swiglu_grad8_f32(const float (&g)[8], const float (&u)[8], const float (&d)[8], uint4 &dg, uint4 &du)
{
    float a[8], b[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) swiglu_grad<LEFT>(g[k], u[k], d[k], a[k], b[k]);
    dg = round8(a);
    du = round8(b);
}

template <int FMT>
__global__ void __launch_bounds__(256) k_swiglu_bwd_ckpt(const uint8_t *__restrict__ c, const float *__restrict__ cs,
                                                      const uint16_t *__restrict__ dh, int64_t rows, int64_t F, int log_rows,
                                                      uint16_t *__restrict__ dgu, int *status)
{
    dependents_launch();
    dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r = ((int64_t)blockIdx.x << log_rows) + (warp & ((1 << log_rows) - 1));
    const int64_t j = (((int64_t)blockIdx.y << (3 - log_rows)) + (warp >> log_rows)) * 512 + lane * 16;
    if (r >= rows || j >= F) return;
    const uint8_t *src = c + r * 2 * F + j;
    const uint4 qg = ldg_stream(src), qu = ldg_stream(src + F);
    const uint4 d0 = ldg_stream(dh + r * F + j), d1 = ldg_stream(dh + r * F + j + 8);
    const float sg = __ldg(cs + (j >> 7) * rows + r), su = __ldg(cs + ((F + j) >> 7) * rows + r);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float g[8], u[8], d[8];
        kept8<FMT>(k ? make_uint2(qg.z, qg.w) : make_uint2(qg.x, qg.y), sg, g);
        kept8<FMT>(k ? make_uint2(qu.z, qu.w) : make_uint2(qu.x, qu.y), su, u);
        widen8(k ? d1 : d0, d);
        float least = g[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) least = fminf(least, g[e]);
        uint4 og, ou;
        if (least < -64.0f) swiglu_grad8_f32<true>(g, u, d, og, ou);
        else swiglu_grad8_f32<false>(g, u, d, og, ou);
        const int64_t at = r * 2 * F + j + 8 * k;
        if (dbg_span(at + F, 8, rows * 2 * F, status)) {
            *reinterpret_cast<uint4 *>(dgu + at) = og;
            *reinterpret_cast<uint4 *>(dgu + at + F) = ou;
        }
    }
}

// ------------------------------------------------------------------ launchers

namespace {

// Calls f(NT, VPT) as compile-time numbers for rows of `cols` columns (up to
// kNormMaxCols).  Rows of 513 to 1024 columns: a warp each where they come in
// order through a ring, 128 threads each where a CTA has one row and no more
// (8192 x 1024 forward: 14.8 us, a warp each 18.1).
template <int N> struct Int { static constexpr int v = N; };
template <bool RING, typename F>
int norm_shape(int64_t cols, F &&f)
{
    if (cols <= 256) return f(Int<32>{}, Int<1>{});
    if (cols <= 512) return f(Int<32>{}, Int<2>{});
    if (cols <= 1024) return f(Int<RING ? 32 : 128>{}, Int<RING ? 4 : 1>{});
    if (cols <= 2048) return f(Int<256>{}, Int<1>{});
    if (cols <= 4096) return f(Int<256>{}, Int<2>{});
    if (cols <= 8192) return f(Int<512>{}, Int<2>{});
    return f(Int<512>{}, Int<4>{});
}

template <int FMT>
int norm_fwd(const NormFwdArgs &g, cudaStream_t st)
{
    return norm_shape<false>(g.cols, [&](auto nt, auto vpt) {
        constexpr int NT = decltype(nt)::v, VPT = decltype(vpt)::v;
        const int64_t blocks = (g.rows + norm_rows<NT>() - 1) / norm_rows<NT>();
        return launch_dependent(k_rmsnorm_fwd<FMT, NT, VPT>, dim3((unsigned)blocks), norm_threads<NT>(), 0, st, g);
    });
}

template <int FMT>
int norm_bwd(NormBwdArgs &g, float *dw, int accumulate, cudaStream_t st)
{
    return norm_shape<true>(g.cols, [&](auto nt, auto vpt) {
        constexpr int NT = decltype(nt)::v, VPT = decltype(vpt)::v, kCtas = norm_ctas<NT, VPT>();
        constexpr int kRing = 220 * 1024 / kCtas - 2048;    // an SM's shared memory, shared by its CTAs
        constexpr int kRows = norm_rows<NT>();
        const int row = g.cols * (g.dsum ? 5 : 3) * kRows;
        g.stages = std::min(kNormStages, kRing / row);
        const size_t smem = std::max<size_t>((size_t)g.stages * row, NT == 32 ? (size_t)g.cols * kRows * sizeof(float) : 0);
        static bool attr_done[64] = {};
        int dev = 0;
        cudaGetDevice(&dev);
        if (!attr_done[dev & 63]) {
            if (cudaFuncSetAttribute(k_rmsnorm_bwd<FMT, NT, VPT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing) != cudaSuccess)
                return (int)FP8_ERR_CUDA;
            attr_done[dev & 63] = true;
        }
        const int64_t grid = std::min<int64_t>((g.rows + kRows - 1) / kRows, (int64_t)sm_count() * kCtas);
        const int rc = launch_dependent(k_rmsnorm_bwd<FMT, NT, VPT>, dim3((unsigned)grid), norm_threads<NT>(), smem, st, g);
        if (rc != FP8_OK) return rc;
        return launch_dependent(k_column_sums, dim3((unsigned)(g.cols / 32)), 1024, 0, st, static_cast<const float *>(g.part), (int)grid, g.cols,
                                dw, accumulate, g.status);
    });
}

}  // namespace

int launch_rmsnorm_fwd_ckpt(const void *x, int64_t rows, int64_t cols, int64_t ldx, const void *res, int64_t ldres, const void *w, float eps,
                            int fmt, void *y, int64_t ldy, void *sum, int64_t ldsum, void *c, float *cs, float *rstd, int *status,
                            cudaStream_t st)
{
    NormFwdArgs g{};
    g.x = static_cast<const uint16_t *>(x);
    g.res = static_cast<const uint16_t *>(res);
    g.w = static_cast<const uint16_t *>(w);
    g.y = static_cast<uint16_t *>(y);
    g.sum = static_cast<uint16_t *>(sum);
    g.c = static_cast<uint8_t *>(c);
    g.cs = cs;
    g.rstd = rstd;
    g.rows = rows;
    g.cols = (int)cols;
    g.ldx = ldx;
    g.ldres = ldres;
    g.ldy = ldy;
    g.ldsum = ldsum;
    g.eps = eps;
    g.status = status;
    return fmt == FP8_E5M2 ? norm_fwd<FP8_E5M2>(g, st) : norm_fwd<FP8_E4M3>(g, st);
}

size_t rmsnorm_workspace_bytes(int64_t cols)
{
    const int ctas = norm_shape<true>(cols, [](auto nt, auto vpt) { return norm_ctas<decltype(nt)::v, decltype(vpt)::v>(); });
    return (size_t)sm_count() * ctas * (size_t)cols * sizeof(float);
}

int launch_rmsnorm_bwd_ckpt(const void *c, const float *cs, const float *rstd, int fmt, int64_t rows, int64_t cols, const void *w,
                            const void *dy, int64_t lddy, const void *dsum, int64_t lddsum, void *dx, int64_t lddx, float *dw,
                            int accumulate, void *ws, int *status, cudaStream_t st)
{
    if (rows == 0) {
        if (accumulate) return FP8_OK;
        return cudaMemsetAsync(dw, 0, (size_t)cols * sizeof(float), st) == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
    }
    NormBwdArgs g{};
    g.c = static_cast<const uint8_t *>(c);
    g.cs = cs;
    g.rstd = rstd;
    g.w = static_cast<const uint16_t *>(w);
    g.dy = static_cast<const uint16_t *>(dy);
    g.dsum = static_cast<const uint16_t *>(dsum);
    g.dx = static_cast<uint16_t *>(dx);
    g.part = static_cast<float *>(ws);
    g.rows = rows;
    g.cols = (int)cols;
    g.lddy = lddy;
    g.lddsum = lddsum;
    g.lddx = lddx;
    g.status = status;
    return fmt == FP8_E5M2 ? norm_bwd<FP8_E5M2>(g, dw, accumulate, st) : norm_bwd<FP8_E4M3>(g, dw, accumulate, st);
}

int launch_swiglu_fwd_ckpt(const void *gu, int64_t rows, int64_t F, int fmt, void *h, void *c, float *cs, int *status, cudaStream_t st)
{
    const int64_t items = rows * ((F / 128 + 3) / 4);
    const int64_t blocks = std::min<int64_t>((items + 15) / 16, (int64_t)1 << 20);
    return launch_dependent(fmt == FP8_E5M2 ? k_swiglu_fwd_ckpt<FP8_E5M2> : k_swiglu_fwd_ckpt<FP8_E4M3>, dim3((unsigned)blocks), 256, 0, st,
                            static_cast<const uint16_t *>(gu), rows, (int)(F / 128), static_cast<uint16_t *>(h), static_cast<uint8_t *>(c), cs,
                            status);
}

int launch_swiglu_bwd_ckpt(const void *c, const float *cs, const void *dh, int64_t rows, int64_t F, int fmt, void *dgu, int *status,
                           cudaStream_t st)
{
    int log_rows = 3;       // rows of a CTA; it takes 4096 columns over them
    while (log_rows > 0 && F > (int64_t)512 << (3 - log_rows)) --log_rows;
    const int64_t cols = (int64_t)512 << (3 - log_rows);
    return launch_dependent(fmt == FP8_E5M2 ? k_swiglu_bwd_ckpt<FP8_E5M2> : k_swiglu_bwd_ckpt<FP8_E4M3>,
                            dim3((unsigned)((rows + (1 << log_rows) - 1) >> log_rows), (unsigned)((F + cols - 1) / cols)), 256, 0, st,
                            static_cast<const uint8_t *>(c), cs, static_cast<const uint16_t *>(dh), rows, F, log_rows,
                            static_cast<uint16_t *>(dgu), status);
}

}  // namespace fp8fg
