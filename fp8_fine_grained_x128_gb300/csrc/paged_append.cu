// paged_append.cu -- new keys and values into a paged cache, with the rotation
// of queries and keys by their positions (sm_103a).
//
// FP8-RL article, "KV cache compression": the cache of a layer is kept in FP8
// with per-tensor scales.  Here the scales are given (per-tensor current
// scaling calibrates them) and every new token is rotated, scaled and rounded
// on its way from the projection's output to its page: one read of q, k, v,
// one write of q_out and of the cache rows, nothing in between.
//
// Rotation (Su et al., "RoFormer: Enhanced Transformer with Rotary Position
// Embedding", 2021): with c, s = cos and sin of position * frequency i, the
// pair (x1, x2) becomes (x1 c - x2 s, x2 c + x1 s), in FP32.
//
// Bound: HBM bandwidth.  A warp takes one token and a run of head rows; a
// lane owns the same two 8-element chunks in each of its rows, so its part of
// the table row (16 FP32 values) is loaded once and stays in registers.  All of
// a lane's loads are in flight together, and the query, key and value rows are dealt
// over a token's warps in turn, since only keys and values cost divisions.
// Measured, 32 query and 8 cache heads of 128: 8 x 4096 tokens into a BF16 cache
// 118 us (the measured copy rate), 8192 tokens into an E4M3 cache 35.5 us (0.78 of it: the ramp and
// the last wave; the FP8 divisions fill half the issue slots), 16 single tokens
// 9.4 us (a launch's latency).
#include <algorithm>

#include "kernels.h"
#include "paged.cuh"

namespace fp8fg {

constexpr int kAppendThreads = 128;
constexpr int kAppendRows = 4;   // head rows of a lane, their loads in flight together

struct AppendArgs {
    fp8_paged_kv_t c;
    fp8_paged_batch_t b;
    int64_t tokens, q_ld, k_ld, v_ld, q_out_ld, rope_len;
    const uint16_t *q, *k, *v;
    const float *rope;
    uint16_t *q_out;
    int q_heads, rot_dim, parts;
    unsigned check_ctas;   // CTAs that check the batch's arrays
    int *status;
};

struct Vec16 {   // two chunks of 8 BF16
    uint4 a, b;
};

__device__ __forceinline__ bool has_nonfinite16(const Vec16 &v) { return max(absmax8(v.a), absmax8(v.b)) >= 0x7F80u; }

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack8_bf16(const float (&f)[8])
{
    return make_uint4(bf16x2_rn(f[0], f[1]), bf16x2_rn(f[2], f[3]), bf16x2_rn(f[4], f[5]), bf16x2_rn(f[6], f[7]));
}

// 8 FP8 codes of x / s.  The packed division is the IEEE quotient wherever it
// can decide a code; a scale outside its range, or a quotient that overflows
// it (seen as a NaN code), takes the IEEE division.
template <int FMT>
__device__ __forceinline__ uint2 pack8_fp8(const float (&f)[8], const Divider2 &d)
{
    uint32_t c[4];
    bool redo = !d.fast;
    if (d.fast) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x, y;
            d.fast_div_f32(f[2 * i], f[2 * i + 1], x, y);
            c[i] = cvt2<FMT>(x, y);
        }
        redo = has_nan_code<FMT>(c[0] | (c[1] << 16)) || has_nan_code<FMT>(c[2] | (c[3] << 16));
    }
    if (redo) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = cvt2<FMT>(__fdiv_rn(f[2 * i], d.s), __fdiv_rn(f[2 * i + 1], d.s));
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// One head row's two chunks (a at element ea, b at eb of the row at dst).
template <int FMT>
__device__ __forceinline__ void store_row(void *base, int64_t at, int ea, int eb, const float (&x)[8],
                                          const float (&y)[8], const Divider2 &d)
{
    if (FMT == FP8_KV_BF16) {
        uint16_t *p = static_cast<uint16_t *>(base) + at;
        *reinterpret_cast<uint4 *>(p + ea) = pack8_bf16(x);
        *reinterpret_cast<uint4 *>(p + eb) = pack8_bf16(y);
    } else {
        uint8_t *p = static_cast<uint8_t *>(base) + at;
        *reinterpret_cast<uint2 *>(p + ea) = pack8_fp8<FMT>(x, d);
        *reinterpret_cast<uint2 *>(p + eb) = pack8_fp8<FMT>(y, d);
    }
}

// Where the cache's last row begins (debug build).
__device__ __forceinline__ int64_t last_row(const fp8_paged_kv_t &c, int64_t page, int64_t head, int64_t row)
{
    return (c.num_pages - 1) * page + (c.heads - 1) * head + (c.page_size - 1) * row;
}

// One warp's rows of its token.
template <int D, int FMT, bool INTERLEAVED>
__device__ __forceinline__ void append_rows(const AppendArgs &g)
{
    constexpr int kLanes = D / 16;             // lanes of a head row
    constexpr int kSlots = 32 / kLanes;        // head rows side by side in a warp
    const int lane = threadIdx.x & 31;
    const int64_t w = ((int64_t)blockIdx.x * kAppendThreads + threadIdx.x) >> 5;
    const int64_t t = w / g.parts;
    if (t >= g.tokens) return;
    const int part = (int)(w - t * g.parts);
    const int c = lane % kLanes, slot = lane / kLanes;
    const int rows = g.q_heads + 2 * g.c.heads;

    // the rows' loads first: they depend on nothing but the token
    const int half = g.rot_dim / 2, rot_lanes = g.rot_dim / 16;
    const bool turn = c < rot_lanes;
    const int ea = turn ? 8 * c : g.rot_dim + 16 * (c - rot_lanes);
    const int eb = turn ? 8 * c + half : ea + 8;
    Vec16 x[kAppendRows];
    int row[kAppendRows];
#pragma unroll
    for (int i = 0; i < kAppendRows; ++i) {
        const int r = (i * g.parts + part) * kSlots + slot;   // (every warp has its share of the keys and values)
        row[i] = r < rows ? r : -1;
        if (r >= rows) continue;
        const uint16_t *p = r < g.q_heads                ? g.q + t * g.q_ld + (int64_t)r * D
                            : r < g.q_heads + g.c.heads ? g.k + t * g.k_ld + (int64_t)(r - g.q_heads) * D
                                                        : g.v + t * g.v_ld + (int64_t)(r - g.q_heads - g.c.heads) * D;
        x[i].a = *reinterpret_cast<const uint4 *>(p + ea);
        x[i].b = *reinterpret_cast<const uint4 *>(p + eb);
    }

    const int seq = seq_of_token(g.b.q_offsets, g.b.seqs, t, lane);
    if (seq < 0 || seq >= g.b.seqs) return;   // a row of no sequence
    const int first = g.b.q_offsets[seq], next = g.b.q_offsets[seq + 1], len = g.b.kv_lens[seq];
    const int64_t pos = (int64_t)len - next + t;
    const int64_t pg = pos >= 0 ? pos >> (31 - __clz(g.c.page_size)) : -1;
    int page = -1;
    if (pg >= 0 && pg < g.b.pages_per_seq) page = g.b.page_table[seq * g.b.page_table_ld + pg];

    // The table row does not wait for the page: both are on their way before either is looked at (the page
    // first, then the row: 8 x 4096 tokens into a BF16 cache 128 us, FP8 prompt 38; side by side 118 and 35.5).
    float ca[8], sa[8], cb[8], sb[8];   // table values of chunk a and of chunk b
    if (turn && pos >= 0 && pos < g.rope_len) {
        const float *p = g.rope + pos * g.rot_dim;
        if (INTERLEAVED) {   // pair j of a chunk: elements 2j, 2j + 1
            const float4 c0 = *reinterpret_cast<const float4 *>(p + ea / 2);
            const float4 s0 = *reinterpret_cast<const float4 *>(p + half + ea / 2);
            const float4 c1 = *reinterpret_cast<const float4 *>(p + eb / 2);
            const float4 s1 = *reinterpret_cast<const float4 *>(p + half + eb / 2);
            ca[0] = c0.x; ca[1] = c0.y; ca[2] = c0.z; ca[3] = c0.w;
            sa[0] = s0.x; sa[1] = s0.y; sa[2] = s0.z; sa[3] = s0.w;
            cb[0] = c1.x; cb[1] = c1.y; cb[2] = c1.z; cb[3] = c1.w;
            sb[0] = s1.x; sb[1] = s1.y; sb[2] = s1.z; sb[3] = s1.w;
        } else {             // pair j: element j of chunk a with element j of chunk b
            const float4 c0 = *reinterpret_cast<const float4 *>(p + ea), c1 = *reinterpret_cast<const float4 *>(p + ea + 4);
            const float4 s0 = *reinterpret_cast<const float4 *>(p + half + ea);
            const float4 s1 = *reinterpret_cast<const float4 *>(p + half + ea + 4);
            ca[0] = c0.x; ca[1] = c0.y; ca[2] = c0.z; ca[3] = c0.w;
            ca[4] = c1.x; ca[5] = c1.y; ca[6] = c1.z; ca[7] = c1.w;
            sa[0] = s0.x; sa[1] = s0.y; sa[2] = s0.z; sa[3] = s0.w;
            sa[4] = s1.x; sa[5] = s1.y; sa[6] = s1.z; sa[7] = s1.w;
        }
    }
    const Divider2 kd(FMT == FP8_KV_BF16 || !g.c.k_scale ? 1.0f : *g.c.k_scale);
    const Divider2 vd(FMT == FP8_KV_BF16 || !g.c.v_scale ? 1.0f : *g.c.v_scale);

    // (offsets that decrease name a sequence whose rows the token is not among)
    const bool ok = t >= first && t < next && seq_rows_ok(g.b, g.tokens, first, next) && seq_len_ok(g.b, g.c.page_size, len);
    if (!ok || page < 0 || page >= g.c.num_pages || (g.rot_dim > 0 && pos >= g.rope_len)) {
        if (lane == 0) set_status(g.status, FP8_ERR_INVALID_ARG);
        return;
    }
    const int64_t rip = pos & (g.c.page_size - 1);

#pragma unroll
    for (int i = 0; i < kAppendRows; ++i) {
        if (row[i] < 0) continue;
        const bool is_q = row[i] < g.q_heads, is_v = row[i] >= g.q_heads + g.c.heads;
        float a[8], b[8];
        unpack8(x[i].a, a);
        unpack8(x[i].b, b);
        if (!is_q && has_nonfinite16(x[i])) set_status(g.status, FP8_ERR_NONFINITE);
        if (turn && !is_v) {
            if (INTERLEAVED) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float a1 = a[2 * j], a2 = a[2 * j + 1], b1 = b[2 * j], b2 = b[2 * j + 1];
                    a[2 * j] = a1 * ca[j] - a2 * sa[j];
                    a[2 * j + 1] = a2 * ca[j] + a1 * sa[j];
                    b[2 * j] = b1 * cb[j] - b2 * sb[j];
                    b[2 * j + 1] = b2 * cb[j] + b1 * sb[j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float x1 = a[j], x2 = b[j];
                    a[j] = x1 * ca[j] - x2 * sa[j];
                    b[j] = x2 * ca[j] + x1 * sa[j];
                }
            }
        }
        if (is_q) {
            uint16_t *p = g.q_out + t * g.q_out_ld + (int64_t)row[i] * D;
            if (dbg_span(t * g.q_out_ld + (int64_t)row[i] * D, D, (g.tokens - 1) * g.q_out_ld + (int64_t)g.q_heads * D, g.status)) {
                *reinterpret_cast<uint4 *>(p + ea) = pack8_bf16(a);
                *reinterpret_cast<uint4 *>(p + eb) = pack8_bf16(b);
            }
        } else if (is_v) {
            const int64_t at = page * g.c.v_page_stride + (row[i] - g.q_heads - g.c.heads) * g.c.v_head_stride + rip * g.c.v_row_stride;
            if (dbg_span(at, D, last_row(g.c, g.c.v_page_stride, g.c.v_head_stride, g.c.v_row_stride) + D, g.status))
                store_row<FMT>(g.c.v, at, ea, eb, a, b, vd);
        } else {
            const int64_t at = page * g.c.k_page_stride + (row[i] - g.q_heads) * g.c.k_head_stride + rip * g.c.k_row_stride;
            if (dbg_span(at, D, last_row(g.c, g.c.k_page_stride, g.c.k_head_stride, g.c.k_row_stride) + D, g.status))
                store_row<FMT>(g.c.k, at, ea, eb, a, b, kd);
        }
    }
}

template <int D, int FMT, bool INTERLEAVED>
__global__ void __launch_bounds__(kAppendThreads) k_rope_append(AppendArgs g)
{
    dependents_launch();
    dependency_wait();
    append_rows<D, FMT, INTERLEAVED>(g);
    // Sequences whose values are out of range are announced even where no token falls to them, by the first
    // CTAs (at the end: values loaded ahead cost the fifth CTA of an SM its registers).
    if (blockIdx.x >= g.check_ctas) return;
    for (int b = blockIdx.x * kAppendThreads + threadIdx.x; b < g.b.seqs; b += g.check_ctas * kAppendThreads) {
        const int first = g.b.q_offsets[b], next = g.b.q_offsets[b + 1];
        if (!seq_rows_ok(g.b, g.tokens, first, next) || (next != first && !seq_len_ok(g.b, g.c.page_size, g.b.kv_lens[b])))
            set_status(g.status, FP8_ERR_INVALID_ARG);
    }
}

template <int D, int FMT>
static int run_append(AppendArgs &g, int interleaved, cudaStream_t st)
{
    const int per_warp = kAppendRows * (32 / (D / 16));
    g.parts = (g.q_heads + 2 * g.c.heads + per_warp - 1) / per_warp;
    const int64_t warps = g.tokens * g.parts, blocks = (warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
    if (blocks >= (int64_t)1 << 31) return FP8_ERR_SHAPE;
    g.check_ctas = (unsigned)std::min<int64_t>(blocks, (g.b.seqs + kAppendThreads - 1) / kAppendThreads);
    return launch_dependent(interleaved ? k_rope_append<D, FMT, true> : k_rope_append<D, FMT, false>, dim3((unsigned)blocks),
                            kAppendThreads, 0, st, g);
}

int launch_rope_append_kv(const fp8_paged_kv_t &c, const fp8_paged_batch_t &b, int64_t tokens, const void *q,
                          int64_t q_ld, int q_heads, const void *k, int64_t k_ld, const void *v, int64_t v_ld,
                          const float *rope, int64_t rope_len, int rot_dim, int interleaved, void *q_out,
                          int64_t q_out_ld, int *status, cudaStream_t st)
{
    AppendArgs g{};
    g.c = c;
    g.b = b;
    g.tokens = tokens;
    g.q = static_cast<const uint16_t *>(q);
    g.q_ld = q_ld;
    g.q_heads = q_heads;
    g.k = static_cast<const uint16_t *>(k);
    g.k_ld = k_ld;
    g.v = static_cast<const uint16_t *>(v);
    g.v_ld = v_ld;
    g.rope = rope;
    g.rope_len = rope_len;
    g.rot_dim = rot_dim;
    g.q_out = static_cast<uint16_t *>(q_out);
    g.q_out_ld = q_out_ld;
    g.status = status;
    if (c.head_dim == 128) {
        if (c.format == FP8_KV_BF16) return run_append<128, FP8_KV_BF16>(g, interleaved, st);
        if (c.format == FP8_KV_E5M2) return run_append<128, FP8_KV_E5M2>(g, interleaved, st);
        return run_append<128, FP8_KV_E4M3>(g, interleaved, st);
    }
    if (c.format == FP8_KV_BF16) return run_append<64, FP8_KV_BF16>(g, interleaved, st);
    if (c.format == FP8_KV_E5M2) return run_append<64, FP8_KV_E5M2>(g, interleaved, st);
    return run_append<64, FP8_KV_E4M3>(g, interleaved, st);
}

}  // namespace fp8fg
