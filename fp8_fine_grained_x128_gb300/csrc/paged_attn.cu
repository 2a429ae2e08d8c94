// paged_attn.cu -- attention of a chunk of new tokens over a paged key/value
// cache (sm_103a).
//
// One warp per (token, query head): the keys are read one by one through the
// page table, with the running maximum and sum of the softmax.
#include <algorithm>

#include "kernels.h"
#include "paged.cuh"

namespace fp8fg {

struct AttnArgs {
    fp8_paged_kv_t c;
    fp8_paged_batch_t b;
    int64_t tokens, q_ld, out_ld;
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    float scale;   // softmax scale
    int q_heads, group;
    int *status;
};

size_t paged_attention_workspace_bytes() { return 16; }

template <int FMT>
__device__ __forceinline__ float kv_value(const void *base, int64_t i)
{
    if (FMT == FP8_KV_BF16) return __uint_as_float((uint32_t) static_cast<const uint16_t *>(base)[i] << 16);
    uint32_t h;
    const uint16_t w = static_cast<const uint8_t *>(base)[i];
    if (FMT == FP8_KV_E4M3)
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(w));
    else
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(w));
    float f;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}" : "=f"(f) : "r"(h));
    return f;
}

template <int D, int FMT>
__global__ void __launch_bounds__(128) k_attn_rows(AttnArgs g)
{
    constexpr int kE = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = ((int64_t)blockIdx.x * 128 + threadIdx.x) >> 5;
    const int64_t t = w / g.q_heads;
    if (t >= g.tokens) return;
    const int h = (int)(w - t * g.q_heads), hk = h / g.group;
    const int seq = seq_of_token(g.b.q_offsets, g.b.seqs, t, lane);
    if (seq < 0 || seq >= g.b.seqs) return;
    const int64_t len = g.b.kv_lens[seq];
    const int64_t pos = len - g.b.q_offsets[seq + 1] + t;
    if (len < 0 || len > (int64_t)g.b.pages_per_seq * g.c.page_size) {
        if (lane == 0) set_status(g.status, FP8_ERR_INVALID_ARG);
        return;
    }
    const float ks = g.c.k_scale ? *g.c.k_scale : 1.0f, vs = g.c.v_scale ? *g.c.v_scale : 1.0f;
    float q[kE], o[kE] = {}, m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int e = 0; e < kE; ++e)
        q[e] = __uint_as_float((uint32_t)g.q[t * g.q_ld + (int64_t)h * D + lane + 32 * e] << 16);
    for (int64_t j = 0; j <= pos && j < len; ++j) {
        const int page = g.b.page_table[seq * g.b.page_table_ld + j / g.c.page_size];
        if (page < 0 || page >= g.c.num_pages) {
            if (lane == 0) set_status(g.status, FP8_ERR_INVALID_ARG);
            return;
        }
        const int64_t r = j % g.c.page_size;
        const int64_t ka = page * g.c.k_page_stride + hk * g.c.k_head_stride + r * g.c.k_row_stride;
        const int64_t va = page * g.c.v_page_stride + hk * g.c.v_head_stride + r * g.c.v_row_stride;
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < kE; ++e) s += q[e] * kv_value<FMT>(g.c.k, ka + lane + 32 * e);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= g.scale * ks;
        const float mn = fmaxf(m, s), a = expf(m - mn), p = expf(s - mn);
        l = l * a + p;
#pragma unroll
        for (int e = 0; e < kE; ++e) o[e] = o[e] * a + p * kv_value<FMT>(g.c.v, va + lane + 32 * e);
        m = mn;
    }
    const float inv = l > 0.0f ? vs / l : 0.0f;
    const int64_t at = t * g.out_ld + (int64_t)h * D;
    if (dbg_span(at, D, (g.tokens - 1) * g.out_ld + (int64_t)g.q_heads * D, g.status)) {
#pragma unroll
        for (int e = 0; e < kE; ++e) g.out[at + lane + 32 * e] = (uint16_t)bf16x2_rn(o[e] * inv, 0.0f);
    }
    if (g.lse && lane == 0) g.lse[t * g.q_heads + h] = l > 0.0f ? m + logf(l) : -INFINITY;
}

template <int D, int FMT>
static int run_attn(const AttnArgs &g, cudaStream_t st)
{
    const int64_t blocks = (g.tokens * g.q_heads + 3) / 4;
    k_attn_rows<D, FMT><<<(unsigned)blocks, 128, 0, st>>>(g);
    return cudaGetLastError() == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

int launch_paged_attention(const fp8_paged_kv_t &c, const fp8_paged_batch_t &b, int64_t tokens, const void *q,
                           int64_t q_ld, int q_heads, float scale, void *out, int64_t out_ld, float *lse, void *ws,
                           int *status, cudaStream_t st)
{
    (void)ws;
    AttnArgs g{};
    g.c = c;
    g.b = b;
    g.tokens = tokens;
    g.q = static_cast<const uint16_t *>(q);
    g.q_ld = q_ld;
    g.q_heads = q_heads;
    g.group = q_heads / c.heads;
    g.scale = scale;
    g.out = static_cast<uint16_t *>(out);
    g.out_ld = out_ld;
    g.lse = lse;
    g.status = status;
    if (c.head_dim == 128) {
        if (c.format == FP8_KV_BF16) return run_attn<128, FP8_KV_BF16>(g, st);
        if (c.format == FP8_KV_E5M2) return run_attn<128, FP8_KV_E5M2>(g, st);
        return run_attn<128, FP8_KV_E4M3>(g, st);
    }
    if (c.format == FP8_KV_BF16) return run_attn<64, FP8_KV_BF16>(g, st);
    if (c.format == FP8_KV_E5M2) return run_attn<64, FP8_KV_E5M2>(g, st);
    return run_attn<64, FP8_KV_E4M3>(g, st);
}

}  // namespace fp8fg
