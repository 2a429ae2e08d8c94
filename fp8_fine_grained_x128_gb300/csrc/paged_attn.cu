// paged_attn.cu -- attention of a chunk of new tokens over a paged key/value
// cache: the choice of kernel and the workspace.
//
// Softmax over the keys in one pass with a running maximum and sum (Milakov
// and Gimelshein, "Online normalizer calculation for softmax", 2018): scores
// are kept as log2 values x, a part of the keys is summed up as m = max x,
// l = sum 2^(x - m), o = sum 2^(x - m) v, and parts join by rescaling to the
// larger m.  A sequence whose rows (new tokens x query heads of a group) fit
// one 16-row operand is bound by the cache's bytes and goes to k_attn_few
// (mma.sync); the others go to k_attn_many (tcgen05, 256 rows a unit).  Each
// kernel reads the lengths on the device and leaves the other's sequences
// alone; a batch that can hold only short ones launches k_attn_few alone.
//
// Up to 32 rows k_attn_few (two groups of rows) still is the faster one where there
// are pairs enough that few parts of each have to be joined: with 32 query and 8
// cache heads of 128, k_attn_few / k_attn_many take 96 / 119 us for 32 sequences
// x 8 tokens over 4000 E4M3 keys, 60 / 106 for 64 x 5 over 1000 (75 / 99 BF16), 118 / 115
// for 32 x 5 over 4000 BF16 keys, 30 / 30 for 8 x 8 over 1500 (64 pairs), but 53 / 33
// for 1 x 8 over 8000 (8 pairs).  From 33 rows on the tensor cores win: 157 (with a form of
// k_attn_few that had four groups) / 119 for 32 x 12 over 4000 E4M3 keys, 201 / 116 over BF16 ones.
#include "kernels.h"
#include "paged.cuh"

namespace fp8fg {

// Workspace: k_attn_few's counters and parts, then k_attn_many's.
// The counters alone have to start as zeros; the header promises their place.
constexpr size_t kCounterBytes = 16384;
static size_t align256(size_t n) { return (n + 255) / 256 * 256; }

size_t paged_attention_workspace_bytes()
{
    return kCounterBytes + align256(few_parts_bytes()) + align256(many_joins_bytes()) +
           many_parts_bytes();
}

int launch_paged_attention(const fp8_paged_kv_t &c, const fp8_paged_batch_t &b, int64_t tokens, const void *q,
                           int64_t q_ld, int q_heads, float scale, void *out, int64_t out_ld, float *lse, void *ws,
                           int *status, cudaStream_t st)
{
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
    if (few_grid() * sizeof(int) > kCounterBytes) return FP8_ERR_UNSUPPORTED;   // (over 1365 SMs)
    uint8_t *p = static_cast<uint8_t *>(ws);
    g.few_count = reinterpret_cast<int *>(p);
    p += kCounterBytes;
    g.few_parts = p;
    p += align256(few_parts_bytes());
    g.many_joins = p;
    p += align256(many_joins_bytes());
    g.many_parts = reinterpret_cast<float *>(p);
    const int64_t rows = (int64_t)b.max_new * g.group, pairs = (int64_t)b.seqs * c.heads;
    if (rows <= kFewRows || (rows <= kFewMost && pairs * kDirectParts >= few_grid())) return run_few(g, (int)rows, st);
    const int rc = run_few(g, kFewRows, st);
    return rc != FP8_OK ? rc : run_many(g, st);
}

}  // namespace fp8fg
