// embed.cu -- embedding lookup with scaling, and its gradient (sm_103a).
//
// Forward: out[t] = scale * w[ids[t]], a copy bound by HBM.
// Backward: dw[v] (+)= scale * sum of dout[t] over the tokens with ids[t] = v.
// Adding rows with atomics would give sums that change from run to run with
// their order; here the tokens are sorted by id, each id's in their order, and
// every id's rows are summed in FP32 in that order: by one warp per 256 columns
// where they lie in one piece of the sorted tokens, else piece by piece and then
// over the pieces.  The order depends on the ids, the sizes and the number of SMs
// alone, so the results repeat.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace fp8fg {

// ---------------------------------------------------------------------------
// Forward: a warp takes up to 128 vectors (1024 columns) of one token.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) k_embedding_fwd(const int32_t *__restrict__ ids, int64_t tokens, const uint16_t *__restrict__ w, int64_t vocab,
                                                     int64_t ldw, int nv, int segs, float scale, uint16_t *__restrict__ out, int64_t ldo,
                                                     int *status)
{
    dependents_launch();
    dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t t = item / segs;
    if (t >= tokens) return;
    const int v0 = (int)(item - t * segs) * 128 + lane;
    const int64_t id = ids[t];
    if (id >= vocab && lane == 0) set_status(status, FP8_ERR_INVALID_ARG);
    const bool in = id >= 0 && id < vocab;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = in && v0 + 32 * i < nv ? __ldg(reinterpret_cast<const uint4 *>(w + id * ldw) + v0 + 32 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = v0 + 32 * i;
        uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = bf16x2_rn(scale * bf16_lo(x[k]), scale * bf16_hi(x[k]));
        if (!in) x[0] = x[1] = x[2] = x[3] = 0;    // not scale * 0, which an infinite scale makes NaN
        if (at < nv && dbg_span(t * ldo + at * 8, 8, (tokens - 1) * ldo + (int64_t)nv * 8, status))
            *reinterpret_cast<uint4 *>(out + t * ldo + at * 8) = make_uint4(x[0], x[1], x[2], x[3]);
    }
}

// ---------------------------------------------------------------------------
// Backward, sorting.  Tokens without an id, or with one out of range, sort
// behind the vocabulary.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int sort_key(int32_t id, int vocab) { return id < 0 || id >= vocab ? vocab : id; }

// Both sorts are stable radix sorts by digits of 9 bits.  A warp ranks 32 * K
// consecutive keys, 32 at a time: lanes of equal digits find one another by ballots
// of the digits' bits (many keys; the sort of 32768: 20 -> 17 us) or a match (two
// a thread), and the warp's counter of that digit holds how many came before.
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;

template <int K, bool BALLOTS, typename N>
__device__ __forceinline__ void rank_keys(const int (&key)[K], int shift, N *counter, int (&rank)[K])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int d = key[k] < 0 ? kDigits : (key[k] >> shift) & (kDigits - 1);
        unsigned same = 0xffffffffu;
        if (BALLOTS) {
#pragma unroll
            for (int b = 0; b <= kDigitBits; ++b) {
                const unsigned set = __ballot_sync(0xffffffffu, d >> b & 1);
                same &= d >> b & 1 ? set : ~set;
            }
        } else {
            same = __match_any_sync(0xffffffffu, d);
        }
        const int had = d < kDigits ? counter[d] : 0;
        rank[k] = had + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (d < kDigits && lane == __ffs(same) - 1) counter[d] = (N)(had + __popc(same));
        __syncwarp();
    }
}

// Up to 65536 tokens: all passes in one launch, by one cluster of up to 8 CTAs
// that hold the keys in their shared memory, add their digits' counts up and
// send each key to the CTA of its place.
constexpr int kClusterThreads = 1024, kClusterWarps = kClusterThreads / 32, kClusterCtas = 8, kClusterKeys = 8;
constexpr int kClusterMost = kClusterThreads * kClusterCtas * kClusterKeys;

template <int K>
struct ClusterSort {
    uint16_t cnt[kClusterWarps][kDigits];   // a CTA's keys fit 16 bits
    int tot[2][kDigits], start[kDigits], own[kDigits];
    int sums[2][kClusterWarps];
    int2 held[2][K * kClusterThreads];      // key, token
};

__device__ __forceinline__ int ld_cluster(uint32_t addr)
{
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, int x, int y)
{
    asm volatile("st.shared::cluster.v2.s32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}

// The sort by CTA `me` of `ctas`; emit(place, key, token) gets every token.  A
// cluster's CTA puts its keys in their order among themselves first and sends them
// from there, so that neighbouring lanes write neighbouring places (scattered from
// where they lay, 32768 keys took 23 us).
template <int K, bool CLUSTER, typename Emit>
__device__ __forceinline__ void sort_cluster(ClusterSort<K> &m, const int32_t *__restrict__ ids, int tokens, int vocab, int passes, int ctas,
                                             int me, int *status, Emit &&emit)
{
    constexpr int kOwn = K * kClusterThreads;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int at = warp * 32 * K + lane;        // this thread's keys: at + 32 k of the CTA's
    int key[K], val[K], rank[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = me * kOwn + at + 32 * k;
        val[k] = i;
        key[k] = -1;
        if (i < tokens) {
            const int id = ids[i];
            if (id >= vocab) set_status(status, FP8_ERR_INVALID_ARG);
            key[k] = sort_key(id, vocab);
        }
    }
    for (int p = 0; p < passes; ++p) {
        const int shift = p * kDigitBits;
        int *tot = m.tot[p & 1];
        for (int i = t; i < kClusterWarps * kDigits / 2; i += kClusterThreads) reinterpret_cast<int *>(m.cnt)[i] = 0;
        __syncthreads();
        rank_keys<K, CLUSTER>(key, shift, m.cnt[warp], rank);
        __syncthreads();
        int n = 0;
        if (t < kDigits) {      // a thread per digit: exclusive over the warps
#pragma unroll 8
            for (int w = 0; w < kClusterWarps; ++w) {
                const int c = m.cnt[w][t];
                m.cnt[w][t] = (uint16_t)n;
                n += c;
            }
            tot[t] = n;
        }
        if (CLUSTER) cluster_sync();
        int before = 0, all = n;
        if (CLUSTER && t < kDigits) {       // the CTAs before this one, and all of them
            all = 0;
#pragma unroll
            for (int c = 0; c < kClusterCtas; ++c) {
                const int of = c < ctas ? ld_cluster(cluster_addr(&tot[t], c)) : 0;
                all += of;
                before += c < me ? of : 0;
            }
        }
        int sum = all, mine = n;        // exclusive over the digits: all CTAs' keys, and this one's
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += u;
            if (CLUSTER) {
                const int v = __shfl_up_sync(0xffffffffu, mine, o);
                if (lane >= o) mine += v;
            }
        }
        if (lane == 31) {
            m.sums[0][warp] = sum;
            m.sums[1][warp] = mine;
        }
        __syncthreads();
        if (t < kDigits) {
            int base = sum - all + before, own = mine - n;
            for (int w = 0; w < warp; ++w) {
                base += m.sums[0][w];
                own += m.sums[1][w];
            }
            m.start[t] = CLUSTER ? base - own : base;
            m.own[t] = own;
        }
        __syncthreads();
        const bool last = p + 1 == passes;
        if (CLUSTER) {
            int2 *sorted = m.held[(p + 1) & 1];     // the pass before has been read out of it
            const int count = min(kOwn, max(0, tokens - me * kOwn));
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (key[k] < 0) continue;
                const int d = (key[k] >> shift) & (kDigits - 1);
                sorted[m.own[d] + m.cnt[warp][d] + rank[k]] = make_int2(key[k], val[k]);
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int i = t + k * kClusterThreads;
                if (i >= count) break;
                const int2 h = sorted[i];
                const int to = m.start[(h.x >> shift) & (kDigits - 1)] + i;
                if (last) emit(to, h.x, h.y);
                else st_cluster(cluster_addr(&m.held[p & 1][to % kOwn], to / kOwn), h.x, h.y);
            }
            cluster_sync();     // the keys are there; nobody still reads this CTA's counts
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (key[k] < 0) continue;
                const int d = (key[k] >> shift) & (kDigits - 1), to = m.start[d] + m.cnt[warp][d] + rank[k];
                if (last) emit(to, key[k], val[k]);
                else m.held[p & 1][to] = make_int2(key[k], val[k]);
            }
            __syncthreads();
        }
        if (last) break;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int2 h = m.held[p & 1][at + 32 * k];
            const bool in = me * kOwn + at + 32 * k < tokens;
            key[k] = in ? h.x : -1;
            val[k] = h.y;
        }
    }
}

// The first cluster sorts.  The CTAs behind it meanwhile clear dw where it is not
// added to (the rows that have tokens too, which are not known yet: they are
// written twice, but the sort of 32768 tokens is hidden).
struct ClearArgs {
    uint4 *dw;
    int64_t rows, ld;       // ld, n: vectors of a row and of its part that is cleared
    int n;
};

template <int K>
__global__ void __launch_bounds__(kClusterThreads) k_sort_cluster(const int32_t *__restrict__ ids, int tokens, int vocab, int passes, int ctas,
                                                                ClearArgs clear, int32_t *__restrict__ keys_out, int32_t *__restrict__ vals_out,
                                                                int *status)
{
    extern __shared__ __align__(16) uint8_t raw[];
    dependency_wait();
    if ((int)blockIdx.x >= ctas) {
        const int warps = (gridDim.x - ctas) * kClusterWarps;
        for (int64_t r = (blockIdx.x - ctas) * kClusterWarps + (threadIdx.x >> 5); r < clear.rows; r += warps)
            for (int v = threadIdx.x & 31; v < clear.n; v += 32)
                if (dbg_cell(r, v, 1, clear.rows, clear.ld, status)) clear.dw[r * clear.ld + v] = make_uint4(0, 0, 0, 0);
        return;
    }
    sort_cluster<K, true>(*reinterpret_cast<ClusterSort<K> *>(raw), ids, tokens, vocab, passes, ctas, (int)blockIdx.x, status,
                    [&](int to, int key, int val) {
                        if (!dbg_span(to, 1, tokens, status)) return;
                        keys_out[to] = key;
                        vals_out[to] = val;
                    });
}

// More tokens: through memory, a kernel that counts, then one a digit that places the keys,
// and before it one that adds the counts up where there are many: every placing CTA doing
// so for itself costs the square of the tokens, but spares a launch (D 8, two digits:
// 114689 tokens 51 us, with the launches 59; 150001 61 and 65; 170001 84 and 66; 2^24
// 225 ms and 1.8).
constexpr int kSortThreads = 256, kSortKeys = 8, kSortTile = kSortThreads * kSortKeys;   // keys of one CTA
static_assert(kDigits == 2 * kSortThreads, "two digits a thread");
constexpr int kScanBlocks = 76;     // more blocks' counts are added up by k_sort_scan
// Counts of a digit lie this far from the next one's: not a power of two, whose loads would all meet in few banks of the L2.
__host__ __device__ constexpr int count_stride(int blocks) { return blocks | 1; }

// counts[digit][block] of the first digit; the other digits' are cleared.
__global__ void __launch_bounds__(kSortThreads) k_sort_count(const int32_t *__restrict__ ids, int tokens, int vocab, int *__restrict__ counts,
                                                           int passes, int *status)
{
    __shared__ int n[kDigits];
    dependents_launch();
    dependency_wait();
    for (int i = threadIdx.x; i < kDigits; i += kSortThreads) n[i] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSortKeys; ++k) {
        const int i = blockIdx.x * kSortTile + k * kSortThreads + threadIdx.x;
        if (i >= tokens) break;
        if (ids[i] >= vocab) set_status(status, FP8_ERR_INVALID_ARG);
        atomicAdd(&n[sort_key(ids[i], vocab) & (kDigits - 1)], 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kDigits; i += kSortThreads) {
        counts[(int64_t)i * count_stride(gridDim.x) + blockIdx.x] = n[i];
        for (int p = 1; p < passes; ++p) counts[((int64_t)p * kDigits + i) * count_stride(gridDim.x) + blockIdx.x] = 0;
    }
}

// A CTA for every digit: its counts become what the blocks before have of it, totals[digit]
// what all have.
__global__ void __launch_bounds__(kSortThreads) k_sort_scan(int *__restrict__ counts, int blocks, int *__restrict__ totals, int *status)
{
    constexpr int kWarps = kSortThreads / 32;
    __shared__ int warp_sums[kWarps];
    dependents_launch();
    dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int *c = counts + (int64_t)blockIdx.x * count_stride(blocks);
    int before = 0;
    for (int b0 = 0; b0 < blocks; b0 += kSortThreads) {
        const int b = b0 + threadIdx.x, n = b < blocks ? c[b] : 0;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += u;
        }
        __syncthreads();        // the round before has read its sums
        if (lane == 31) warp_sums[warp] = sum;
        __syncthreads();
        int all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            sum += w < warp ? warp_sums[w] : 0;
            all += warp_sums[w];
        }
        if (b < blocks) c[b] = before + sum - n;
        before += all;
    }
    if (threadIdx.x == 0 && dbg_span(blockIdx.x, 1, kDigits, status)) totals[blockIdx.x] = before;
}

// Places every key behind the equal digits before it.  Without totals each CTA adds the
// counts up for itself.  The next digit is counted for the block that a key goes to (whole
// numbers: the atomics' order changes nothing).
__global__ void __launch_bounds__(kSortThreads) k_sort_place(const int32_t *__restrict__ keys, const int32_t *__restrict__ vals, int tokens,
                                                           int vocab, int shift, const int *__restrict__ counts, const int *__restrict__ totals,
                                                           int *__restrict__ next_counts, int32_t *__restrict__ keys_out,
                                                           int32_t *__restrict__ vals_out, int *status)
{
    constexpr int kWarps = kSortThreads / 32;
    __shared__ int n[kWarps][kDigits];
    __shared__ int warp_sums[kWarps];
    dependents_launch();
    dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, blocks = gridDim.x;
    for (int i = threadIdx.x; i < kWarps * kDigits; i += kSortThreads) n[i / kDigits][i % kDigits] = 0;
    __syncthreads();
    int key[kSortKeys], rank[kSortKeys];
    const int i0 = blockIdx.x * kSortTile + warp * 32 * kSortKeys + lane;
#pragma unroll
    for (int k = 0; k < kSortKeys; ++k) {
        const int i = i0 + 32 * k;
        key[k] = i < tokens ? (vals ? keys[i] : sort_key(keys[i], vocab)) : -1;
    }
    // this thread's digits 2t, 2t + 1: keys of the blocks before this one, and of all
    int before[2], total[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int *c = counts + (int64_t)(2 * threadIdx.x + h) * count_stride(blocks);
        if (totals) {
            before[h] = c[blockIdx.x];
            total[h] = totals[2 * threadIdx.x + h];
            continue;
        }
        before[h] = total[h] = 0;
#pragma unroll 8
        for (int b = 0; b < blocks; ++b) {
            total[h] += c[b];
            before[h] += b < (int)blockIdx.x ? c[b] : 0;
        }
    }
    rank_keys<kSortKeys, true>(key, shift, n[warp], rank);
    int start = total[0] + total[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, start, o);
        if (lane >= o) start += u;
    }
    if (lane == 31) warp_sums[warp] = start;
    __syncthreads();
    start -= total[0] + total[1];
    for (int w = 0; w < warp; ++w) start += warp_sums[w];
#pragma unroll
    for (int h = 0; h < 2; ++h) {       // exclusive over the warps, from the block's start
        const int d = 2 * threadIdx.x + h;
        int at = start + before[h];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int c = n[w][d];
            n[w][d] = at;
            at += c;
        }
        start += total[h];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSortKeys; ++k) {
        const int at = key[k] < 0 ? -1 : n[warp][(key[k] >> shift) & (kDigits - 1)] + rank[k], i = i0 + 32 * k;
        if (at >= 0 && dbg_span(at, 1, tokens, status)) {
            keys_out[at] = key[k];
            vals_out[at] = vals ? vals[i] : i;
        }
        if (next_counts) {      // one addition for the lanes of one digit and block: a frequent id has thousands
            const int d = (key[k] >> (shift + kDigitBits)) & (kDigits - 1), block = at / kSortTile;
            const unsigned same = __match_any_sync(0xffffffffu, at < 0 ? -1 : block << kDigitBits | d);
            if (at >= 0 && lane == __ffs(same) - 1) atomicAdd(&next_counts[(int64_t)d * count_stride(blocks) + block], __popc(same));
        }
    }
}

// ---------------------------------------------------------------------------
// Backward, sums over the sorted tokens.  They are cut into equal pieces, so many
// that a warp for 256 columns of each fills the GPU once (pieces of 32 took more
// than two rounds of warps, the last one mostly empty, and left more runs that
// reach over pieces: 43 us of 137 at 32768 x 128000 x 2048).
// ---------------------------------------------------------------------------
constexpr int kSumWarps = 24;       // an SM holds, by their registers

struct EmbedSumArgs {
    const int32_t *keys, *vals;     // sorted
    const uint16_t *dout;
    void *dw;
    float *part;                    // [pieces][2][dim]: sums of runs that begin before a piece, and that reach beyond it
    int64_t lddo, lddw;
    int tokens, vocab, dim, piece, pieces, segs;
    float scale;
    int *status;
};

enum { SUM_F32 = 0, SUM_ADD = 1, SUM_BF16 = 2 };

// a, times scale, to row v of dw.  SUM_ADD: added by the L2 (one addition an
// element and call, so its order is not in question), which spares the round
// trip of reading it here.
template <int OUT>
__device__ __forceinline__ void store_row8(const EmbedSumArgs &g, int64_t v, int col, const float (&a)[8])
{
    if (!dbg_span(v * g.lddw + col, 8, (int64_t)(g.vocab - 1) * g.lddw + g.dim, g.status)) return;
    const float s = g.scale;
    if (OUT == SUM_BF16) {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(g.dw) + v * g.lddw + col) =
            make_uint4(bf16x2_rn(a[0] * s, a[1] * s), bf16x2_rn(a[2] * s, a[3] * s), bf16x2_rn(a[4] * s, a[5] * s), bf16x2_rn(a[6] * s, a[7] * s));
        return;
    }
    float *p = static_cast<float *>(g.dw) + v * g.lddw + col;
    if (OUT == SUM_ADD) {
#pragma unroll
        for (int h = 0; h < 8; h += 4)
            asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p + h), "f"(a[h] * s), "f"(a[h + 1] * s),
                         "f"(a[h + 2] * s), "f"(a[h + 3] * s)
                         : "memory");
        return;
    }
    reinterpret_cast<float4 *>(p)[0] = make_float4(a[0] * s, a[1] * s, a[2] * s, a[3] * s);
    reinterpret_cast<float4 *>(p)[1] = make_float4(a[4] * s, a[5] * s, a[6] * s, a[7] * s);
}

// One warp sums 256 columns of one piece, 8 rows' loads in flight.  A run of
// equal ids inside the piece goes to dw, one that reaches beyond it to the
// workspace.
template <int OUT>
__global__ void __launch_bounds__(256, 3) k_embedding_sums(EmbedSumArgs g)
{
    dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t item = (int64_t)blockIdx.x * 8 + warp;
    const int piece = (int)(item / g.segs), col = (int)(item - (int64_t)piece * g.segs) * 256 + lane * 8;
    if (piece >= g.pieces) return;
    const int a = piece * g.piece, end = min(a + g.piece, g.tokens);
    const int prev = a > 0 ? g.keys[a - 1] : -1, next = end < g.tokens ? g.keys[end] : -1;
    const bool in = col < g.dim;
    float acc[8] = {};
    auto fetch = [&](int i, int &key, int &tok, int &after) {   // token i and the one behind it in the piece
        key = i < end ? g.keys[i] : g.vocab;
        tok = i < end ? g.vals[i] : 0;
        after = i + 1 < end ? g.keys[i + 1] : -1;
    };
    int key, tok, after;
    fetch(a + lane, key, tok, after);
    for (int b = a; b < end; b += 32) {
        int key2, tok2, after2;
        fetch(b + 32 + lane, key2, tok2, after2);
        // this lane's token ends its run in the piece; the run reaches back, or on
        const unsigned ends = __ballot_sync(0xffffffffu, key < g.vocab && after != key);
        const unsigned back = __ballot_sync(0xffffffffu, key == prev), on = __ballot_sync(0xffffffffu, b + lane == end - 1 && key == next);
#pragma unroll 1
        for (int i0 = 0; i0 < 32 && b + i0 < end; i0 += 8) {
            uint4 x[8];
            int kk[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                kk[k] = __shfl_sync(0xffffffffu, key, i0 + k);
                const int tt = __shfl_sync(0xffffffffu, tok, i0 + k);
                x[k] = in && kk[k] < g.vocab ? ldg_stream(g.dout + (int64_t)tt * g.lddo + col) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int i = i0 + k;
                if (kk[k] >= g.vocab) return;      // the tokens without an id are the last
                const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[2 * e] += bf16_lo(w[e]);
                    acc[2 * e + 1] += bf16_hi(w[e]);
                }
                if (!(ends >> i & 1)) continue;
                if (in && !((back | on) >> i & 1)) {
                    store_row8<OUT>(g, kk[k], col, acc);
                } else if (in) {
                    const int64_t at = ((int64_t)piece * 2 + (back >> i & 1 ? 0 : 1)) * g.dim + col;
                    if (dbg_span(at, 8, (int64_t)g.pieces * 2 * g.dim, g.status)) {
                        *reinterpret_cast<float4 *>(g.part + at) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                        *reinterpret_cast<float4 *>(g.part + at + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
            }
        }
        key = key2;
        tok = tok2;
        after = after2;
    }
}

// The runs that reach over pieces: the piece where one begins owns it.  A warp
// looks at one piece for 256 columns, and adds up an owned run of up to
// kJoinAlone pieces by itself, in order; of a longer one the CTA's 8 warps take
// every 8th piece each, and their sums are added in order.
constexpr int kJoinAlone = 16;

template <int OUT>
__global__ void __launch_bounds__(256) k_embedding_joins(EmbedSumArgs g)
{
    __shared__ int run_last[8];         // last piece of the long run that piece w owns, or -1
    __shared__ float sums[8][256];
    dependents_launch();
    dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int p0 = blockIdx.x * 8, col = blockIdx.y * 256 + lane * 8;
    const bool in = col < g.dim;
    // the run is its first piece's last, and every other piece's first
    auto add_pieces = [&](float (&acc)[8], int p, int r0, int last, int step) {
        if (!in) return;
#pragma unroll 4
        for (int r = r0; r <= last; r += step) {
            const float4 *src = reinterpret_cast<const float4 *>(g.part + ((int64_t)r * 2 + (r == p ? 1 : 0)) * g.dim + col);
            const float4 x = src[0], y = src[1];
            acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
            acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
        }
    };
    {
        int last = -1;
        const int p = p0 + warp, end = (p + 1) * g.piece;    // one behind the piece's last token
        if (p < g.pieces && end < g.tokens) {
            const int key = g.keys[end - 1], then = g.keys[end], before = p > 0 ? g.keys[end - g.piece - 1] : -1;
            // it begins here unless the whole piece, and the token before it, has this id
            if (key < g.vocab && then == key && before != key) {
                for (last = p;;) {      // pieces that begin with it follow one another
                    const int q = last + 1 + lane;
                    const unsigned same = __ballot_sync(0xffffffffu, q < g.pieces && g.keys[q * g.piece] == key);
                    last += same == 0xffffffffu ? 32 : __ffs(~same) - 1;
                    if (same != 0xffffffffu) break;
                }
                if (last - p < kJoinAlone) {
                    float acc[8] = {};
                    add_pieces(acc, p, p, last, 1);
                    if (in) store_row8<OUT>(g, key, col, acc);
                    last = -1;
                }
            }
        }
        if (lane == 0) run_last[warp] = last;
    }
    __syncthreads();
    for (int w = 0; w < 8; ++w) {
        const int p = p0 + w, last = run_last[w];
        if (last < 0) continue;
        float acc[8] = {};
        add_pieces(acc, p, p + warp, last, 8);
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[warp][e * 32 + lane] = acc[e];
        __syncthreads();
        if (warp == 0 && in) {
            const int v = g.keys[(p + 1) * g.piece - 1];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                for (int o = 1; o < 8; ++o) acc[e] += sums[o][e * 32 + lane];
            store_row8<OUT>(g, v, col, acc);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Backward of few tokens in one launch: every CTA sorts all of them for itself
// (2 keys a thread, in its shared memory) and then sums 32 columns: 4 lanes take
// a piece of 8 sorted tokens, and the runs that reach over pieces are added up
// from shared memory (1000 x 1024: 10 us, three launches of the form above 16).
// ---------------------------------------------------------------------------
constexpr int kSmallKeys = 2, kSmallMost = kSmallKeys * kClusterThreads, kSmallPieces = kSmallMost / 8;

static_assert(sizeof(ClusterSort<kSmallKeys>) % 16 == 0, "16-byte vectors follow");

struct SmallEmbed {
    ClusterSort<kSmallKeys> sort;
    int2 sorted[kSmallMost + 1];            // key, token; behind the last: -1
    alignas(16) float part[kSmallPieces][2][32];
};

template <int OUT>
__global__ void __launch_bounds__(kClusterThreads) k_embedding_small(const int32_t *__restrict__ ids, int passes, EmbedSumArgs g)
{
    extern __shared__ __align__(16) uint8_t raw[];
    SmallEmbed &m = *reinterpret_cast<SmallEmbed *>(raw);
    dependents_launch();
    dependency_wait();
    sort_cluster<kSmallKeys, false>(m.sort, ids, g.tokens, g.vocab, passes, 1, 0, g.status, [&](int to, int key, int val) { m.sorted[to] = make_int2(key, val); });
    if (threadIdx.x == 0) m.sorted[g.tokens] = make_int2(-1, 0);
    __syncthreads();

    const int piece = threadIdx.x >> 2, c = (threadIdx.x & 3) * 8, col = blockIdx.x * 32 + c, a = piece * 8;
    const int n = min(8, g.tokens - a);     // may be negative
    const bool in = col < g.dim;
    const int prev = a > 0 && n > 0 ? m.sorted[a - 1].x : -1;
    auto add8 = [](float (&x)[8], const float4 *p) {
        const float4 u = p[0], v = p[1];
        x[0] += u.x; x[1] += u.y; x[2] += u.z; x[3] += u.w;
        x[4] += v.x; x[5] += v.y; x[6] += v.z; x[7] += v.w;
    };
    {
        uint4 x[8];
        int key[9];
#pragma unroll
        for (int k = 0; k < 9; ++k) key[k] = k <= n ? m.sorted[a + k].x : -1;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const bool use = k < n && in && key[k] < g.vocab;
            x[k] = use ? ldg_stream(g.dout + (int64_t)m.sorted[a + k].y * g.lddo + col) : make_uint4(0, 0, 0, 0);
        }
        float acc[8] = {};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k >= n || key[k] >= g.vocab) break;
            const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc[2 * e] += bf16_lo(w[e]);
                acc[2 * e + 1] += bf16_hi(w[e]);
            }
            const bool on = key[k + 1] == key[k];
            if (on && k + 1 < n) continue;
            // the run ends here, or with the piece
            if (!on && key[k] != prev) {
                if (in) store_row8<OUT>(g, key[k], col, acc);
            } else {
                float4 *p = reinterpret_cast<float4 *>(&m.part[piece][key[k] == prev ? 0 : 1][c]);
                p[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
                p[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
        }
    }
    __syncthreads();
    if (n < 8 || !in) return;       // the last piece owns no run that goes on
    const int key = m.sorted[a + 7].x;
    if (key >= g.vocab || key == prev || m.sorted[a + 8].x != key) return;
    float acc[8] = {};
    add8(acc, reinterpret_cast<const float4 *>(&m.part[piece][1][c]));
    for (int q = a + 8; q < g.tokens && m.sorted[q].x == key; q += 8) add8(acc, reinterpret_cast<const float4 *>(&m.part[q / 8][0][c]));
    store_row8<OUT>(g, key, col, acc);
}

// ------------------------------------------------------------------ launchers

namespace {

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

struct EmbedLayout {    // byte offsets in the workspace
    int64_t keys[2], vals[2], counts, totals, part, bytes;
    int blocks, passes, piece, pieces;
    EmbedLayout(int64_t tokens, int64_t vocab, int64_t dim)
    {
        blocks = (int)((tokens + kSortTile - 1) / kSortTile);
        int bits = 1;       // of the largest key, which is vocab itself
        while ((vocab >> bits) != 0) ++bits;
        passes = (bits + kDigitBits - 1) / kDigitBits;
        const int64_t warps = (int64_t)sm_count() * kSumWarps, segs = (dim + 255) / 256;
        piece = (int)std::max<int64_t>(8, up((tokens * segs + warps - 1) / warps, 8));
        pieces = (int)((tokens + piece - 1) / piece);
        // pieces * dim of this call and of every smaller one: there are at most warps / segs + 1 pieces, and dim <= 256 segs
        const int64_t most = std::min((tokens + 7) / 8 * dim, warps * 256 + dim);
        int64_t at = 0;
        auto take = [&](int64_t n) { const int64_t p = at; at += up(n, 16); return p; };
        for (int i = 0; i < 2; ++i) {
            keys[i] = take(tokens * 4);
            vals[i] = take(tokens * 4);
        }
        counts = take(tokens <= kClusterMost ? 0 : (int64_t)passes * kDigits * count_stride(blocks) * 4);
        totals = take(tokens <= kClusterMost ? 0 : kDigits * 4);
        part = take(most * 2 * 4);
        bytes = at;
    }
};

template <typename K>
int allow_smem(K kernel, int bytes)
{
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

template <int K>
int run_sort_cluster(const int32_t *ids, int tokens, int vocab, int passes, int ctas, const ClearArgs &clear, int32_t *keys, int32_t *vals,
                     int *status, cudaStream_t st)
{
    static bool attr_done[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (!attr_done[dev & 63]) {
        const int rc = allow_smem(k_sort_cluster<K>, (int)sizeof(ClusterSort<K>));
        if (rc != FP8_OK) return rc;
        attr_done[dev & 63] = true;
    }
    const int64_t clearing = clear.dw ? std::min<int64_t>((clear.rows + kClusterWarps - 1) / kClusterWarps, (int64_t)sm_count() * 2) : 0;
    const unsigned grid = (unsigned)(ctas + (clearing + ctas - 1) / ctas * ctas);
    return launch_dependent_cluster(k_sort_cluster<K>, dim3(grid), (unsigned)ctas, kClusterThreads, sizeof(ClusterSort<K>), st, ids, tokens, vocab,
                                    passes, ctas, clear, keys, vals, status);
}

// The most CTAs with a key a thread first: the passes' rounds are what takes time.
int run_sort(const int32_t *ids, int tokens, int vocab, int passes, const ClearArgs &clear, int32_t *keys, int32_t *vals, int *status,
             cudaStream_t st)
{
    int ctas = 1;
    while (ctas < kClusterCtas && ctas * kClusterThreads < tokens) ctas *= 2;
    const int per = (tokens + ctas * kClusterThreads - 1) / (ctas * kClusterThreads);
    if (per <= 1) return run_sort_cluster<1>(ids, tokens, vocab, passes, ctas, clear, keys, vals, status, st);
    if (per <= 2) return run_sort_cluster<2>(ids, tokens, vocab, passes, ctas, clear, keys, vals, status, st);
    if (per <= 4) return run_sort_cluster<4>(ids, tokens, vocab, passes, ctas, clear, keys, vals, status, st);
    return run_sort_cluster<8>(ids, tokens, vocab, passes, ctas, clear, keys, vals, status, st);
}

template <int OUT>
int embed_small(const int32_t *ids, int passes, const EmbedSumArgs &g, cudaStream_t st)
{
    static bool attr_done[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (!attr_done[dev & 63]) {
        const int rc = allow_smem(k_embedding_small<OUT>, (int)sizeof(SmallEmbed));
        if (rc != FP8_OK) return rc;
        attr_done[dev & 63] = true;
    }
    return launch_dependent(k_embedding_small<OUT>, dim3((unsigned)((g.dim + 31) / 32)), kClusterThreads, sizeof(SmallEmbed), st, ids, passes, g);
}

template <int OUT>
int embed_sums(EmbedSumArgs &g, cudaStream_t st)
{
    const int64_t ctas = ((int64_t)g.pieces * g.segs + 7) / 8;
    if (ctas >= (int64_t)1 << 31) return FP8_ERR_SHAPE;
    const int rc = launch_dependent(k_embedding_sums<OUT>, dim3((unsigned)ctas), 256, 0, st, g);
    if (rc != FP8_OK) return rc;
    return launch_dependent(k_embedding_joins<OUT>, dim3((unsigned)((g.pieces + 7) / 8), (unsigned)g.segs), 256, 0, st, g);
}

}  // namespace

size_t embedding_workspace_bytes(int64_t tokens, int64_t vocab, int64_t dim) { return (size_t)EmbedLayout(tokens, vocab, dim).bytes; }

int launch_embedding_fwd(const int32_t *ids, int64_t tokens, const void *w, int64_t vocab, int64_t dim, int64_t ldw, float scale, void *out,
                         int64_t ldo, int *status, cudaStream_t st)
{
    const int nv = (int)(dim / 8), segs = (nv + 127) / 128;
    const int64_t blocks = (tokens * segs + 7) / 8;
    if (blocks >= (int64_t)1 << 31) return FP8_ERR_SHAPE;
    return launch_dependent(k_embedding_fwd, dim3((unsigned)blocks), 256, 0, st, ids, tokens, static_cast<const uint16_t *>(w), vocab, ldw, nv,
                            segs, scale, static_cast<uint16_t *>(out), ldo, status);
}

int launch_embedding_bwd(const int32_t *ids, int64_t tokens, const void *dout, int64_t lddo, int64_t vocab, int64_t dim, float scale, void *dw,
                         int out_dtype, int64_t lddw, int accumulate, void *ws, int *status, cudaStream_t st)
{
    const bool f32 = out_dtype == FP8_OUT_F32;
    const int esz = f32 ? 4 : 2;
    auto clear = [&] {
        if (lddw == dim) return cudaMemsetAsync(dw, 0, (size_t)(vocab * dim * esz), st) == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
        return cudaMemset2DAsync(dw, (size_t)lddw * esz, 0, (size_t)dim * esz, (size_t)vocab, st) == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
    };
    if (tokens == 0) return accumulate ? FP8_OK : clear();
    const EmbedLayout L(tokens, vocab, dim);
    const int n = (int)tokens, V = (int)vocab;
    uint8_t *base = static_cast<uint8_t *>(ws);
    int32_t *keys[2], *vals[2];
    for (int i = 0; i < 2; ++i) {
        keys[i] = reinterpret_cast<int32_t *>(base + L.keys[i]);
        vals[i] = reinterpret_cast<int32_t *>(base + L.vals[i]);
    }
    EmbedSumArgs g{};
    g.dout = static_cast<const uint16_t *>(dout);
    g.dw = dw;
    g.part = reinterpret_cast<float *>(base + L.part);
    g.lddo = lddo;
    g.lddw = lddw;
    g.tokens = n;
    g.vocab = V;
    g.dim = (int)dim;
    g.piece = L.piece;
    g.pieces = L.pieces;
    g.segs = (int)((dim + 255) / 256);
    g.scale = scale;
    g.status = status;
    if (g.segs > 65535) return FP8_ERR_SHAPE;
    int rc, sorted = 0;
    if (n <= kSmallMost) {
        if (!accumulate && (rc = clear()) != FP8_OK) return rc;
        return !f32 ? embed_small<SUM_BF16>(ids, L.passes, g, st)
                    : accumulate ? embed_small<SUM_ADD>(ids, L.passes, g, st) : embed_small<SUM_F32>(ids, L.passes, g, st);
    }
    if (n <= kClusterMost) {
        ClearArgs c{};
        if (!accumulate) {
            c.dw = static_cast<uint4 *>(dw);
            c.rows = vocab;
            c.ld = lddw * esz / 16;
            c.n = (int)(dim * esz / 16);
        }
        if ((rc = run_sort(ids, n, V, L.passes, c, keys[0], vals[0], status, st)) != FP8_OK) return rc;
    } else {
        if (!accumulate && (rc = clear()) != FP8_OK) return rc;
        int *counts = reinterpret_cast<int *>(base + L.counts), *totals = reinterpret_cast<int *>(base + L.totals);
        const int64_t stride = (int64_t)kDigits * count_stride(L.blocks);
        if ((rc = launch_dependent(k_sort_count, dim3((unsigned)L.blocks), kSortThreads, 0, st, ids, n, V, counts, L.passes, status)) != FP8_OK)
            return rc;
        for (int p = 0; p < L.passes; ++p) {
            const int from = (p + 1) & 1;
            const bool scan = L.blocks > kScanBlocks;
            const int32_t *in = p == 0 ? ids : keys[from], *in_vals = p == 0 ? nullptr : vals[from];
            int *c = counts + p * stride, *next = p + 1 < L.passes ? c + stride : nullptr;
            sorted = p & 1;
            if (scan && (rc = launch_dependent(k_sort_scan, dim3(kDigits), kSortThreads, 0, st, c, L.blocks, totals, status)) != FP8_OK) return rc;
            if ((rc = launch_dependent(k_sort_place, dim3((unsigned)L.blocks), kSortThreads, 0, st, in, in_vals, n, V, p * kDigitBits,
                                       static_cast<const int *>(c), static_cast<const int *>(scan ? totals : nullptr), next, keys[sorted], vals[sorted],
                                       status)) != FP8_OK)
                return rc;
        }
    }
    g.keys = keys[sorted];
    g.vals = vals[sorted];
    return !f32 ? embed_sums<SUM_BF16>(g, st) : accumulate ? embed_sums<SUM_ADD>(g, st) : embed_sums<SUM_F32>(g, st);
}

}  // namespace fp8fg
