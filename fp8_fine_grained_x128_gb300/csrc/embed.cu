// embed.cu -- embedding lookup with scaling, and its gradient (sm_103a).
//
// Forward: out[t] = scale * w[ids[t]], a copy bound by HBM.
// Backward: dw[v] (+)= scale * sum of dout[t] over the tokens with ids[t] = v.
// Adding rows with atomics would give sums that change from run to run with
// their order; here the tokens are sorted by id (a stable radix sort, so that
// each id's tokens stay in order), and every id's rows are summed in FP32 in
// that order: by one warp per 256 columns where they lie in one piece of
// kPiece sorted tokens, else piece by piece and then over the pieces.  The
// order depends on the ids alone, so the results do too.
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
// Backward: stable radix sort of (id, token) by digits of up to 9 bits.
// Tokens without an id, or with one out of range, sort behind the vocabulary.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 256, kSortKeys = 8, kSortTile = kSortThreads * kSortKeys;   // keys of one CTA
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int kPiece = 32;      // sorted tokens of one warp's sum

__device__ __forceinline__ int sort_key(int32_t id, int vocab) { return id < 0 || id >= vocab ? vocab : id; }

// counts[digit][block]; the first pass also marks the ids that occur.
__global__ void __launch_bounds__(kSortThreads) k_sort_count(const int32_t *__restrict__ keys, int tokens, int vocab, int shift, int first,
                                                           int *__restrict__ counts, uint8_t *__restrict__ occurs, int *status)
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
        const int32_t id = keys[i];
        const int key = first ? sort_key(id, vocab) : id;
        if (first && id >= vocab) set_status(status, FP8_ERR_INVALID_ARG);
        if (occurs && key < vocab && dbg_span(key, 1, vocab, status)) occurs[key] = 1;
        atomicAdd(&n[(key >> shift) & (kDigits - 1)], 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kDigits; i += kSortThreads) counts[i * gridDim.x + blockIdx.x] = n[i];
}

// Exclusive sums of counts[0 .. n), in place, by one CTA.
__global__ void __launch_bounds__(1024) k_sort_scan(int *counts, int n)
{
    __shared__ int sums[32];
    dependents_launch();
    dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (n + 1023) / 1024, i0 = min(n, (int)threadIdx.x * per), i1 = min(n, i0 + per);
    int mine = 0;
    for (int i = i0; i < i1; ++i) mine += counts[i];
    int v = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    int before = v - mine;
    for (int w = 0; w < warp; ++w) before += sums[w];
    for (int i = i0; i < i1; ++i) {
        const int c = counts[i];
        counts[i] = before;
        before += c;
    }
}

// Places every key behind the equal digits before it.  A warp ranks 32 * 8
// consecutive keys, 32 at a time: lanes of equal digits find one another by a
// match, and the warp's counter of that digit holds how many came before.
__global__ void __launch_bounds__(kSortThreads) k_sort_place(const int32_t *__restrict__ keys, const int32_t *__restrict__ vals, int tokens,
                                                           int vocab, int shift, int first, const int *__restrict__ starts,
                                                           int32_t *__restrict__ keys_out, int32_t *__restrict__ vals_out, int *status)
{
    constexpr int kWarps = kSortThreads / 32;
    __shared__ int n[kWarps][kDigits];
    dependents_launch();
    dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < kWarps * kDigits; i += kSortThreads) n[i / kDigits][i % kDigits] = 0;
    __syncthreads();
    int key[kSortKeys], rank[kSortKeys];
    const int i0 = blockIdx.x * kSortTile + warp * 32 * kSortKeys + lane;
#pragma unroll
    for (int k = 0; k < kSortKeys; ++k) {
        const int i = i0 + 32 * k;
        key[k] = i < tokens ? (first ? sort_key(keys[i], vocab) : keys[i]) : -1;
    }
#pragma unroll
    for (int k = 0; k < kSortKeys; ++k) {
        const int d = key[k] < 0 ? kDigits : (key[k] >> shift) & (kDigits - 1);
        const unsigned same = __match_any_sync(0xffffffffu, d);
        const int before = d < kDigits ? n[warp][d] : 0;
        rank[k] = before + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (d < kDigits && lane == __ffs(same) - 1) n[warp][d] = before + __popc(same);
        __syncwarp();
    }
    __syncthreads();
    for (int d = threadIdx.x; d < kDigits; d += kSortThreads) {     // exclusive over the warps, from the block's start
        int at = starts[d * gridDim.x + blockIdx.x];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int c = n[w][d];
            n[w][d] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSortKeys; ++k) {
        if (key[k] < 0) continue;
        const int at = n[warp][(key[k] >> shift) & (kDigits - 1)] + rank[k], i = i0 + 32 * k;
        if (!dbg_span(at, 1, tokens, status)) continue;
        keys_out[at] = key[k];
        vals_out[at] = first ? i : vals[i];
    }
}

// ---------------------------------------------------------------------------
// The sums over the sorted tokens.
// ---------------------------------------------------------------------------
struct EmbedSumArgs {
    const int32_t *keys, *vals;     // sorted
    const uint16_t *dout;
    const uint8_t *occurs;          // accumulate = 0: the ids that have tokens
    void *dw;
    float *part;                    // [pieces][2][dim]: sums of a piece's first and last run that reach beyond it
    int64_t lddo, lddw;
    int tokens, vocab, dim, pieces, segs;
    unsigned sum_ctas;
    float scale;
    int accumulate;
    int *status;
};

template <bool F32>
__device__ __forceinline__ void store_row8(const EmbedSumArgs &g, int64_t v, int col, const float (&a)[8])
{
    if (!dbg_span(v * g.lddw + col, 8, (int64_t)(g.vocab - 1) * g.lddw + g.dim, g.status)) return;
    if (F32) {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(g.dw) + v * g.lddw + col);
        float4 x = make_float4(a[0], a[1], a[2], a[3]), y = make_float4(a[4], a[5], a[6], a[7]);
        if (g.accumulate) {
            const float4 p0 = p[0], p1 = p[1];
            x = make_float4(p0.x + x.x, p0.y + x.y, p0.z + x.z, p0.w + x.w);
            y = make_float4(p1.x + y.x, p1.y + y.y, p1.z + y.z, p1.w + y.w);
        }
        p[0] = x;
        p[1] = y;
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(g.dw) + v * g.lddw + col) =
            make_uint4(bf16x2_rn(a[0], a[1]), bf16x2_rn(a[2], a[3]), bf16x2_rn(a[4], a[5]), bf16x2_rn(a[6], a[7]));
    }
}

// One warp sums 256 columns of one piece, 8 rows' loads in flight.  A run of
// equal ids that lies inside the piece goes to dw; one that reaches beyond its
// first or last token goes to the workspace.  The CTAs behind the pieces'
// write zeros to the rows without tokens.
template <bool F32>
__global__ void __launch_bounds__(256) k_embedding_sums(EmbedSumArgs g)
{
    dependents_launch();
    dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x >= g.sum_ctas) {
        const float zero[8] = {};
        const int stride = (gridDim.x - g.sum_ctas) * 8;
        for (int v = (blockIdx.x - g.sum_ctas) * 8 + warp; v < g.vocab; v += stride)
            if (!g.occurs[v])
                for (int col = lane * 8; col < g.dim; col += 256) store_row8<F32>(g, v, col, zero);
        return;
    }
    const int64_t item = (int64_t)blockIdx.x * 8 + warp;
    const int piece = (int)(item / g.segs), col = (int)(item - (int64_t)piece * g.segs) * 256 + lane * 8;
    if (piece >= g.pieces) return;
    const int a = piece * kPiece, n = min(kPiece, g.tokens - a);
    const int key = lane < n ? g.keys[a + lane] : g.vocab, tok = lane < n ? g.vals[a + lane] : 0;
    const int prev = a > 0 ? g.keys[a - 1] : -1, next = a + n < g.tokens ? g.keys[a + n] : -1;
    const bool in = col < g.dim;
    float acc[8] = {};
    bool first = true;
    for (int i0 = 0; i0 < n; i0 += 8) {
        uint4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int kk = __shfl_sync(0xffffffffu, key, i0 + k), tt = __shfl_sync(0xffffffffu, tok, i0 + k);
            x[k] = in && kk < g.vocab ? ldg_stream(g.dout + (int64_t)tt * g.lddo + col) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + k;
            const int kk = __shfl_sync(0xffffffffu, key, i);
            const int then = i + 1 < kPiece ? __shfl_sync(0xffffffffu, key, (i + 1) & 31) : -2;
            if (kk >= g.vocab) return;      // the tokens without an id are the last
            const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc[2 * e] += bf16_lo(w[e]);
                acc[2 * e + 1] += bf16_hi(w[e]);
            }
            if (i + 1 < n && then == kk) continue;
            // the run ends here, or with the piece
            const bool whole = !(first && kk == prev) && !(i + 1 == n && kk == next);
            if (in) {
                if (whole) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[e] *= g.scale;
                    store_row8<F32>(g, kk, col, acc);
                } else {
                    const int64_t at = ((int64_t)piece * 2 + (first && kk == prev ? 0 : 1)) * g.dim + col;
                    if (dbg_span(at, 8, (int64_t)g.pieces * 2 * g.dim, g.status)) {
                        *reinterpret_cast<float4 *>(g.part + at) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                        *reinterpret_cast<float4 *>(g.part + at + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
            first = false;
        }
    }
}

// The runs that reach over pieces: the piece where one begins owns it.  Each
// CTA looks at 8 pieces (one a warp) for 256 columns; for each owned run its 8
// warps add every 8th of the run's pieces, and their sums are added in order.
template <bool F32>
__global__ void __launch_bounds__(256) k_embedding_joins(EmbedSumArgs g)
{
    __shared__ int run_last[8];         // last piece of the run that piece w owns, or -1
    __shared__ float sums[8][256];
    dependents_launch();
    dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int p0 = blockIdx.x * 8, col = blockIdx.y * 256 + lane * 8;
    if (lane == 0) {
        int last = -1;
        const int p = p0 + warp, end = p * kPiece + kPiece;    // one behind the piece's last token
        if (end < g.tokens) {
            const int key = g.keys[end - 1];
            if (key < g.vocab && g.keys[end] == key) {
                // it begins here unless the whole piece, and the token before it, has this id
                const bool begins = p == 0 || g.keys[end - kPiece - 1] != key;
                if (begins) {
                    int lo = end, hi = g.tokens;     // first token behind the run, by bisection
                    while (lo < hi) {
                        const int mid = lo + (hi - lo) / 2;
                        if (g.keys[mid] > key) hi = mid;
                        else lo = mid + 1;
                    }
                    last = (lo - 1) / kPiece;
                }
            }
        }
        run_last[warp] = last;
    }
    __syncthreads();
    for (int w = 0; w < 8; ++w) {
        const int p = p0 + w, last = run_last[w];
        if (last < 0) continue;
        float acc[8] = {};
        if (col < g.dim) {
#pragma unroll 4
            for (int r = p + warp; r <= last; r += 8) {
                // the run is its first piece's last, and every other piece's first
                const float4 *src = reinterpret_cast<const float4 *>(g.part + ((int64_t)r * 2 + (r == p ? 1 : 0)) * g.dim + col);
                const float4 x = src[0], y = src[1];
                acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
                acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[warp][e * 32 + lane] = acc[e];
        __syncthreads();
        if (warp == 0 && col < g.dim) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                for (int v = 1; v < 8; ++v) acc[e] += sums[v][e * 32 + lane];
                acc[e] *= g.scale;
            }
            store_row8<F32>(g, g.keys[p * kPiece + kPiece - 1], col, acc);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ launchers

namespace {

int64_t up16(int64_t n) { return (n + 15) & ~(int64_t)15; }

struct EmbedLayout {    // byte offsets in the workspace
    int64_t keys[2], vals[2], counts, occurs, part, bytes;
    int blocks, pieces;
    EmbedLayout(int64_t tokens, int64_t vocab, int64_t dim)
    {
        blocks = (int)((tokens + kSortTile - 1) / kSortTile);
        pieces = (int)((tokens + kPiece - 1) / kPiece);
        int64_t at = 0;
        auto take = [&](int64_t n) { const int64_t p = at; at += up16(n); return p; };
        for (int i = 0; i < 2; ++i) keys[i] = take(tokens * 4);
        for (int i = 0; i < 2; ++i) vals[i] = take(tokens * 4);
        counts = take((int64_t)blocks * kDigits * 4);
        occurs = take(vocab);
        part = take((int64_t)pieces * 2 * dim * 4);
        bytes = at;
    }
};

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
    const int64_t row = dim * (f32 ? 4 : 2);
    if (tokens == 0) {
        if (accumulate) return FP8_OK;
        return cudaMemset2DAsync(dw, (size_t)lddw * (f32 ? 4 : 2), 0, (size_t)row, (size_t)vocab, st) == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
    }
    const EmbedLayout L(tokens, vocab, dim);
    uint8_t *base = static_cast<uint8_t *>(ws);
    int *counts = reinterpret_cast<int *>(base + L.counts);
    uint8_t *occurs = accumulate ? nullptr : base + L.occurs;
    if (occurs && cudaMemsetAsync(occurs, 0, (size_t)vocab, st) != cudaSuccess) return FP8_ERR_CUDA;
    const int n = (int)tokens;
    int bits = 1;       // of the largest key, which is vocab itself
    while ((vocab >> bits) != 0) ++bits;
    const int32_t *keys = ids, *vals = nullptr;
    int rc, to = 0;
    for (int shift = 0, first = 1; shift < bits; shift += kDigitBits, first = 0, to ^= 1) {
        int32_t *k2 = reinterpret_cast<int32_t *>(base + L.keys[to]), *v2 = reinterpret_cast<int32_t *>(base + L.vals[to]);
        if ((rc = launch_dependent(k_sort_count, dim3(L.blocks), kSortThreads, 0, st, keys, n, (int)vocab, shift, first, counts,
                                   first ? occurs : static_cast<uint8_t *>(nullptr), status)) != FP8_OK ||
            (rc = launch_dependent(k_sort_scan, dim3(1), 1024, 0, st, counts, L.blocks * kDigits)) != FP8_OK ||
            (rc = launch_dependent(k_sort_place, dim3(L.blocks), kSortThreads, 0, st, keys, vals, n, (int)vocab, shift, first,
                                   static_cast<const int *>(counts), k2, v2, status)) != FP8_OK)
            return rc;
        keys = k2;
        vals = v2;
    }
    EmbedSumArgs g{};
    g.keys = keys;
    g.vals = vals;
    g.dout = static_cast<const uint16_t *>(dout);
    g.occurs = occurs;
    g.dw = dw;
    g.part = reinterpret_cast<float *>(base + L.part);
    g.lddo = lddo;
    g.lddw = lddw;
    g.tokens = n;
    g.vocab = (int)vocab;
    g.dim = (int)dim;
    g.pieces = L.pieces;
    g.segs = (int)((dim + 255) / 256);
    g.scale = scale;
    g.accumulate = accumulate;
    g.status = status;
    const int64_t sum_ctas = ((int64_t)L.pieces * g.segs + 7) / 8;
    const int64_t zero_ctas = accumulate ? 0 : std::min<int64_t>((vocab + 7) / 8, (int64_t)sm_count() * 4);
    if (sum_ctas + zero_ctas >= (int64_t)1 << 31) return FP8_ERR_SHAPE;
    g.sum_ctas = (unsigned)sum_ctas;
    if ((rc = launch_dependent(f32 ? k_embedding_sums<true> : k_embedding_sums<false>, dim3((unsigned)(sum_ctas + zero_ctas)), 256, 0, st, g)) !=
        FP8_OK)
        return rc;
    return launch_dependent(f32 ? k_embedding_joins<true> : k_embedding_joins<false>, dim3((unsigned)((L.pieces + 7) / 8), (unsigned)g.segs), 256,
                            0, st, g);
}

}  // namespace fp8fg
