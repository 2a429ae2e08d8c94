// paged_few.cu -- attention over a paged cache when up to 32 rows (new tokens x
// query heads of a group) share a cache head: single tokens and short drafts
// (sm_103a).
//
// Bound: HBM bandwidth, every key and value read once (32 query and 8 cache heads
// of 128: 64 ragged sequences of up to 8000 BF16 keys 201 us, 0.93 of the measured
// copy rate; 16 x 65536 E4M3 keys 338 us, 0.94; one of 524287 BF16 keys 327 us,
// 0.97).  With two groups of rows and FP8 codes it is the warps' mix of
// conversions, products and softmax (about 1900 cycles a tile, three CTAs side by side, no
// unit above half its rate), and the two warps of a slice each convert all of its codes:
// 32 x 5 tokens over up to 4001 E4M3 keys 58 us against 20 us for the bytes.  Of 20 rows, 12
// places of the second group stand empty besides.
//
// All (sequence, head) pairs' tiles (64 keys with one group of rows, 32 with two) stand
// in one line that is cut into equal runs, one per
// CTA, so ragged batches and a single long cache balance alike; a CTA's run
// covers whole pairs, which it finishes alone, and at most two broken ones,
// whose partial maxima, sums and outputs go to the workspace.  The last CTA
// to announce its part of a broken pair joins the parts in order (the result
// does not depend on who is last).
//
// One group of rows: a warp takes 16 keys of each tile and never waits for another
// warp; its copies (cp.async, zero-filled past the sequence's end) go through its own
// ring.  Two groups: the two warps that share 16 keys share a ring too, one copies the
// keys and the other the values, and they meet at a named barrier every tile.
// S = Q K^T and O += P V run on m16n8k16 mma.sync; its rate is far
// from binding here (the rows are padded to 16 and the copies still take
// longer).  The contraction order over head_dim is free, so a lane reads 16
// contiguous bytes of a key as operand registers, and Q is laid out to match.
// FP8 codes become FP16 exactly (one conversion per two codes); Q is scaled
// by a power of two per row to fit FP16, and P by 2^6.
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "paged.cuh"

namespace fp8fg {

constexpr int kFewThreads = 128, kFewCtas = 3;

// MG groups of 16 rows (1 or 2) and 4 / MG slices of 16 keys: a warp has one
// group and one slice, and the MG warps of a slice share its ring.  Three CTAs
// of four warps per SM (168 registers a thread fill it): while one starts or
// ends a pair, the others' copies go on.  (One CTA of twelve warps left the
// memory idle meanwhile: 84 against 60 us for 32 sequences x 5 tokens.)
template <int D, int FMT, int MG>
struct Few {
    static constexpr int kEsz = FMT == FP8_KV_BF16 ? 2 : 1;
    static constexpr int kSlices = 4 / MG;
    static constexpr int kTile = 16 * kSlices;                  // keys
    static constexpr int kRows = 16 * MG;
    static constexpr int kPairCost = 2 * MG;                    // a pair's own time (start, join) in tiles' times
    // A shorter run of places costs more in joining its part (16 MG rows) than its tiles take.
    static constexpr int kMinRun = 2 * MG;
    static constexpr int kRowB = D * kEsz;
    static constexpr int kCh = kRowB / 16;                      // 16-byte chunks of a row
    static constexpr int kStage = 2 * 16 * kRowB;               // K and V of 16 keys
    static constexpr int kFit = 64 * 1024 / (kSlices * kStage);
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr int kRing = kSlices * kStages * kStage;
    static constexpr int kORow = D + (FMT == FP8_KV_BF16 ? 8 : 4);   // floats of a merge row (no bank met twice)
    static constexpr int kMerge = kSlices * kRows * kORow * 4;
    static constexpr int kBytes = kRing > kMerge ? kRing : kMerge;
    static constexpr float kOff = FMT == FP8_KV_BF16 ? 0.0f : 6.0f;   // P is kept as 2^kOff p
};

// Tiles of a pair of a sequence of these lengths (0: not one of this kernel's), and
// sequence b's places in the line: kPairCost for a pair, then its tiles.
template <class C>
__device__ __forceinline__ int few_tiles(int rows, int len)
{
    return rows < 1 || rows > C::kRows ? 0 : max(1, (len + C::kTile - 1) / C::kTile);
}

template <class C>
__device__ __forceinline__ int64_t few_places(const AttnArgs &g, int b)
{
    if (b >= g.b.seqs) return 0;
    int first, rows, len;
    if (!seq_lengths(g, b, first, rows, len)) set_status(g.status, FP8_ERR_INVALID_ARG);
    const int nt = few_tiles<C>(rows, len);
    return nt > 0 ? (int64_t)(C::kPairCost + nt) * g.c.heads : 0;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int FMT>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (FMT == FP8_KV_BF16)
        mma_bf16(c, a, b0, b1);
    else
        mma_f16(c, a, b0, b1);
}

// Four products of P with FP8 values: a and b hold the codes of two keys each (bytes 2i and 2i + 1:
// column i of the first two, of the last two products).
template <int FMT>
__device__ __forceinline__ void pv4(float (&o0)[4], float (&o1)[4], float (&o2)[4], float (&o3)[4], const uint32_t (&p)[4],
                                    uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1)
{
    uint32_t al, ah, bl, bh;
    fp8x4_f16<FMT>(a0, al, ah);
    fp8x4_f16<FMT>(b0, bl, bh);
    mma16<FMT>(o0, p, al, bl);
    mma16<FMT>(o1, p, ah, bh);
    fp8x4_f16<FMT>(a1, al, ah);
    fp8x4_f16<FMT>(b1, bl, bh);
    mma16<FMT>(o2, p, al, bl);
    mma16<FMT>(o3, p, ah, bh);
}

__device__ __forceinline__ uint2 lds64(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// 16-byte copy; bytes 0: zero fill, nothing read.
__device__ __forceinline__ void cp_async16z(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Where chunk c of row r lies in a ring block: the chunk index is exchanged
// so that a warp's reads meet every bank once (64-byte FP8 value rows: twice).
template <int CH, bool V8>
__device__ __forceinline__ uint32_t few_at(int r, int c)
{
    if (CH == 4) return (uint32_t)(r * 64 + ((V8 ? c ^ ((r >> 1) & 3) : c) << 4));
    const int x = V8 ? r & 7 : ((r & 1) << 2) | ((r >> 1) & 3);
    return (uint32_t)(r * CH * 16 + ((c ^ x) << 4));
}

template <int ROWS>
struct FewPart {   // a broken pair's part in the workspace
    float m[ROWS], l[ROWS];
    float o[ROWS * 128];
};

template <int D, int FMT, int MG>
__global__ void __launch_bounds__(kFewThreads, kFewCtas) k_attn_few(AttnArgs g)
{
    using C = Few<D, FMT, MG>;
    using Part = FewPart<C::kRows>;
    constexpr int kThreads = kFewThreads, kSlices = C::kSlices;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_sums[kThreads / 32], s_start[2];
    __shared__ float s_m[kSlices][C::kRows], s_l[kSlices][C::kRows];
    __shared__ struct Broken {
        int first, rows, head, last;
        int64_t c0, c1;
    } s_broken[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gr = lane >> 2, t4 = lane & 3;
    const int slice = warp / MG, mrow = 16 * (warp % MG);   // this warp's keys of a tile and first row

    dependents_launch();
    dependency_wait();
    // this CTA's run [s, s_end) of the line of tiles, and the sequence it starts in
    int64_t total = 0, sum, ctas, s, s_end, n, incl;
    int b = 0;
    int64_t before = 0;   // places of the sequences before b
    for (int b0 = 0; b0 < g.b.seqs; b0 += kThreads) {
        n = few_places<C>(g, b0 + tid);
        incl = cta_scan(n, s_sums, sum);
        total += sum;
    }
    if (total == 0) return;
    ctas = min((int64_t)gridDim.x, (total + C::kMinRun - 1) / C::kMinRun);
    if (blockIdx.x >= ctas) return;
    s = div_short(blockIdx.x * total, ctas);
    s_end = div_short((blockIdx.x + 1) * total, ctas);
    for (int b0 = 0; b0 < g.b.seqs; b0 += kThreads) {
        if (g.b.seqs > kThreads) {   // (else the sums are still here)
            n = few_places<C>(g, b0 + tid);
            incl = cta_scan(n, s_sums, sum);
        }
        if (s < before + sum) {
            if (s >= before + incl - n && s < before + incl) {
                s_start[0] = b0 + tid;
                s_start[1] = before + incl - n;
            }
            __syncthreads();
            b = (int)s_start[0];
            before = s_start[1];
            break;
        }
        before += sum;
    }

    const float ks = g.c.k_scale ? *g.c.k_scale : 1.0f, vs = g.c.v_scale ? *g.c.v_scale : 1.0f;
    const uint32_t ring = smem_u32(smem) + slice * (C::kStages * C::kStage);
    float *merge = reinterpret_cast<float *>(smem);
    const int page_shift = 31 - __clz(g.c.page_size);

    // This lane's copies of a slice's 16 rows: kRpi rows an instruction of a warp, kCh lanes a row.  One
    // group: the warp copies keys and values; two groups: one warp each.
    constexpr int kRpi = 32 / C::kCh;
    const int cp_row = lane / C::kCh, cp_chunk = lane % C::kCh;
    const uint8_t *cp_src[2];
    int64_t page_b[2], head_b[2];
    uint32_t row_b[2], cp_dst[2], cp_flip[2];
#pragma unroll
    for (int k = 0; k < (MG == 1 ? 2 : 1); ++k) {
        const bool v = MG == 1 ? k == 1 : (warp & 1) != 0;
        row_b[k] = (uint32_t)(C::kEsz * (v ? g.c.v_row_stride : g.c.k_row_stride));
        page_b[k] = C::kEsz * (v ? g.c.v_page_stride : g.c.k_page_stride);
        head_b[k] = C::kEsz * (v ? g.c.v_head_stride : g.c.k_head_stride);
        cp_src[k] = static_cast<const uint8_t *>(v ? g.c.v : g.c.k) + (int64_t)cp_row * row_b[k] + cp_chunk * 16;
        const bool v8 = v && FMT != FP8_KV_BF16;
        cp_dst[k] = (v ? C::kStage / 2 : 0) + (v8 ? few_at<C::kCh, true>(cp_row, cp_chunk) : few_at<C::kCh, false>(cp_row, cp_chunk));
        // what few_at exchanges from one instruction to the next (kRpi rows on)
        cp_flip[k] = C::kCh == 8 ? (v8 ? 64 : 32) : 0;
    }
    auto copy = [&](uint32_t dst, const uint8_t *src, uint32_t step, uint32_t flip, int left) {
#pragma unroll
        for (int e = 0; e < 16 / kRpi; ++e) {
            const uint32_t d = C::kCh == 16 ? dst ^ ((e & 3) << 4) : (e & 1) ? dst ^ flip : dst;
            cp_async16z(d + e * 512, src + (uint32_t)(e * kRpi) * step, e * kRpi < left ? 16u : 0u);
        }
    };

    auto write_row = [&](int first, int h, int row, int d, float4 v, float mr, float lr) {
        const float inv = lr == 0.0f ? 0.0f : vs / lr;   // (a NaN stays one)
        const int64_t tok = first + row / g.group;
        const int head = h * g.group + row % g.group;
        const int64_t at = tok * g.out_ld + (int64_t)head * D + d;
        if (dbg_span(at, 4, (g.tokens - 1) * g.out_ld + (int64_t)g.q_heads * D, g.status))
            *reinterpret_cast<uint2 *>(g.out + at) = make_uint2(bf16x2_rn(v.x * inv, v.y * inv), bf16x2_rn(v.z * inv, v.w * inv));
        if (g.lse && d == 0 && dbg_lse(g, tok * g.q_heads + head))
            g.lse[tok * g.q_heads + head] = lr == 0.0f ? -INFINITY : (mr - C::kOff + log2f(lr)) * kLn2;
    };
    int nbroken = 0;   // pairs of this run that others have parts of
    int pages = 0, pbase = 0, pages_of = -1;
    while (s < s_end && b < g.b.seqs) {   // (b ends the walk only if the lengths changed meanwhile)
        int first, rows, len;
        seq_lengths(g, b, first, rows, len);
        const int nt = few_tiles<C>(rows, len);   // (of this read: rows and tiles fit the buffers whatever it gave)
        const int64_t seq_end = before + (nt > 0 ? (int64_t)(C::kPairCost + nt) * g.c.heads : 0);
        if (seq_end <= s) {   // the next sequence with tiles
            before = seq_end;
            ++b;
            pages_of = -1;
            continue;
        }
        const int h = (int)div_short(s - before, C::kPairCost + nt);
        const int64_t pair0 = before + (int64_t)h * (C::kPairCost + nt) + C::kPairCost;   // the place of its first tile
        const int tile0 = (int)max((int64_t)0, s - pair0), tile1 = (int)min((int64_t)nt, s_end - pair0);
        s = min(s_end, pair0 + nt);
        if (tile1 <= tile0) continue;   // a run that ends before the pair's tiles
        const int new_tokens = rows / g.group;
        const int32_t *table = g.b.page_table + b * g.b.page_table_ld;

        // this lane's chunks of Q rows gr and gr + 8: on their way before the copies
        uint4 qv[2][D / 32];
        int pos[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int row = mrow + gr + 8 * u, tok = row / g.group;
            pos[u] = row < rows ? len - new_tokens + tok : -1;
            const uint16_t *qp = g.q + (int64_t)(first + tok) * g.q_ld + (int64_t)(h * g.group + row % g.group) * D;
            // BF16: chunk t4 + 4c of 8 values; FP8: 16 values, two chunks side by side
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                const int d = FMT == FP8_KV_BF16 ? 8 * (t4 + 4 * c) : 16 * (t4 + 4 * (c / 2)) + 8 * (c % 2);
                qv[u][c] = row < rows ? *reinterpret_cast<const uint4 *>(qp + d) : make_uint4(0, 0, 0, 0);
            }
        }

        // copies of tile i's 16 keys of this slice into its ring, spread over its warps
        // (the pages of 32 tiles at a time, a tile a lane; those at hand serve a sequence's next head too)
        if (pages_of != b || tile0 < pbase || tile0 >= pbase + 32) pbase = tile0 - 32;
        pages_of = b;
        const uint8_t *ph[2];
#pragma unroll
        for (int k = 0; k < (MG == 1 ? 2 : 1); ++k) ph[k] = cp_src[k] + h * head_b[k];
        auto issue = [&](int i) {
            if (i < tile1) {
                if (i - pbase >= 32) {
                    pbase = i;
                    const int key = (i + lane) * C::kTile + slice * 16;
                    pages = (i + lane < nt && key < len) ? table[key >> page_shift] : 0;
                    if (pages < 0 || pages >= g.c.num_pages) {
                        set_status(g.status, FP8_ERR_INVALID_ARG);
                        pages = -1;
                    }
                }
                const int key0 = i * C::kTile + slice * 16;
                const int page = __shfl_sync(0xffffffffu, pages, i - pbase);
                if (key0 < len && page >= 0) {
                    const uint32_t rip = key0 & (g.c.page_size - 1), dst = ring + ((i - tile0) % C::kStages) * C::kStage;
                    const int left = len - key0 - cp_row;   // rows of this lane at or past it: zeros
                    if (MG == 1) {
                        copy(dst + cp_dst[0], ph[0] + page * page_b[0] + rip * row_b[0], row_b[0], cp_flip[0], left);
                        copy(dst + cp_dst[1], ph[1] + page * page_b[1] + rip * row_b[1], row_b[1], cp_flip[1], left);
                    } else {
                        copy(dst + cp_dst[0], ph[0] + page * page_b[0] + rip * row_b[0], row_b[0], cp_flip[0], left);
                    }
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < (MG == 1 ? C::kStages : C::kStages - 1); ++i) issue(tile0 + i);

        // Q as the A operand of D / 16 contraction steps; rows gr and gr + 8
        uint32_t qa[D / 16][4];
        float mul[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint4 (&v)[D / 32] = qv[u];
            mul[u] = g.scale * kLog2e * ks;
            float up = 1.0f;
            if (FMT != FP8_KV_BF16) {   // a power of two that brings the row's largest value into [2^14, 2^15)
                uint32_t m = 0;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) m = max(m, absmax8(v[c]));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const int e = min(max((int)(m >> 7), 15), 254) - 127;   // exponent of the largest value
                up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
                mul[u] *= __uint_as_float((uint32_t)(127 - 14 + e) << 23);
            }
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)   // word i: step 2c + i / 2, register u + 2 (i % 2)
                    qa[2 * c + i / 2][u + 2 * (i % 2)] =
                        FMT == FP8_KV_BF16 ? w[i] : f16x2_rn(bf16_lo(w[i]) * up, bf16_hi(w[i]) * up);
            }
        }

        const bool fine = len - new_tokens < kFineKeys, two = rows > mrow + 8;
        constexpr float lazy = FMT == FP8_KV_BF16 ? 0.0f : kLazy;
        float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;

        for (int i = tile0; i < tile1; ++i) {
            if (MG == 1) {
                cp_async_wait<C::kStages - 1>();
                __syncwarp();
            } else {   // tile i has landed for the slice's warps, and they are done with tile i - 1: its slot is free
                cp_async_wait<C::kStages - 2>();
                named_bar_sync(1 + slice, 32 * MG);
                issue(i + C::kStages - 1);
            }
            const int key0 = i * C::kTile + slice * 16;
            const uint32_t kb = ring + ((i - tile0) % C::kStages) * C::kStage, vb = kb + C::kStage / 2;
            if (key0 < len && mrow < rows) {   // (a page out of range left the slot as it was: unspecified outputs)
                float x[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.0f;
#pragma unroll
                    for (int c = 0; c < C::kCh / 4; ++c) {
                        const uint4 w = lds128(kb + few_at<C::kCh, false>(n * 8 + gr, t4 + 4 * c));
                        if (FMT == FP8_KV_BF16) {
                            mma16<FMT>(x[n], qa[2 * c], w.x, w.y);
                            mma16<FMT>(x[n], qa[2 * c + 1], w.z, w.w);
                        } else {
                            const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint32_t b0, b1;
                                fp8x4_f16<FMT>(v[e], b0, b1);
                                mma16<FMT>(x[n], qa[4 * c + e], b0, b1);
                            }
                        }
                    }
                }
                // log2 scores; keys a row does not see: -inf
                float v[2][4];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[u][e] = x[e / 2][2 * u + (e & 1)] * mul[u];
                    if (key0 + 15 > len - new_tokens) {   // some row may not see some of the keys
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (key0 + (e / 2) * 8 + 2 * t4 + (e & 1) > pos[u]) v[u][e] = -INFINITY;
                    }
                }
                // The four lanes of a row raise its maximum together, and only when one of them has to: the
                // shuffles are left out of nearly every block.
                float mx[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) mx[u] = fmaxf(fmaxf(v[u][0], v[u][1]), fmaxf(v[u][2], v[u][3]));
                if (__any_sync(0xffffffffu, mx[0] > m[0] + lazy || mx[1] > m[1] + lazy)) {
                    float up[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
                        mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
                        up[u] = 1.0f;
                        if (mx[u] > m[u] + lazy) {
                            up[u] = ex2_approx_ftz(m[u] - mx[u]);
                            m[u] = mx[u];
                        }
                        l[u] *= up[u];
                    }
#pragma unroll
                    for (int j = 0; j < D / 8; ++j) {
                        o[j][0] *= up[0];
                        o[j][1] *= up[0];
                        o[j][2] *= up[1];
                        o[j][3] *= up[1];
                    }
                }
                uint32_t pa[4], pl[4];   // P, and its second term
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (u == 1 && !two) {   // rows 8 to 15 of the group: none
                        pa[1] = pa[3] = pl[1] = pl[3] = 0;
                        continue;
                    }
                    const float base = m[u] == -INFINITY ? 0.0f : m[u] - C::kOff;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[u][e] = ex2_approx_ftz(v[u][e] - base);
                    l[u] += (v[u][0] + v[u][1]) + (v[u][2] + v[u][3]);
                    pa[u] = FMT == FP8_KV_BF16 ? bf16x2_rn(v[u][0], v[u][1]) : f16x2_rn(v[u][0], v[u][1]);
                    pa[u + 2] = FMT == FP8_KV_BF16 ? bf16x2_rn(v[u][2], v[u][3]) : f16x2_rn(v[u][2], v[u][3]);
                    if (FMT == FP8_KV_BF16) {
                        pl[u] = bf16x2_rn(v[u][0] - bf16_lo(pa[u]), v[u][1] - bf16_hi(pa[u]));
                        pl[u + 2] = bf16x2_rn(v[u][2] - bf16_lo(pa[u + 2]), v[u][3] - bf16_hi(pa[u + 2]));
                    }
                }
                if (FMT == FP8_KV_BF16) {
#pragma unroll
                    for (int j = 0; j < D / 8; j += 2) {
                        uint32_t w[4];
                        ldsm_x4_t(vb + few_at<C::kCh, false>(lane & 15, j + (lane >> 4)), w);
                        mma16<FMT>(o[j], pa, w[0], w[1]);
                        mma16<FMT>(o[j + 1], pa, w[2], w[3]);
                        if (fine) {
                            mma16<FMT>(o[j], pl, w[0], w[1]);
                            mma16<FMT>(o[j + 1], pl, w[2], w[3]);
                        }
                    }
                } else if (D == 128) {   // column n of product j is head element 16 n + j
                    uint4 r[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        r[e] = lds128(vb + few_at<C::kCh, true>(2 * t4 + (e & 1) + 8 * (e >> 1), gr));
                    const uint32_t w[4][4] = {{r[0].x, r[0].y, r[0].z, r[0].w}, {r[1].x, r[1].y, r[1].z, r[1].w},
                                              {r[2].x, r[2].y, r[2].z, r[2].w}, {r[3].x, r[3].y, r[3].z, r[3].w}};
#pragma unroll
                    for (int i4 = 0; i4 < 4; ++i4) {
                        const uint32_t a0 = __byte_perm(w[0][i4], w[1][i4], 0x5140), a1 = __byte_perm(w[0][i4], w[1][i4], 0x7362);
                        const uint32_t b0 = __byte_perm(w[2][i4], w[3][i4], 0x5140), b1 = __byte_perm(w[2][i4], w[3][i4], 0x7362);
                        pv4<FMT>(o[4 * i4], o[4 * i4 + 1], o[4 * i4 + 2], o[4 * i4 + 3], pa, a0, a1, b0, b1);
                    }
                } else {                 // column n of product j is head element 8 n + j
                    uint2 r[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        r[e] = lds64(vb + few_at<C::kCh, true>(2 * t4 + (e & 1) + 8 * (e >> 1), gr >> 1) + 8 * (gr & 1));
                    const uint32_t w[4][2] = {{r[0].x, r[0].y}, {r[1].x, r[1].y}, {r[2].x, r[2].y}, {r[3].x, r[3].y}};
#pragma unroll
                    for (int i2 = 0; i2 < 2; ++i2) {
                        const uint32_t a0 = __byte_perm(w[0][i2], w[1][i2], 0x5140), a1 = __byte_perm(w[0][i2], w[1][i2], 0x7362);
                        const uint32_t b0 = __byte_perm(w[2][i2], w[3][i2], 0x5140), b1 = __byte_perm(w[2][i2], w[3][i2], 0x7362);
                        pv4<FMT>(o[4 * i2], o[4 * i2 + 1], o[4 * i2 + 2], o[4 * i2 + 3], pa, a0, a1, b0, b1);
                    }
                }
            }
            if (MG == 1) {
                __syncwarp();   // all lanes have read the slot before it is filled again
                issue(i + C::kStages);
            }
        }
        cp_async_wait<0>();
        __syncthreads();    // the ring becomes the merge buffer

        // the slices' parts of the run joined
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
            l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
            if (t4 == 0) {
                s_m[slice][mrow + gr + 8 * u] = m[u];
                s_l[slice][mrow + gr + 8 * u] = l[u];
            }
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                if (mrow + gr + 8 * u >= rows) continue;
                float *p = merge + (slice * C::kRows + mrow + gr + 8 * u) * C::kORow;
                if (FMT == FP8_KV_BF16)
                    *reinterpret_cast<float2 *>(p + 8 * j + 2 * t4) = make_float2(o[j][2 * u], o[j][2 * u + 1]);
                else if (j % 4 == 0)   // column n's j-th four elements are the row's piece 8 (j / 4) + n
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        *reinterpret_cast<float4 *>(p + 4 * (2 * j + 2 * t4 + k)) =
                            make_float4(o[j][2 * u + k], o[j + 1][2 * u + k], o[j + 2][2 * u + k], o[j + 3][2 * u + k]);
            }
        }
        __syncthreads();
        const bool whole = tile0 == 0 && tile1 == nt;
        Part *part = static_cast<Part *>(g.few_parts) + 2 * blockIdx.x + (tile0 == 0 ? 1 : 0);
        for (int e = tid; e < rows * (D / 4); e += kThreads) {
            const int row = e / (D / 4), piece = e % (D / 4);
            const int d = FMT == FP8_KV_BF16 ? 4 * piece : (D / 8) * (piece % 8) + 4 * (piece / 8);
            float mr = s_m[0][row];
#pragma unroll
            for (int w = 1; w < kSlices; ++w) mr = fmaxf(mr, s_m[w][row]);
            float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float lr = 0.0f;
#pragma unroll
            for (int w = 0; w < kSlices; ++w) {
                const float f = mr == -INFINITY ? 0.0f : ex2_approx_ftz(s_m[w][row] - mr);
                const float4 v = *reinterpret_cast<const float4 *>(merge + (w * C::kRows + row) * C::kORow + 4 * piece);
                a.x += f * v.x;
                a.y += f * v.y;
                a.z += f * v.z;
                a.w += f * v.w;
                lr += f * s_l[w][row];
            }
            if (whole) {
                write_row(first, h, row, d, a, mr, lr);
            } else {
                *reinterpret_cast<float4 *>(part->o + row * D + d) = a;
                if (d == 0) {
                    part->m[row] = mr;
                    part->l[row] = lr;
                }
            }
        }
        if (!whole) {
            // CTA c's run starts at floor(c total / ctas): c holds place p iff c = ceil((p + 1) ctas / total) - 1
            if (tid == 0)
                s_broken[nbroken] = {first, rows, h, 0, div_short((pair0 + 1) * ctas + total - 1, total) - 1,
                                     min(div_short((pair0 + nt) * ctas + total - 1, total), ctas) - 1};
            ++nbroken;
        }
        __syncthreads();    // the merge buffer becomes the ring again
    }

    // The broken pairs' parts are announced when the run is done: a fence in its middle waited several
    // microseconds for the stores under the other CTAs' copies.
    if (nbroken == 0) return;
    if (tid == 0) {
        __threadfence();    // the CTA's stores (the barrier above), by one thread for them all
        for (int k = 0; k < nbroken; ++k)
            s_broken[k].last = atomicAdd(&g.few_count[s_broken[k].c0], 1) == (int)(s_broken[k].c1 - s_broken[k].c0);
        __threadfence();
    }
    __syncthreads();
    for (int k = 0; k < nbroken; ++k) {
        const Broken q = s_broken[k];
        if (!q.last) continue;
        const Part *parts = static_cast<const Part *>(g.few_parts);
        const int parts_n = (int)(q.c1 - q.c0) + 1;
        auto part_of = [&](int i) -> const Part & { return parts[2 * (q.c0 + i) + (i == 0)]; };
        // Few parts: each thread takes the maxima itself.  More than kDirectParts: they are found once a
        // row, the parts side by side (5 sequences x 8 rows, 45 parts: 32 against 23 us; 32 x 20 rows, 2 to
        // 3 parts: 57 against 62 us).
        auto direct = [&](auto elements) {
            constexpr int kE = decltype(elements)::value;
            for (int e0 = tid; e0 < q.rows * (D / 4); e0 += kThreads * kE) {
                const int d = (e0 % (D / 4)) * 4;   // (kThreads is a multiple of D / 4)
                int row[kE];
                float mr[kE], lr[kE];
                float4 acc[kE];
#pragma unroll
                for (int k = 0; k < kE; ++k) {
                    row[k] = min(e0 / (D / 4) + k * (kThreads / (D / 4)), q.rows - 1);
                    mr[k] = -INFINITY;
                    lr[k] = 0.0f;
                    acc[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
#pragma unroll 4
                for (int i = 0; i < parts_n; ++i)
#pragma unroll
                    for (int k = 0; k < kE; ++k) mr[k] = fmaxf(mr[k], __ldcg(&part_of(i).m[row[k]]));
#pragma unroll 4
                for (int i = 0; i < parts_n; ++i) {
                    const Part &p = part_of(i);
#pragma unroll
                    for (int k = 0; k < kE; ++k) {
                        const float f = mr[k] == -INFINITY ? 0.0f : ex2_approx_ftz(__ldcg(&p.m[row[k]]) - mr[k]);
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.o + row[k] * D + d));
                        acc[k].x += f * v.x;
                        acc[k].y += f * v.y;
                        acc[k].z += f * v.z;
                        acc[k].w += f * v.w;
                        lr[k] += f * __ldcg(&p.l[row[k]]);
                    }
                }
#pragma unroll
                for (int k = 0; k < kE; ++k)
                    if (e0 + k * kThreads < q.rows * (D / 4)) write_row(q.first, q.head, row[k], d, acc[k], mr[k], lr[k]);
            }
        };
        if (tid == 0) g.few_count[q.c0] = 0;
        if (parts_n <= kDirectParts) {
            if (q.rows * (D / 4) <= kThreads)
                direct(std::integral_constant<int, 1>());
            else
                direct(std::integral_constant<int, 4>());
            continue;
        }
        constexpr int kR = 4;
        for (int row0 = warp * kR; row0 < q.rows; row0 += kR * (kThreads / 32)) {
            float mr[kR], lr[kR] = {};
#pragma unroll
            for (int k = 0; k < kR; ++k) mr[k] = -INFINITY;
            for (int i = lane; i < parts_n; i += 32)   // (rows past the last exist in the part: unused)
#pragma unroll
                for (int k = 0; k < kR; ++k) mr[k] = fmaxf(mr[k], __ldcg(&part_of(i).m[row0 + k]));
#pragma unroll
            for (int k = 0; k < kR; ++k)
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mr[k] = fmaxf(mr[k], __shfl_xor_sync(0xffffffffu, mr[k], o));
            for (int i = lane; i < parts_n; i += 32)
#pragma unroll
                for (int k = 0; k < kR; ++k)
                    lr[k] += (mr[k] == -INFINITY ? 0.0f : ex2_approx_ftz(__ldcg(&part_of(i).m[row0 + k]) - mr[k])) *
                             __ldcg(&part_of(i).l[row0 + k]);
#pragma unroll
            for (int k = 0; k < kR; ++k) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) lr[k] += __shfl_xor_sync(0xffffffffu, lr[k], o);
                if (lane == 0) {
                    s_m[0][row0 + k] = mr[k];
                    s_l[0][row0 + k] = lr[k];
                }
            }
        }
        __syncthreads();
        // the outputs: two elements a thread and eight parts at a time in flight
        constexpr int kE = 2;
        for (int e0 = tid; e0 < q.rows * (D / 4); e0 += kThreads * kE) {
            const int d = (e0 % (D / 4)) * 4;   // (kThreads is a multiple of D / 4)
            int row[kE];
            float4 acc[kE];
#pragma unroll
            for (int k = 0; k < kE; ++k) {
                row[k] = min(e0 / (D / 4) + k * (kThreads / (D / 4)), q.rows - 1);
                acc[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll 8
            for (int i = 0; i < parts_n; ++i) {
                const Part &p = part_of(i);
#pragma unroll
                for (int k = 0; k < kE; ++k) {
                    const float mr = s_m[0][row[k]];
                    const float f = mr == -INFINITY ? 0.0f : ex2_approx_ftz(__ldcg(&p.m[row[k]]) - mr);
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.o + row[k] * D + d));
                    acc[k].x += f * v.x;
                    acc[k].y += f * v.y;
                    acc[k].z += f * v.z;
                    acc[k].w += f * v.w;
                }
            }
#pragma unroll
            for (int k = 0; k < kE; ++k)
                if (e0 + k * kThreads < q.rows * (D / 4)) write_row(q.first, q.head, row[k], d, acc[k], s_m[0][row[k]], s_l[0][row[k]]);
        }
        __syncthreads();   // (the other broken pair's maxima replace these)
    }
}

int few_grid() { return kFewCtas * sm_count(); }

size_t few_parts_bytes() { return (size_t)few_grid() * 2 * sizeof(FewPart<kFewMost>); }

template <int D, int FMT, int MG>
static int launch_few(const AttnArgs &g, cudaStream_t st)
{
    using C = Few<D, FMT, MG>;
    static_assert(kFewCtas * C::kBytes <= 224 * 1024 && C::kStages >= 2, "the rings do not fit the SM");
    static bool attr_done[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (!attr_done[dev & 63]) {
        if (cudaFuncSetAttribute(k_attn_few<D, FMT, MG>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes) !=
            cudaSuccess)
            return FP8_ERR_CUDA;
        attr_done[dev & 63] = true;
    }
    return launch_dependent(k_attn_few<D, FMT, MG>, dim3(few_grid()), kFewThreads, C::kBytes, st, g);
}

template <int D, int FMT>
static int launch_few_rows(const AttnArgs &g, int rows, cudaStream_t st)
{
    return rows <= 16 ? launch_few<D, FMT, 1>(g, st) : launch_few<D, FMT, 2>(g, st);
}

int run_few(const AttnArgs &g, int rows, cudaStream_t st)
{
    if (g.c.head_dim == 128) {
        if (g.c.format == FP8_KV_BF16) return launch_few_rows<128, FP8_KV_BF16>(g, rows, st);
        if (g.c.format == FP8_KV_E5M2) return launch_few_rows<128, FP8_KV_E5M2>(g, rows, st);
        return launch_few_rows<128, FP8_KV_E4M3>(g, rows, st);
    }
    if (g.c.format == FP8_KV_BF16) return launch_few_rows<64, FP8_KV_BF16>(g, rows, st);
    if (g.c.format == FP8_KV_E5M2) return launch_few_rows<64, FP8_KV_E5M2>(g, rows, st);
    return launch_few_rows<64, FP8_KV_E4M3>(g, rows, st);
}

}  // namespace fp8fg
