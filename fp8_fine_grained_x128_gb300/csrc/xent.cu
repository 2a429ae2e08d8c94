// xent.cu -- softmax cross entropy of a linear head, and its gradient, without
// keeping the logits (sm_103a).
//
// With z = scale * x w^T over a vocabulary of V rows of w, per counted token:
//   lse = log sum_v exp z_v,  loss = lse - z_t,
// and for the gradients gl, gz of loss and lse
//   g_v = scale * ((gl + gz) p_v - gl [v = t]),  p_v = exp(z_v - lse),
//   dx = g w,  dw = g^T x.
// p_t - 1 is taken as expm1(-loss), not as a difference, so that a token the
// model is sure of keeps its small gradient; and the loss itself is formed as
// log(1 + sum_{v != t} exp(z_v - z_t)) from a sum that leaves the target out,
// so that it does not vanish in the rounding of lse.
//
// Everything is a product on the tensor cores (BF16 operands, FP32
// accumulators): the forward's logits, and per piece of the vocabulary the
// backward's logits (again), g w and g^T x.  One kernel does all (k_xent<MODE>);
// they differ in which operands run along K.  Up to 4 tokens are multiplied in
// registers instead, in FP32, while W streams past (k_xent_few, k_xent_few_grad).
//
// Forward: the epilogue keeps, per row, a running maximum and sum over a unit
// of up to 8 tiles and writes 8 bytes a row and half unit, 1/32 of a BF16 logit row
// and less (1/16 with tiles of 128 columns); k_xent_join adds them in order.
// Backward: for a piece of the vocabulary, g is rounded to BF16 (the tensor
// cores' operand type) and kept in the workspace, [tokens][piece]; dx is summed
// over the pieces in FP32.  A token's g is mostly its target's entry, whose
// rounding would reach all of the token's dx and all that it adds to dw.  So each
// row is taken relative to that entry, which is then +-1: dx gets it back in FP32,
// and dw from a copy of x times it, rounded to BF16.
//
// Tokens that do not count are left out from the start: k_xent_pack copies the
// counted rows of x together, so neither the work nor the results see the
// others, whatever they hold.  (Up to 128 tokens, and small forwards, keep their
// rows: the others' are independent of them, or zeros.)
//
// k_xent is a persistent kernel of CTA pairs (cta_group::2): a pair computes
// 256 x 256 tiles, each CTA holding 128 rows of A and 128 columns of B of every
// 64-deep stage, so that an SM fetches 32 KB where a CTA alone would fetch 48 KB
// for its half of the tile.  Warp 0 copies (TMA, 4 to 7 stages), one thread of the
// even CTA's warp 1 issues the MMAs, warps 2..9 drain one of two accumulators
// while the next tile fills the other.  Few tokens take tiles of single CTAs.
#include <limits.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "tmap.h"

namespace fp8fg {

namespace {

enum { XENT_LOSS = 0, XENT_GRAD = 1, XENT_SUMS = 2 };     // SUMS: dx and dw

constexpr int kTile = 256;              // rows and columns of a pair's tile
constexpr int kBK = 64;                 // K of a stage
constexpr int kEpiWarp0 = 2, kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kBox = 4096;              // staging for one copy: 32 rows of 128 bytes

// PAIR: 256 x BN tiles by two CTAs, of 128 rows and BN / 2 columns each; else
// 128 x BN tiles by one.  A box of staging for every epilogue warp (LOSS has no
// matrix to write); the rest of the shared memory is stages.
template <int MODE, bool PAIR, int BN>
struct Form {
    static constexpr int kM = PAIR ? 256 : 128, kOwnN = PAIR ? BN / 2 : BN;
    static constexpr int kA = 128 * kBK * 2, kB = kOwnN * kBK * 2, kStage = kA + kB;
    static constexpr int kStaging = MODE == XENT_LOSS ? 0 : kEpiWarps * kBox;
    static constexpr int kStages = (226 * 1024 - 1024 - kStaging) / kStage;
    static constexpr int kBars = 2 * kStages + 2 * 2 + 1;
    static constexpr int kSmem = 1024 + kStages * kStage + kStaging + kBars * 8 + 16;
    static_assert(kSmem + 1024 <= 227 * 1024, "dynamic shared memory above the per-CTA limit");
};

// The tensor cores' sums lean towards zero, by up to a last place for every 16 of K
// (1.1e-6 of the loss at dim 4096; in one sum over 65536 tokens, 1.8e-4 of dw): LOSS and
// SUMS take 2048 of K at a time, and add those to nearest.  (GRAD's K is dim, 2e-5 of a
// logit at 8192: less than g's rounding to BF16 shows.)  SUMS without a longer K is
// compiled apart (100 x 8000 x 256 backward 18.7 us, 19.1 with the code for longer ones;
// 64 x 128000 x 4096, where dx's parts are long, 605 us in one sum and 608 in pieces).
constexpr int kChunk = 2048 / kBK;

// Sums of a tile whose K is `blocks` blocks; one, of nothing, where there are none.
__device__ __forceinline__ int chunks_of(int blocks) { return max(1, (blocks + kChunk - 1) / kChunk); }

constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

struct XentArgs {
    const int *count;           // counted tokens (nullptr: all `tokens` rows)
    int tokens, vocab, dim;
    int v0, vn;                 // this piece's vocabulary: columns [v0, v0 + vn)
    int per_unit;               // LOSS: tiles of a unit
    int splits;                 // dx: parts of K
    int band;                   // M tiles of a raster band
    int box;                    // single CTAs: rows of x that are fetched for a tile (the others' results are not used)
    float scale;
    const int32_t *target;      // LOSS: of every row; GRAD: of every token
    // LOSS
    float2 *part;               // [unit][half][rows]: maximum (times scale log2 e), sum of 2^(. - maximum)
    int64_t rows;               // rows of the packed buffers
    // GRAD
    const float4 *info;         // [rows]: see row_info; nullptr: the rows are the tokens and not packed, and made of
    const float *loss, *lse, *dloss, *dlse;
    const uint16_t *x;          // then also: x, and where it goes, times norm, in this launch (xn nullptr: it has already)
    int64_t ldx;
    uint16_t *xn;
    float *norm;
    // SUMS
    int dx_add;                 // dx's parts (FP32, [splits][rows][dim]) are added to
    int dw_f32, dw_add;
    int *status;
};

// The units of a pair (or single CTA), in the same order for every role: tiles
// in columns [nt0, nt1) of row mt, K blocks [k0, k1).  Where a unit lies takes
// several divisions, half a microsecond for one thread, so a warp works them out
// for 32 units at a time.
struct Unit { int mt, nt0, nt1, k0, k1, split, dw; };

struct Grid {       // of one product
    int num_mt, num_nt, num_ng, per, units, nkb, per_split, band;
    __device__ __forceinline__ Grid(int M, int N, int K, int kM, int kN, int per_, int splits, int band_) : per(per_), band(band_)
    {
        num_mt = (M + kM - 1) / kM;
        num_nt = (N + kN - 1) / kN;
        num_ng = (num_nt + per - 1) / per;
        nkb = (K + kBK - 1) / kBK;
        per_split = (nkb + splits - 1) / splits;
        units = num_mt * num_ng * splits;
    }
};

// What a DW tile costs at least, in K blocks of 64: its writing.
constexpr int kTileCost = 6;

template <int MODE, bool PAIR, int BN>
struct Walk {
    static constexpr int kM = PAIR ? 256 : 128;
    const int mine, step;
    Grid p, w;          // LOSS, GRAD: p; SUMS: p is dx, w is dw
    // SUMS: dx's units go round the pairs first.  The pairs past the last, unfinished
    // round (from `rem` on) then take `extra` rounds of dw's, as long as one of dx's
    // units lasts, and the rest of dw's go round all pairs.
    int rem, extra;
    __device__ __forceinline__ Walk(const XentArgs &a, int rows, int mine_, int step_)
        : mine(mine_), step(step_), p(rows, MODE == XENT_SUMS ? a.dim : a.vn, MODE == XENT_SUMS ? a.vn : a.dim, kM, BN,
                                      MODE == XENT_LOSS ? a.per_unit : 1, MODE == XENT_SUMS ? a.splits : 1, a.band),
          w(MODE == XENT_SUMS ? a.vn : 0, a.dim, rows, kM, BN, 1, 1, a.band)
    {
        rem = p.units % step;
        extra = rem == 0 ? 0 : min(p.per_split / max(w.nkb, kTileCost), w.units / (step - rem));
    }
    // The pair's unit i; whether there is one.
    __device__ __forceinline__ bool unit(int i, Unit &t) const
    {
        const int j = i - (p.units / step + (mine < rem));      // beyond this pair's units of p
        const bool dw = MODE == XENT_SUMS && j >= 0;
        int64_t u = mine + (int64_t)i * step;
        if (dw) {
            const int ahead = mine >= rem ? extra : 0;
            u = j < ahead ? (int64_t)j * (step - rem) + mine - rem : (int64_t)extra * (step - rem) + (int64_t)(j - ahead) * step + mine;
        }
        const Grid &g = dw ? w : p;
        if (u >= g.units) return false;
        const int flat = g.num_mt * g.num_ng;
        t.split = (int)u / flat;
        tile_coords_raster((int)u - t.split * flat, g.num_mt, g.num_ng, g.band, t.mt, t.nt0);
        t.nt0 *= p.per;
        t.dw = dw;
        t.k0 = min(g.nkb, t.split * g.per_split);
        t.k1 = min(g.nkb, t.k0 + g.per_split);
        return true;
    }
    // body(unit, row of tiles of the next one where that is known), by the whole warp
    template <typename Body>
    __device__ __forceinline__ void each(bool &ok, Body &&body) const
    {
        const int lane = threadIdx.x & 31;
        for (int base = 0; ok; base += 32) {
            Unit mine_{};
            const int todo = __popc(__ballot_sync(0xffffffffu, unit(base + lane, mine_)));      // the valid ones are the first
            for (int k = 0; k < todo && ok; ++k) {
                auto from = [&](int v, int i) { return __shfl_sync(0xffffffffu, v, i); };
                Unit t{};
                t.mt = from(mine_.mt, k);
                t.nt0 = from(mine_.nt0, k);
                if (MODE == XENT_SUMS) {
                    t.dw = from(mine_.dw, k);
                    t.k0 = from(mine_.k0, k);
                    t.k1 = from(mine_.k1, k);
                    t.split = from(mine_.split, k);
                }
                t.nt1 = min(t.dw ? w.num_nt : p.num_nt, t.nt0 + p.per);
                body(t, MODE <= XENT_GRAD && k + 1 < todo ? from(mine_.mt, k + 1) : -1);
            }
            if (todo < 32) break;
        }
    }
    // body(unit) by lane 0 alone, until it returns false: the warp does not meet
    // between the units (700 cycles a unit, which a pair's tensor cores would wait)
    template <typename Body>
    __device__ __forceinline__ bool each_alone(int4 *list, Body &&body) const
    {
        const int lane = threadIdx.x & 31;
        for (int base = 0;; base += 32) {
            Unit t{};
            const bool valid = unit(base + lane, t);
            list[lane] = make_int4(t.mt, t.nt0, t.k0, t.k1 << 1 | t.dw);
            const int todo = __popc(__ballot_sync(0xffffffffu, valid));
            __syncwarp();
            bool ok = true;
            if (lane == 0) {
                for (int k = 0; k < todo && ok; ++k) {
                    const int4 i = list[k];
                    t.mt = i.x;
                    t.nt0 = i.y;
                    t.k0 = i.z;
                    t.k1 = i.w >> 1;
                    t.dw = i.w & 1;
                    t.nt1 = min(t.dw ? w.num_nt : p.num_nt, t.nt0 + p.per);
                    ok = body(t);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok || todo < 32) return ok;
        }
    }
};

// Tensor maps: A, B and the result, of dx and then of dw for SUMS.
template <int MODE>
struct Maps { CUtensorMap m[MODE == XENT_SUMS ? 6 : 3]; };

// g at the target, of a token with this loss.
__device__ __forceinline__ float target_entry(float scale, float loss, float gl, float gz)
{
    return scale * (gl * expm1f(-loss) + gz * expf(-loss));
}

// What a row of g is made of: lse log2 e, the factor of p, the entry at the target, the
// target as an int; relative to `by`, the size of that entry.
__device__ __forceinline__ float4 row_info(float scale, float loss, float lse, float gl, float gz, int target, float &by)
{
    const float entry = target_entry(scale, loss, gl, gz), factor = scale * (gl + gz), n = fabsf(entry), c = fabsf(factor);
    // the row stays as it is where that entry, or the others relative to it, are beyond all measure
    const bool relative = n >= 0x1p-100f && n <= 0x1p100f && c <= n * 0x1p120f && c * -expm1f(-loss) <= n * 0x1p60f;
    by = relative ? n : 1.0f;
    return make_float4(lse * kLog2e, factor / by, entry / by, __int_as_float(target));
}

// 8 BF16 values, times `by`.
__device__ __forceinline__ uint4 times8(uint4 v, float by)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = bf16x2_rn(bf16_lo(w[k]) * by, bf16_hi(w[k]) * by);
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// 8 FP32 values to 16 bytes of BF16.
__device__ __forceinline__ uint4 bf16x8(const uint32_t *r)
{
    auto f = [&](int i) { return __uint_as_float(r[i]); };
    return make_uint4(bf16x2_rn(f(0), f(1)), bf16x2_rn(f(2), f(3)), bf16x2_rn(f(4), f(5)), bf16x2_rn(f(6), f(7)));
}

}  // namespace

// LONG: SUMS of which some K is longer than kChunk.
template <int MODE, bool PAIR, int BN, bool LONG>
__global__ void __launch_bounds__(kThreads, 1)
    k_xent(const __grid_constant__ Maps<MODE> maps, const XentArgs a)
{
    using F = Form<MODE, PAIR, BN>;
    constexpr bool kSums = MODE == XENT_SUMS;
    constexpr int kStages = F::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int4 units[2][32];       // of the copying and of the issuing warp
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kStages * F::kStage + F::kStaging);
    uint64_t *empty = full + kStages;
    uint64_t *tfull = empty + kStages;
    uint64_t *tempty = tfull + 2;
    uint64_t *mma_done = tempty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_rank() : 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], (PAIR ? 2 : 1) * kEpiWarps);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_barrier_init();
        for (const CUtensorMap &m : maps.m) prefetch_tensormap(&m);
    }
    if (warp == 1) {
        if (PAIR) {
            tmem_alloc_pair(tmem_slot, 2 * BN);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_slot, 2 * BN);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();   // the pair's barriers are there before either CTA signals the other's
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    dependency_wait();
    const int rows = a.count ? *a.count : a.tokens;
    // accumulators of a tile, one for every kChunk blocks of K: of LOSS here, of SUMS by the unit
    const int loss_chunks = MODE == XENT_LOSS ? chunks_of((a.dim + kBK - 1) / kBK) : 1;
    const Walk<MODE, PAIR, BN> walk(a, rows, PAIR ? blockIdx.x >> 1 : blockIdx.x, PAIR ? gridDim.x >> 1 : gridDim.x);

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        uint32_t it = 0;
        const bool ok = walk.each_alone(units[0], [&](const Unit &t) {
            const int m = t.mt * F::kM + rank * 128;
            for (int nt = t.nt0; nt < t.nt1; ++nt) {
                const int n = nt * BN + rank * F::kOwnN;
                for (int kb = t.k0; kb < t.k1; ++kb, ++it) {
                    const int s = it % kStages;
                    if (!thread_wait(smem_u32(&empty[s]), ((it / kStages) & 1) ^ 1, abort_flag, a.status)) return false;
                    // what of a copy lies outside its matrix is filled with zeros and counts its bytes all the same
                    const int bytes = PAIR || kSums ? (PAIR ? 2 : 1) * F::kStage : a.box * (kBK * 2) + F::kB;
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
                    const uint32_t bar = PAIR ? cluster_addr(&full[s], 0) : 0;
                    uint8_t *sa = smem + s * F::kStage, *sb = sa + F::kA;
                    auto load = [&](uint8_t *to, const CUtensorMap *map, int x, int y) {
                        if (PAIR) tma_load_2d_pair(to, map, bar, x, y);
                        else tma_load_2d(to, map, &full[s], x, y);
                    };
                    if (kSums) {        // dx: g along K, W across it; dw: both across
                        const CUtensorMap *A = &maps.m[t.dw ? 3 : 0], *B = A + 1;
                        if (t.dw) {
                            load(sa, A, m, kb * kBK);
                            load(sa + 8192, A, m + 64, kb * kBK);
                        } else {
                            load(sa, A, kb * kBK, m);
                        }
                        const int k = (t.dw ? 0 : a.v0) + kb * kBK;
#pragma unroll
                        for (int j = 0; j < F::kOwnN / 64; ++j) load(sb + j * 8192, B, n + 64 * j, k);
                    } else {            // x and W along K
                        load(sa, &maps.m[0], kb * kBK, m);
#pragma unroll
                        for (int j = 0; j < F::kOwnN; j += 128) load(sb + j * 128, &maps.m[1], kb * kBK, a.v0 + n + j);
                    }
                }
            }
            return true;
        });
        // the next kernel may be set up (k_xent_join reads this call's inputs before it waits: so not before this one has)
        dependents_launch();
        // the copies in flight land (the even CTA's barrier counts both CTAs'),
        // and the last stages' releases arrive, before the pair may leave
        if (lane == 0) {
            for (uint32_t j = it > (uint32_t)kStages ? it - kStages : 0; j < it; ++j) {
                if (rank == 0) mbar_wait_bounded(&full[j % kStages], (j / kStages) & 1, nullptr);
                if (ok) mbar_wait_bounded(&empty[j % kStages], (j / kStages) & 1, abort_flag);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer
        auto commit = [&](uint64_t *bar) {
            if (PAIR) tc_commit_pair(bar);
            else tc_commit(bar);
        };
        if (rank == 0) {
            uint32_t it = 0, tc = 0;
            walk.each_alone(units[1], [&](const Unit &t) {
                const uint32_t idesc = kSums && t.dw ? idesc_bf16(F::kM, BN, true, true) : idesc_bf16(F::kM, BN, false, kSums);
                const int chunks = kSums ? (LONG ? chunks_of(t.k1 - t.k0) : 1) : loss_chunks;
                const int parts = (t.nt1 - t.nt0) * chunks;     // of the unit, an accumulator each
                for (int i = 0; i < parts; ++i, ++tc) {
                    const int c0 = chunks == 1 ? t.k0 : t.k0 + i % chunks * kChunk, c1 = chunks == 1 ? t.k1 : min(t.k1, c0 + kChunk);
                    const uint32_t buf = tc & 1;
                    if (!thread_wait(smem_u32(&tempty[buf]), ((tc >> 1) & 1) ^ 1, abort_flag, a.status)) return false;
                    tc_fence_after();
                    const uint32_t d = tmem_base + buf * BN;
                    for (int kb = c0; kb < c1; ++kb, ++it) {
                        const int s = it % kStages;
                        if (!thread_wait(smem_u32(&full[s]), (it / kStages) & 1, abort_flag, a.status)) return false;
                        tc_fence_after();
                        const uint32_t sa = smem_u32(smem + s * F::kStage), sb = sa + F::kA;
                        // 16 of K: 32 bytes along a row, or two 1024-byte swizzle atoms of rows
                        const uint64_t ad = kSums && t.dw ? sdesc_mnmajor_sw128(sa, 8192, 1024) : sdesc_kmajor_sw128(sa);
                        const uint64_t bd = kSums ? sdesc_mnmajor_sw128(sb, 8192, 1024) : sdesc_kmajor_sw128(sb);
                        const uint64_t a_step = (kSums && t.dw ? 2048 : 32) >> 4, b_step = (kSums ? 2048 : 32) >> 4;
#pragma unroll
                        for (int k = 0; k < kBK / 16; ++k) {
                            const uint32_t more = kb > c0 || k > 0;
                            if (PAIR) tc_mma_f16_pair(d, ad + k * a_step, bd + k * b_step, idesc, more);
                            else tc_mma_f16(d, ad + k * a_step, bd + k * b_step, idesc, more);
                        }
                        commit(&empty[s]);
                    }
                    commit(&tfull[buf]);
                }
                return true;
            });
            if (lane == 0) commit(mma_done);
        }
        if (lane == 0) mbar_wait_bounded(mma_done, 0, nullptr);
        __syncwarp();
    } else if (warp >= kEpiWarp0) {
        // ------------------------------------------------------ epilogue
        const int lq = warp & 3;                 // TMEM lane quarter of this warp
        const int half = (warp - kEpiWarp0) >> 2;       // and its columns
        const uint32_t tm_lane = tmem_base + ((uint32_t)(lq * 32) << 16);
        constexpr int kCols = BN / 2, kQ = kCols / 32;  // of this warp
        uint8_t *staging = smem + kStages * F::kStage + (warp - kEpiWarp0) * kBox;
        uint32_t tc = 0;
        bool ok = true;

        // A result leaves through this warp's staging, a box of 32 rows of 128 bytes (a
        // second one is worth less than the stage that it costs: 64 x 128000 x 4096
        // backward 624 us, 642 with two), 16-byte chunks swizzled as the copies expect
        // them (neither side meets a bank twice).  stage: 32 values of this lane's row to
        // one half (BF16) of the box or all of it; send: the box to row row0, columns x
        // and on.  What reaches over the matrix's edge is not written; a box beyond it is
        // not sent.
        auto free_box = [&] {
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
        };
        auto stage = [&](const uint32_t (&r)[32], int half_box, bool f32) {
            uint8_t *to = staging + lane * 128;
            if (f32) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<uint4 *>(to + ((j ^ (lane & 7)) << 4)) = make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4 *>(to + (((j + 4 * half_box) ^ (lane & 7)) << 4)) = bf16x8(r + 8 * j);
            }
        };
        auto send = [&](const CUtensorMap *to, int x, int row0, int cols, int rows_end, bool add) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane != 0 || row0 >= rows_end || x >= cols) return;
            if (add) tma_reduce_add_2d(to, staging, x, row0);
            else tma_store_2d(to, staging, x, row0);
            bulk_commit_group();
        };

        auto settle = [](auto &v) {     // loaded values are not used before the wait for them
#pragma unroll
            for (uint32_t &e : v) asm volatile("" : "+r"(e));
        };

        // What this lane has to know of its row (LOSS: the target), fetched a tile ahead
        // where the rows of tiles change.
        auto fetch = [&](int mt) {
            const int row = mt * F::kM + rank * 128 + lq * 32 + lane;
            float4 i = make_float4(0.0f, 0.0f, 0.0f, __int_as_float(-1));
            if constexpr (MODE == XENT_GRAD) {
                if (row < rows && a.info) {
                    i = a.info[row];
                } else if (row < rows) {
                    const int target = a.target[row];
                    float by;
                    if (target >= 0 && target < a.vocab)
                        i = row_info(a.scale, a.loss[row], a.lse[row], a.dloss[row], a.dlse ? a.dlse[row] : 0.0f, target, by);
                }
            } else if constexpr (MODE == XENT_LOSS) {
                if (row < rows) i.w = __int_as_float(a.target[row]);
            }
            return i;
        };
        // Up to 128 tokens: what k_xent_pack does of the work else, while the first tiles come.  Tokens that do
        // not count keep their rows, of zeros (norm 0).
        if (MODE == XENT_GRAD && !PAIR && a.xn) {
            const int e = warp - kEpiWarp0, nv = a.dim / 8;
            for (int r = blockIdx.x; r < (rows + kBK - 1) / kBK * kBK; r += gridDim.x) {
                const int target = r < rows ? a.target[r] : -1;
                const bool counts = target >= 0 && target < a.vocab;
                float by = 0.0f;
                if (counts) row_info(a.scale, a.loss[r], a.lse[r], a.dloss[r], a.dlse ? a.dlse[r] : 0.0f, target, by);
                if (e == 0 && lane == 0 && r < rows) {
                    if (target >= a.vocab) set_status(a.status, FP8_ERR_INVALID_ARG);
                    if (dbg_span(r, 1, a.rows, a.status)) a.norm[r] = by;
                }
                for (int v = e * 32 + lane; v < nv; v += kEpiWarps * 32) {
                    const uint4 q = counts ? times8(ldg_stream(a.x + r * a.ldx + v * 8), by) : make_uint4(0, 0, 0, 0);
                    if (dbg_cell(r, v * 8, 8, a.rows, a.dim, a.status)) *reinterpret_cast<uint4 *>(a.xn + (int64_t)r * a.dim + v * 8) = q;
                }
            }
        }
        int at_mt = -1, ahead_mt = -1;
        float4 info, ahead;
        const float c = a.scale * kLog2e;
        walk.each(ok, [&](const Unit &t, int next_mt) {
            const int row0 = t.mt * F::kM + rank * 128 + lq * 32, row = row0 + lane;
            if (MODE <= XENT_GRAD) {
                if (t.mt != at_mt) info = t.mt == ahead_mt ? ahead : fetch(t.mt);
                at_mt = t.mt;
                if (next_mt >= 0 && next_mt != at_mt) {
                    ahead = fetch(next_mt);
                    ahead_mt = next_mt;
                }
            }
            const int target = __float_as_int(info.w) - a.v0;
            float top = -INFINITY, sum = 0.0f;              // LOSS
            for (int nt = t.nt0; nt < t.nt1; ++nt, ++tc) {
                auto full_accumulator = [&] {
                    const bool there = __all_sync(0xffffffffu, thread_wait(smem_u32(&tfull[tc & 1]), (tc >> 1) & 1, abort_flag, a.status));
                    tc_fence_after();
                    return there;
                };
                auto release = [&] {    // the next accumulation but one may have it
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (PAIR) mbar_arrive_cluster(cluster_addr(&tempty[tc & 1], 0));
                        else mbar_arrive(&tempty[tc & 1]);
                    }
                };
                if (!(ok = full_accumulator())) return;
                const int col0 = nt * BN + half * kCols;    // in the piece, or of dx / dw
                auto load = [&](uint32_t (&to)[32], int q) { tc_ld_32x32b_x32(tm_lane + (tc & 1) * BN + half * kCols + q * 32, to); };
                // f(v, q) for every 32 columns, the next ones on their way meanwhile
                auto each_32 = [&](auto &&f) {
                    uint32_t v[2][32];
                    load(v[0], 0);
                    tc_wait_ld();
                    settle(v[0]);
#pragma unroll
                    for (int q = 0; q < kQ; ++q) {
                        if (q + 1 < kQ) load(v[(q + 1) & 1], q + 1);
                        f(v[q & 1], q);
                        if (q + 1 < kQ) {
                            tc_wait_ld();
                            settle(v[(q + 1) & 1]);
                            if (q + 2 == kQ) release();
                        }
                    }
                };
                // all columns in one go, of the sum of `chunks` accumulators
                auto load_all = [&](uint32_t (&r)[kQ][32], int chunks) {
#pragma unroll
                    for (int q = 0; q < kQ; ++q) load(r[q], q);
                    tc_wait_ld();
#pragma unroll
                    for (int q = 0; q < kQ; ++q) settle(r[q]);
                    release();
                    for (int i = 1; i < chunks; ++i) {
                        ++tc;
                        if (!full_accumulator()) return false;
#pragma unroll
                        for (int h = 0; h < 2 * kQ; ++h) {      // by 16: 32 more registers are not there
                            uint32_t v[16];
                            tc_ld_32x32b_x16(tm_lane + (tc & 1) * BN + half * kCols + h * 16, v);
                            tc_wait_ld();
                            settle(v);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                uint32_t &to = r[h / 2][h % 2 * 16 + e];
                                to = __float_as_uint(__uint_as_float(to) + __uint_as_float(v[e]));
                            }
                        }
                        release();
                    }
                    return true;
                };
                if constexpr (MODE == XENT_LOSS) {
                    uint32_t r[kQ][32];
                    if (!(ok = load_all(r, loss_chunks))) return;
                    const int lim = a.vn - col0, at = target - col0;
                    if (lim < kCols || (unsigned)at < (unsigned)kCols) {    // beyond the vocabulary; the target is left out of the sum
#pragma unroll
                        for (int q = 0; q < kQ; ++q)
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (q * 32 + i >= lim || q * 32 + i == at) r[q][i] = __float_as_uint(-INFINITY);
                    }
                    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int q = 0; q < kQ; ++q)
#pragma unroll
                        for (int i = 0; i < 32; i += 2) m[i / 2 & 3] = max3(m[i / 2 & 3], __uint_as_float(r[q][i]), __uint_as_float(r[q][i + 1]));
                    const float high = max3(m[0], m[1], fmaxf(m[2], m[3])) * c;
                    if (high > top) {
                        sum *= ex2_approx_ftz(top - high);
                        top = high;
                    }
                    const float off = top == -INFINITY ? 0.0f : -top;
                    const uint64_t c2 = f2_pack(c, c), off2 = f2_pack(off, off);
                    uint64_t s[4] = {};
#pragma unroll
                    for (int q = 0; q < kQ; ++q)
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float x, y;
                            f2_unpack(f2_fma_bits(r[q][i], r[q][i + 1], c2, off2), x, y);
                            s[i / 2 & 3] = f2_add(s[i / 2 & 3], f2_pack(ex2_approx_ftz(x), ex2_approx_ftz(y)));
                        }
                    float s0, s1;
                    f2_unpack(f2_add(f2_add(s[0], s[1]), f2_add(s[2], s[3])), s0, s1);
                    sum += s0 + s1;
                } else if constexpr (MODE == XENT_GRAD) {
                    const uint64_t c2 = f2_pack(c, c), off2 = f2_pack(-info.x, -info.x), by2 = f2_pack(info.y, info.y);
                    each_32([&](uint32_t (&r)[32], int q) {
                        const int col = col0 + q * 32, at = target - col;
                        const int lim = __float_as_int(info.w) >= 0 ? a.vn - col : 0;
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float x, y;
                            f2_unpack(f2_fma_bits(r[i], r[i + 1], c2, off2), x, y);
                            f2_unpack(f2_mul_bits(__float_as_uint(ex2_approx_ftz(x)), __float_as_uint(ex2_approx_ftz(y)), by2), x, y);
                            r[i] = __float_as_uint(x);
                            r[i + 1] = __float_as_uint(y);
                        }
                        if (lim < 32 || (unsigned)at < 32u) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                if (i == at) r[i] = __float_as_uint(info.z);
                                if (i >= lim) r[i] = 0;
                            }
                        }
                        if (q % 2 == 0) free_box();
                        stage(r, q % 2, false);
                        if (q % 2 == 1) send(&maps.m[2], col - 32, row0, INT_MAX, INT_MAX, false);
                    });
                } else {
                    uint32_t r[kQ][32];
                    if (!(ok = load_all(r, LONG ? chunks_of(t.k1 - t.k0) : 1))) return;
                    if (t.k0 == t.k1) {         // no K: the accumulator was not written
#pragma unroll
                        for (int q = 0; q < kQ; ++q)
#pragma unroll
                            for (int i = 0; i < 32; ++i) r[q][i] = 0;
                    }
                    const bool f32 = !t.dw || a.dw_f32, add = t.dw ? a.dw_add : a.dx_add;
                    const CUtensorMap *map = &maps.m[t.dw ? 5 : 2];
                    const int to = t.dw ? a.v0 + row0 : (int)(t.split * a.rows) + row0, end = t.dw ? a.vocab : INT_MAX;
                    if (f32) {
#pragma unroll
                        for (int q = 0; q < kQ; ++q) {
                            free_box();
                            stage(r[q], 0, true);
                            send(map, col0 + 32 * q, to, a.dim, end, add);
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < kQ; ++q) {
                            if (q % 2 == 0) free_box();
                            stage(r[q], q % 2, false);
                            if (q % 2 == 1) send(map, col0 + 32 * (q - 1), to, a.dim, end, false);
                        }
                    }
                }
            }
            if (MODE == XENT_LOSS && row < a.rows) {
                const int64_t at = (int64_t)(t.nt0 / walk.p.per * 2 + half) * a.rows + row;
                if (dbg_span(at, 1, (int64_t)walk.p.num_ng * 2 * a.rows, a.status)) a.part[at] = make_float2(top, sum);
            }
        });
        if (lane == 0) bulk_wait_all();     // the results are there before the kernel is done
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();   // neither CTA leaves while the other may still signal it
    if (warp == 1) {
        tc_fence_after();
        if (PAIR) tmem_dealloc_pair(tmem_base, 2 * BN);
        else tmem_dealloc(tmem_base, 2 * BN);
    }
}

// ---------------------------------------------------------------------------
// Forward of up to 4 tokens: bound by reading W once, so it is read straight into
// registers and multiplied there in FP32.  A warp takes 4 rows of W at a time, x
// lies in shared memory as FP32 (each vector of 8 in two halves, so that lanes read
// neighbouring 16 bytes); every CTA leaves one maximum and sum a token.  No tensor
// memory, no barriers to set up, and W's lines are not waited for behind those of x,
// which all SMs would ask one place of the L2 for (1 x 128000 x 4096: 208 us on the
// tensor cores).
// ---------------------------------------------------------------------------
constexpr int kFewTokens = 4, kFewRows = 4, kFewThreads = 256, kFewSmem = 96 * 1024;

template <int T>
__global__ void __launch_bounds__(kFewThreads, 2) k_xent_few(const uint16_t *__restrict__ x, int64_t ldx, const uint16_t *__restrict__ w, int64_t ldw,
                                                          const int32_t *__restrict__ target, int tokens, int vocab, int dim, float scale,
                                                          float2 *__restrict__ part, int64_t rows, int *status)
{
    extern __shared__ __align__(16) float4 xs[];    // [T][2][dim / 8]
    __shared__ float2 warps[kFewThreads / 32][T];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nv = dim / 8;
    dependency_wait();
    dependents_launch();        // k_xent_join reads this call's inputs before it waits
    for (int i = threadIdx.x; i < T * nv; i += kFewThreads) {
        const int t = i / nv, v = i - t * nv;
        const uint4 q = t < tokens ? *(reinterpret_cast<const uint4 *>(x + t * ldx) + v) : make_uint4(0, 0, 0, 0);
        xs[(2 * t) * nv + v] = make_float4(bf16_lo(q.x), bf16_hi(q.x), bf16_lo(q.y), bf16_hi(q.y));
        xs[(2 * t + 1) * nv + v] = make_float4(bf16_lo(q.z), bf16_hi(q.z), bf16_lo(q.w), bf16_hi(q.w));
    }
    int at[T];
    float top[T], sum[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
        at[t] = t < tokens ? target[t] : -1;
        top[t] = -INFINITY;
        sum[t] = 0.0f;
    }
    __syncthreads();
    const float c = scale * kLog2e;
    const int groups = (vocab + kFewRows - 1) / kFewRows;
    for (int g = blockIdx.x * (kFewThreads / 32) + warp; g < groups; g += gridDim.x * (kFewThreads / 32)) {
        const int v0 = g * kFewRows;
        const uint4 *row[kFewRows];
#pragma unroll
        for (int r = 0; r < kFewRows; ++r) row[r] = reinterpret_cast<const uint4 *>(w + (int64_t)min(v0 + r, vocab - 1) * ldw);
        uint64_t acc[kFewRows][T] = {};     // packed pairs
#pragma unroll 2
        for (int v = lane; v < nv; v += 32) {
            uint4 q[kFewRows];
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) q[r] = ldg_stream(row[r] + v);
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const float4 a = xs[(2 * t) * nv + v], b = xs[(2 * t + 1) * nv + v];
                const uint64_t p[4] = {p2(a.x, a.y), p2(a.z, a.w), p2(b.x, b.y), p2(b.z, b.w)};
#pragma unroll
                for (int r = 0; r < kFewRows; ++r) {
                    const uint32_t k[4] = {q[r].x, q[r].y, q[r].z, q[r].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[r][t] = p2_fma(p2_bf16x2(k[e]), p[e], acc[r][t]);
                }
            }
        }
        float z[kFewRows][T];
#pragma unroll
        for (int r = 0; r < kFewRows; ++r)
#pragma unroll
            for (int t = 0; t < T; ++t) {
                float lo, hi;
                f2_unpack(acc[r][t], lo, hi);
                z[r][t] = lo + hi;
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int r = 0; r < kFewRows; ++r)
#pragma unroll
                for (int t = 0; t < T; ++t) z[r][t] += __shfl_xor_sync(0xffffffffu, z[r][t], o);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            float high = top[t];
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) {
                z[r][t] = v0 + r < vocab && v0 + r != at[t] ? z[r][t] * c : -INFINITY;
                high = fmaxf(high, z[r][t]);
            }
            const float off = high == -INFINITY ? 0.0f : high;
            sum[t] *= ex2_approx_ftz(top[t] - off);
            top[t] = high;
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) sum[t] += ex2_approx_ftz(z[r][t] - off);
        }
    }
    if (lane == 0)
#pragma unroll
        for (int t = 0; t < T; ++t) warps[warp][t] = make_float2(top[t], sum[t]);
    __syncthreads();
    if ((int)threadIdx.x >= min(T, tokens)) return;
    float M = -INFINITY, S = 0.0f;
    for (int i = 0; i < kFewThreads / 32; ++i) M = fmaxf(M, warps[i][threadIdx.x].x);
    for (int i = 0; i < kFewThreads / 32; ++i) S += warps[i][threadIdx.x].y * exp2f(warps[i][threadIdx.x].x - (M == -INFINITY ? 0.0f : M));
    if (dbg_cell(blockIdx.x, threadIdx.x, 1, gridDim.x, rows, status)) part[(int64_t)blockIdx.x * rows + threadIdx.x] = make_float2(M, S);
}

// ---------------------------------------------------------------------------
// Backward of up to 4 tokens, W read and dw written once (k_xent reads W twice:
// 1 x 128000 x 4096 616 us, 350 here; 1 x 1151 x 440 21 and 6) and everything in FP32.  A team of warps,
// 8 columns a thread, takes R rows of W at a time: their logits by a reduction over
// the team (halving the values with every exchange, so that each lane ends with one),
// g by each warp for itself, then g x to dw and g w to the thread's sums of dx.  The
// CTAs' sums of dx are added in order by k_xent_few_dx.
// ---------------------------------------------------------------------------
constexpr int kFewGradThreads = 512, kFewGradDim = 8 * kFewGradThreads;

enum { DW_F32 = 0, DW_ADD = 1, DW_BF16 = 2 };

struct FewGradArgs {
    const uint16_t *x, *w;
    int64_t ldx, ldw, lddw;
    const int32_t *target;
    const float *loss, *lse, *dloss, *dlse;
    int tokens, vocab, dim;
    float scale;
    void *dw;
    float *part;            // [CTA][T][dim]: sums of dx
    int team_warps, teams;
    int *status;
};

template <int T, int OUT>
__global__ void __launch_bounds__(kFewGradThreads, 1) k_xent_few_grad(const FewGradArgs a)
{
    constexpr int R = kFewRows, N = R * T, kLanes = 32 / N;     // N values, kLanes lanes each
    extern __shared__ float dxs[];          // [team][T][columns]
    __shared__ float sums[2][kFewGradThreads / 32][N];
    dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, team = warp / a.team_warps, first_warp = team * a.team_warps;
    const int col = (threadIdx.x - first_warp * 32) * 8, cols = a.team_warps * 256;
    const bool in = col < a.dim;
    auto counts = [&](int t) { return t < a.tokens && a.target[t] >= 0 && a.target[t] < a.vocab; };
    if (blockIdx.x == 0 && (int)threadIdx.x < a.tokens && a.target[threadIdx.x] >= a.vocab) set_status(a.status, FP8_ERR_INVALID_ARG);
    uint64_t x[T][4], dx[T][4] = {};
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const uint4 q = in && counts(t) ? *reinterpret_cast<const uint4 *>(a.x + t * a.ldx + col) : make_uint4(0, 0, 0, 0);
        x[t][0] = p2_bf16x2(q.x);
        x[t][1] = p2_bf16x2(q.y);
        x[t][2] = p2_bf16x2(q.z);
        x[t][3] = p2_bf16x2(q.w);
    }
    // this lane's value: of row `row` and token `token`
    const int value = lane / kLanes, row = value / T, token = value % T;
    const float c = a.scale * kLog2e;
    const bool counted = counts(token);
    int target = -1;
    float lse2 = 0.0f, factor = 0.0f, entry = 0.0f;
    if (counted) {
        const float gl = a.dloss[token], gz = a.dlse ? a.dlse[token] : 0.0f;
        target = a.target[token];
        lse2 = a.lse[token] * kLog2e;
        factor = a.scale * (gl + gz);
        entry = target_entry(a.scale, a.loss[token], gl, gz);
    }
    const int groups = (a.vocab + R - 1) / R, step = gridDim.x * a.teams;
    auto fetch = [&](int group, uint4 (&to)[R]) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t v = (int64_t)group * R + r;
            to[r] = in && v < a.vocab ? ldg_stream(a.w + v * a.ldw + col) : make_uint4(0, 0, 0, 0);
        }
    };
    uint4 q[R];
    int group = blockIdx.x * a.teams + team;
    fetch(group, q);
    for (int k = 0; group < groups; group += step, k ^= 1) {
        uint4 next[R];
        fetch(group + step, next);
        float z[N];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint64_t w[4] = {p2_bf16x2(q[r].x), p2_bf16x2(q[r].y), p2_bf16x2(q[r].z), p2_bf16x2(q[r].w)};
#pragma unroll
            for (int t = 0; t < T; ++t) {
                uint64_t acc = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) acc = p2_fma(w[e], x[t][e], acc);
                float lo, hi;
                f2_unpack(acc, lo, hi);
                z[r * T + t] = lo + hi;
            }
        }
#pragma unroll
        for (int o = 16, n = N / 2; o > 0; o >>= 1, n >>= 1) {
            if (n > 0) {
                const bool upper = lane & o;
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const float keep = upper ? z[i + n] : z[i], give = upper ? z[i] : z[i + n];
                    z[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
            } else {
                z[0] += __shfl_xor_sync(0xffffffffu, z[0], o);
            }
        }
        float logit = z[0];
        if (a.team_warps > 1) {
            if (lane % kLanes == 0) sums[k][warp][value] = logit;
            named_bar_sync(1 + team, a.team_warps * 32);
            logit = 0.0f;
            for (int i = 0; i < a.team_warps; ++i) logit += sums[k][first_warp + i][value];
        }
        const int v0 = group * R, v = v0 + row;
        float g = factor * ex2_approx_ftz(fmaf(logit, c, -lse2));
        if (v == target) g = entry;
        if (!counted || v >= a.vocab) g = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint64_t w[4] = {p2_bf16x2(q[r].x), p2_bf16x2(q[r].y), p2_bf16x2(q[r].z), p2_bf16x2(q[r].w)};
            uint64_t out[4] = {};
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const float gt = __shfl_sync(0xffffffffu, g, (r * T + t) * kLanes);
                const uint64_t g2 = f2_pack(gt, gt);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    out[e] = p2_fma(g2, x[t][e], out[e]);
                    dx[t][e] = p2_fma(g2, w[e], dx[t][e]);
                }
            }
            const int64_t at = (int64_t)(v0 + r) * a.lddw + col;
            if (!in || v0 + r >= a.vocab || !dbg_span(at, 8, (int64_t)(a.vocab - 1) * a.lddw + a.dim, a.status)) continue;
            float f[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) f2_unpack(out[e], f[2 * e], f[2 * e + 1]);
            if (OUT == DW_BF16) {
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.dw) + at) =
                    make_uint4(bf16x2_rn(f[0], f[1]), bf16x2_rn(f[2], f[3]), bf16x2_rn(f[4], f[5]), bf16x2_rn(f[6], f[7]));
            } else {
                float *to = static_cast<float *>(a.dw) + at;
#pragma unroll
                for (int h = 0; h < 8; h += 4) {
                    if (OUT == DW_ADD)
                        asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(to + h), "f"(f[h]), "f"(f[h + 1]),
                                     "f"(f[h + 2]), "f"(f[h + 3])
                                     : "memory");
                    else
                        *reinterpret_cast<float4 *>(to + h) = make_float4(f[h], f[h + 1], f[h + 2], f[h + 3]);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) q[r] = next[r];
    }
    dependents_launch();
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float lo, hi;
            f2_unpack(dx[t][e], lo, hi);
            *reinterpret_cast<float2 *>(&dxs[(team * T + t) * cols + col + 2 * e]) = make_float2(lo, hi);
        }
    __syncthreads();
    for (int i = threadIdx.x; i < T * cols; i += blockDim.x) {
        const int t = i / cols, at = i - t * cols;
        float sum = 0.0f;
        for (int m = 0; m < a.teams; ++m) sum += dxs[(m * T + t) * cols + at];
        if (at < a.dim && dbg_cell(blockIdx.x * T + t, at, 1, (int64_t)gridDim.x * T, a.dim, a.status))
            a.part[((int64_t)blockIdx.x * T + t) * a.dim + at] = sum;
    }
}

// dx: a CTA for 32 columns of a token, a warp for every eighth of the parts.
__global__ void __launch_bounds__(256) k_xent_few_dx(const float *__restrict__ part, int parts, int T, const int32_t *__restrict__ target, int vocab,
                                                  int dim, uint16_t *__restrict__ dx, int64_t lddx, int tokens, int *status)
{
    __shared__ float sums[8][32];
    dependents_launch();
    dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = blockIdx.y, col = blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (col < dim) {
#pragma unroll 10
        for (int i = warp; i < parts; i += 8) sum += part[((int64_t)i * T + t) * dim + col];
    }
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp != 0 || col >= dim) return;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += sums[i][lane];
    if (target[t] < 0 || target[t] >= vocab) sum = 0.0f;       // whatever W holds
    if (dbg_span(t * lddx + col, 1, (tokens - 1) * lddx + dim, status)) dx[t * lddx + col] = (uint16_t)bf16x2_rn(sum, 0.0f);
}

// ---------------------------------------------------------------------------
// The counted tokens' rows of x, one behind another, and the token of each.  Every CTA takes a range of tokens and
// counts the ones before it by itself.  Rows of the outputs that belong to
// tokens left out are zeroed here.
// ---------------------------------------------------------------------------
struct PackArgs {
    const int32_t *target;
    const uint16_t *x;
    int64_t ldx;
    int tokens, vocab, dim;
    uint16_t *xp;               // [rows][dim]
    int64_t rows;
    int32_t *map;
    int *count;
    float *loss, *lse;          // forward: zeroed where a token does not count
    uint16_t *dx;               // backward: the same
    int64_t lddx;
    const float *losses, *lses, *dloss, *dlse;      // backward
    float scale;
    int32_t *row_target;        // forward: [rows], the target of each row
    float *norm;                // backward: [rows], the size of g at the target,
    float4 *info;               // and what its gradient is made of
    uint16_t *xn;               // [rows][dim]: x times it
    int *status;
};

__global__ void __launch_bounds__(256) k_xent_pack(PackArgs g)
{
    __shared__ int warp_n[8];
    __shared__ int32_t src[256];
    __shared__ float by[256];
    dependents_launch();
    dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (g.tokens + gridDim.x - 1) / gridDim.x;
    const int t0 = min(g.tokens, (int)blockIdx.x * per), t1 = min(g.tokens, t0 + per);
    auto counts = [&](int t) { const int v = g.target[t]; return v >= 0 && v < g.vocab; };
    auto cta_sum = [&](int n) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        __syncthreads();
        if (lane == 0) warp_n[warp] = n;
        __syncthreads();
        n = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) n += warp_n[i];
        return n;
    };
    int n = 0, all = 0;
#pragma unroll 8
    for (int t = threadIdx.x; t < g.tokens; t += 256) {
        const int c = counts(t);
        all += c;
        n += t < t0 ? c : 0;
    }
    int at = cta_sum(n);
    all = cta_sum(all);
    const int nv = g.dim / 8;
    for (int base = t0; base < t1; base += 256) {
        const int t = base + threadIdx.x;
        const bool mine = t < t1, in = mine && counts(t);
        if (mine && g.target[t] >= g.vocab) set_status(g.status, FP8_ERR_INVALID_ARG);
        const unsigned votes = __ballot_sync(0xffffffffu, in);
        __syncthreads();
        if (lane == 0) warp_n[warp] = __popc(votes);
        __syncthreads();
        int before = __popc(votes & ((1u << lane) - 1)), total = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i < warp) before += warp_n[i];
            total += warp_n[i];
        }
        if (in) {
            src[before] = t;
            const bool fits = dbg_span(at + before, 1, g.rows, g.status);
            if (fits) g.map[at + before] = t;
            if (fits && g.row_target) g.row_target[at + before] = g.target[t];
            if (g.norm) {
                const float4 info = row_info(g.scale, g.losses[t], g.lses[t], g.dloss[t], g.dlse ? g.dlse[t] : 0.0f, g.target[t], by[before]);
                if (fits) {
                    g.norm[at + before] = by[before];
                    g.info[at + before] = info;
                }
            }
        } else if (mine && g.loss) {
            if (dbg_span(t, 1, g.tokens, g.status)) g.loss[t] = g.lse[t] = 0.0f;
        }
        __syncthreads();
        for (int r = warp; r < total; r += 8) {
            const uint16_t *from = g.x + (int64_t)src[r] * g.ldx;
            for (int v0 = lane; v0 < nv; v0 += 128) {
                uint4 x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = v0 + 32 * i < nv ? ldg_stream(from + (v0 + 32 * i) * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int v = v0 + 32 * i;
                    if (v >= nv || !dbg_cell(at + r, v * 8, 8, g.rows, g.dim, g.status)) continue;
                    *reinterpret_cast<uint4 *>(g.xp + (int64_t)(at + r) * g.dim + v * 8) = x[i];
                    if (g.xn) *reinterpret_cast<uint4 *>(g.xn + (int64_t)(at + r) * g.dim + v * 8) = times8(x[i], by[r]);
                }
            }
        }
        if (g.dx)
            for (int r = warp; r < min(256, t1 - base); r += 8)
                if (!counts(base + r))
                    for (int v = lane; v < nv; v += 32)
                        if (dbg_span((base + r) * g.lddx + v * 8, 8, (g.tokens - 1) * g.lddx + g.dim, g.status))
                            *reinterpret_cast<uint4 *>(g.dx + (base + r) * g.lddx + v * 8) = make_uint4(0, 0, 0, 0);
        at += total;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *g.count = all;
    // dw's last K block reads on: zeros there.  (What lies behind xp's rows only makes rows that nobody looks at.)
    const int end = g.xn ? (all + kBK - 1) / kBK * kBK : 0;
    for (int r = all + blockIdx.x * 8 + warp; r < end; r += gridDim.x * 8)
        for (int v = lane; v < nv; v += 32)
            if (dbg_cell(r, v * 8, 8, g.rows, g.dim, g.status))
                *reinterpret_cast<uint4 *>(g.xn + (int64_t)r * g.dim + v * 8) = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// Forward, last step: a CTA adds a row's parts in a fixed order (M, S: maximum
// and sum without the target) and forms the target's logit by itself, in FP32
// with a rounding to nearest for every addition: the tensor cores' sums lean
// towards zero by up to a last place a step, 3e-6 of a logit of 16 at dim 4096,
// and the loss would inherit it.  That logit is formed before k_xent has ended.
// ---------------------------------------------------------------------------
struct JoinArgs {
    const float2 *part;
    int parts;
    int64_t rows;
    const int *count;
    const int32_t *map, *target;
    const uint16_t *x, *w;      // as k_xent read them: packed rows where there is a map
    int64_t ldx, ldw;
    int tokens, vocab, dim;
    float scale;
    float *loss, *lse;
    int *status;
};

__device__ __forceinline__ float dot8(uint4 a, uint4 b, float acc)
{
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) acc = fmaf(bf16_hi(x[k]), bf16_hi(y[k]), fmaf(bf16_lo(x[k]), bf16_lo(y[k]), acc));
    return acc;
}

constexpr int kJoinThreads = 128;

__global__ void __launch_bounds__(kJoinThreads) k_xent_join(JoinArgs g)
{
    __shared__ float dots[4], tops[4], sums[4];
    dependents_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.x;
    const bool here = row < (g.count ? *g.count : g.tokens);
    const int t = here ? (g.map ? g.map[row] : row) : 0, at = here ? g.target[t] : -1;
    const bool counts = at >= 0 && at < g.vocab;
    float dot = 0.0f, M = -INFINITY, S = 0.0f;
    if (counts) {
        const uint4 *px = reinterpret_cast<const uint4 *>(g.x + (int64_t)row * g.ldx), *pw = reinterpret_cast<const uint4 *>(g.w + (int64_t)at * g.ldw);
        const int nv = g.dim / 8;
#pragma unroll 4
        for (int v = threadIdx.x; v < nv; v += kJoinThreads) dot = dot8(px[v], pw[v], dot);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    dependency_wait();      // k_xent's sums
    const float2 *part = g.part + row;
    if (counts)
#pragma unroll 4
        for (int u = threadIdx.x; u < g.parts; u += kJoinThreads) M = fmaxf(M, part[u * g.rows].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) {
        dots[warp] = dot;
        tops[warp] = M;
    }
    __syncthreads();
    M = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    const float off = M == -INFINITY ? 0.0f : M;    // -inf: no other logit, or all of them -inf (or NaN); S is 0 then (or NaN)
    if (counts)
#pragma unroll 4
        for (int u = threadIdx.x; u < g.parts; u += kJoinThreads) {
            const float2 p = part[u * g.rows];
            S += p.y * exp2f(p.x - off);
        }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
    if (lane == 0) sums[warp] = S;
    __syncthreads();
    if (threadIdx.x != 0 || !here) return;
    float l = 0.0f, z = 0.0f;
    if (counts) {
        S = (sums[0] + sums[1]) + (sums[2] + sums[3]);
        const float zt = ((dots[0] + dots[1]) + (dots[2] + dots[3])) * g.scale, yt = zt * kLog2e;
        if (yt >= M) {          // the target leads: log(1 + the rest relative to it)
            l = log1pf(S * exp2f(M - yt));      // 0 times 0 where there is no rest, however small yt; NaN where there is nothing at all
            z = S == 0.0f ? zt : zt + l;
        } else {
            const float s = logf(S + exp2f(yt - M));
            l = (M - yt) * kLn2 + s;
            z = M * kLn2 + s;
        }
        if (zt != zt || zt == INFINITY) l = z = NAN;
    } else if (at >= g.vocab) {
        set_status(g.status, FP8_ERR_INVALID_ARG);
    }
    if (dbg_span(t, 1, g.tokens, g.status)) {
        g.loss[t] = l;
        g.lse[t] = z;
    }
}

// Backward, last step: the parts of dx's K added in a fixed order, times what their row
// is relative to, rounded to BF16, each row where its token is.  LANES threads share
// the parts of 8 columns.
constexpr int kSumThreads = 128;

template <int LANES>
__global__ void __launch_bounds__(kSumThreads) k_xent_dx_join(const float *acc, int splits, int64_t rows, const int *count, const int32_t *map,
                                                    const float *norm, int dim,
                                                    uint16_t *dx, int64_t lddx, int tokens, int *status)
{
    dependents_launch();
    dependency_wait();
    const int nv = dim / 8;
    const int64_t items = (int64_t)(count ? *count : tokens) * nv;
    // whole warps go round, for the exchange
    for (int64_t i = (int64_t)blockIdx.x * kSumThreads + threadIdx.x; (i & ~(int64_t)31) < items * LANES; i += (int64_t)gridDim.x * kSumThreads) {
        const bool valid = i < items * LANES;
        const int64_t item = valid ? i / LANES : 0, row = item / nv;
        const int col = (int)(item - row * nv) * 8;
        float v[8] = {};
        if (valid) {
#pragma unroll 8
            for (int s = i % LANES; s < splits; s += LANES) {
                const float4 *p = reinterpret_cast<const float4 *>(acc + (s * rows + row) * dim + col);
                const float4 x = p[0], y = p[1];
                v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
                v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
            }
        }
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += __shfl_xor_sync(0xffffffffu, v[e], o);
        if (!valid || i % LANES != 0) continue;
        const int64_t at = (map ? map[row] : row) * lddx + col;
        const float by = norm[row];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = by == 0.0f ? 0.0f : v[e] * by;      // 0: does not count, whatever W holds
        if (dbg_span(at, 8, (int64_t)(tokens - 1) * lddx + dim, status))
            *reinterpret_cast<uint4 *>(dx + at) = make_uint4(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]), bf16x2_rn(v[4], v[5]), bf16x2_rn(v[6], v[7]));
    }
}

// ------------------------------------------------------------------ launchers

namespace {

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Whether the forward packs its rows first: not where the whole product lasts
// about as long as the packing kernel (5 us), or all rows fit one tile.
bool packs(int64_t tokens, int64_t vocab, int64_t dim) { return tokens > kTile && tokens * vocab * dim > (int64_t)10000000000; }

// Up to 128 tokens, one CTA's tiles hold them all, and a pair's would be half
// empty: W streams past at 128 x BN tiles by single CTAs (64 x 128000 x 4096 forward:
// 175 us in pairs' tiles, 168 so, HBM's floor is 157).
// So do products that 128 x 128 tiles lay out over the SMs at once, whose length is a
// tile's (783 x 2512 x 304 forward: 10.0 us in pairs' tiles, 8.6 so; 170 x 1594 x 2040
// 19.0 and 16.8), unless W is most of what they read, which a pair fetches once for
// 256 rows (256 x 9000 x 1024: 12.8 and 13.8).
bool single(int64_t tokens, int64_t vocab)
{
    return tokens <= 128 || (vocab <= 16 * tokens && (tokens + 127) / 128 * ((vocab + 127) / 128) <= sm_count());
}

// Whether k_xent_few takes the forward: its x has to fit, twice an SM.
bool few(int64_t tokens, int64_t dim) { return tokens <= kFewTokens && (tokens > 2 ? 4 : tokens) * dim * 4 <= kFewSmem; }

// Whether k_xent_few_grad takes the backward, and the CTAs that it may have.  With 3
// or 4 tokens and one team an SM nothing hides a team's exchanges (4 x 128000 x 4096:
// 696 us, k_xent 617; x 2048, two teams: 339 and 322, but 3 x 3456 x 1672 21 and 32).
bool few_grad(int64_t tokens, int64_t dim) { return tokens <= 2 ? dim <= kFewGradDim : tokens <= kFewTokens && dim <= kFewGradDim / 2; }
int64_t few_grad_ctas(int64_t vocab) { return std::min<int64_t>(sm_count(), (vocab + kFewRows - 1) / kFewRows); }

// Elements of g that the workspace holds (224 MB), unless a tile's columns take more
// (8192 x 128000 x 4096 backward: 15.9 ms, with 192 MB 16.0, with 256 MB 15.8).
constexpr int64_t kGradMost = (int64_t)112 << 20;

// Tiles of a unit, `per` or more.  Short rows' products (8 cycles a tile and column of
// x) last less than a tile's epilogue (2100 cycles, and 1600 for a unit), and longer
// units are worth a less even share (4096 x 32000 x 256 forward: 84 us by single
// tiles, 64 by four; from dim 600 on nothing changes).
int longer_units(int per, int64_t mt, int64_t nt, int64_t groups, int64_t dim)
{
    auto cycles = [&](int64_t n) { return (mt * ((nt + n - 1) / n) + groups - 1) / groups * std::max(n * 8 * dim, n * 2100 + 1600); };
    while (per < 8 && cycles(2 * per) * 33 < cycles(per) * 32) per *= 2;
    return per;
}

// Sizes that follow from those of the call alone.  What is taken of the workspace
// does not shrink when a size grows, so it serves all smaller calls too.
struct XentPlan {
    int64_t rows;                   // of the packed buffers
    int bn;                         // columns of a tile over the vocabulary
    int per_unit, parts;            // forward: tiles of a unit, maxima and sums of a row
    int64_t piece;                  // backward: vocabulary of a piece
    int splits;                     // backward: parts of dx's K
    int64_t count, map, target, xp, xn, norm, info, part, g, acc, bytes;    // byte offsets
    XentPlan(int64_t tokens, int64_t vocab, int64_t dim, bool backward)
    {
        const bool one = single(tokens, vocab);
        rows = up(tokens, kTile);
        const int64_t mt = rows / kTile, groups = std::max(1, one ? sm_count() : sm_count() / 2);
        // narrower tiles where the wider ones would leave CTAs without any
        bn = one && (vocab + 255) / 256 < 2 * groups ? 128 : 256;
        const int64_t nt = (vocab + bn - 1) / bn;
        int64_t at = 0;
        auto take = [&](int64_t n) { const int64_t p = at; at += up(n, 256); return p; };
        count = take(16);
        map = take(rows * 4);
        target = take(rows * 4);
        xp = backward || packs(tokens, vocab, dim) ? take(rows * dim * 2) : 0;
        if (!backward) {
            // long units write less; 16 of them a group keep the groups' shares even
            per_unit = 8;
            while (per_unit > 1 && mt * ((nt + per_unit - 1) / per_unit) < 16 * groups) per_unit /= 2;
            per_unit = longer_units(per_unit, mt, nt, groups, dim);
            parts = (int)((nt + per_unit - 1) / per_unit) * 2;
            if (few(tokens, dim)) parts = (int)std::min<int64_t>((vocab + kFewRows * 8 - 1) / (kFewRows * 8), (int64_t)sm_count() * 2);
            // parts * mt: below 64 groups where units are shorter than 8 tiles
            const int64_t most = std::min(2 * mt * ((vocab + 127) / 128), std::max<int64_t>(32 * sm_count(), mt * ((vocab + 2047) / 2048)));
            part = take(2 * most * kTile * 8);
        } else {
            // pieces of equal length
            const int64_t most = std::max<int64_t>(kTile, kGradMost / rows / kTile * kTile);
            const int64_t pieces = (up(vocab, kTile) + most - 1) / most;
            piece = up((vocab + pieces - 1) / pieces, kTile);
            // dx's K is split until a part lasts no longer than a pair's share of dx and dw
            const int64_t nd = (dim + kTile - 1) / kTile, kv = piece / kBK, kt = std::max<int64_t>(kTileCost, (tokens + kBK - 1) / kBK);
            const int64_t share = (mt * nd * kv + piece / kTile * nd * kt) / std::max(1, sm_count() / 2);
            splits = (int)std::max<int64_t>(1, std::min((kv + share) / (share + 1), kv / 8));
            xn = take(rows * dim * 2);
            norm = take(rows * 4);
            info = take(rows * 16);
            g = take(std::min(rows * up(vocab, kTile), std::max(rows * kTile, kGradMost)) * 2);
            // splits: at most groups / (mt * nd) + 1, and kv / 8
            acc = take(std::min(std::max<int64_t>(1, up(vocab, kTile) / (8 * kBK)) * rows * dim, sm_count() / 2 * kTile * kTile + rows * dim) * 4);
        }
        bytes = backward ? std::max(at, xp + few_grad_ctas(vocab) * kFewTokens * dim * 4) : at;      // k_xent_few_grad's part lies at xp
    }
};

template <int T, int OUT>
int run_few_grad(FewGradArgs &a, void *dx, int64_t lddx, cudaStream_t st)
{
    a.team_warps = (a.dim + 255) / 256;
    a.teams = kFewGradThreads / 32 / a.team_warps;
    const int threads = a.teams * a.team_warps * 32;
    const int64_t groups = (a.vocab + kFewRows - 1) / kFewRows, ctas = std::min((groups + a.teams - 1) / a.teams, few_grad_ctas(a.vocab));
    static bool attr_done[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (!attr_done[dev & 63]) {
        if (cudaFuncSetAttribute(k_xent_few_grad<T, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewGradThreads * 8 * T * 4) != cudaSuccess)
            return FP8_ERR_CUDA;
        attr_done[dev & 63] = true;
    }
    const int rc = launch_dependent(k_xent_few_grad<T, OUT>, dim3((unsigned)ctas), threads, (size_t)threads * 8 * T * 4, st, a);
    if (rc != FP8_OK) return rc;
    return launch_dependent(k_xent_few_dx, dim3((unsigned)((a.dim + 31) / 32), (unsigned)a.tokens), 256, 0, st, a.part, (int)ctas, T, a.target,
                            a.vocab, a.dim, static_cast<uint16_t *>(dx), lddx, a.tokens, a.status);
}

template <int MODE, bool PAIR, int BN, bool LONG = false>
int run(const Maps<MODE> &maps, const XentArgs &a, cudaStream_t st)
{
    using F = Form<MODE, PAIR, BN>;
    static bool attr_done[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (!attr_done[dev & 63]) {
        if (cudaFuncSetAttribute(k_xent<MODE, PAIR, BN, LONG>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::kSmem) != cudaSuccess) return FP8_ERR_CUDA;
        attr_done[dev & 63] = true;
    }
    const int sms = sm_count();
    return launch_dependent_cluster(k_xent<MODE, PAIR, BN, LONG>, dim3((unsigned)(PAIR ? sms / 2 * 2 : sms)), PAIR ? 2 : 1, kThreads, F::kSmem, st, maps,
                                    a);
}

template <int T>
int run_few(const void *x, int64_t ldx, const void *w, int64_t ldw, const int32_t *target, int64_t tokens, int64_t vocab, int64_t dim, float scale,
            float2 *part, const XentPlan &p, int *status, cudaStream_t st)
{
    static bool attr_done[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (!attr_done[dev & 63]) {
        if (cudaFuncSetAttribute(k_xent_few<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem) != cudaSuccess) return FP8_ERR_CUDA;
        attr_done[dev & 63] = true;
    }
    return launch_dependent(k_xent_few<T>, dim3((unsigned)p.parts), kFewThreads, (size_t)(T * dim * 4), st, static_cast<const uint16_t *>(x), ldx,
                            static_cast<const uint16_t *>(w), ldw, target, (int)tokens, (int)vocab, (int)dim, scale, part, p.rows, status);
}

// Rows of x in a copy: up to 128 tokens all that there are, since a copy that lies
// mostly outside its matrix is slow (14 x 67014 x 1896 forward: 84 us with 128 rows, 52
// with 16; from 128 tokens on smaller copies gain nothing).
int x_box(int64_t tokens) { return (int)std::min<int64_t>(128, up(tokens, 8)); }

// K-major operand: rows of K, `box` of them a copy; MN-major: rows along K, boxes of 64 columns.
bool map_k(CUtensorMap *m, const void *p, int64_t cols, int64_t rows, int64_t ld, int box = 128)
{
    return make_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, (uint64_t)cols, (uint64_t)rows, (uint64_t)ld * 2, kBK, (uint32_t)box,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}
bool map_mn(CUtensorMap *m, const void *p, int64_t cols, int64_t rows, int64_t ld)
{
    return make_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, (uint64_t)cols, (uint64_t)rows, (uint64_t)ld * 2, 64, kBK,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}
// Results: boxes of 32 rows of 128 bytes.
bool map_out(CUtensorMap *m, void *p, bool f32, int64_t cols, int64_t rows, int64_t ld)
{
    return make_map_2d(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, (uint64_t)cols, (uint64_t)rows,
                       (uint64_t)ld * (f32 ? 4 : 2), f32 ? 32 : 64, 32, CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

int pack(const XentPlan &p, uint8_t *ws, PackArgs &g, const int32_t *target, const void *x, int64_t ldx, int64_t tokens, int64_t vocab, int64_t dim,
         int *status, cudaStream_t st)
{
    g.target = target;
    g.x = static_cast<const uint16_t *>(x);
    g.ldx = ldx;
    g.tokens = (int)tokens;
    g.vocab = (int)vocab;
    g.dim = (int)dim;
    g.xp = reinterpret_cast<uint16_t *>(ws + p.xp);
    g.rows = p.rows;
    g.map = reinterpret_cast<int32_t *>(ws + p.map);
    g.count = reinterpret_cast<int *>(ws + p.count);
    g.status = status;
    const int64_t grid = std::min<int64_t>(std::max<int64_t>((tokens + 7) / 8, kBK / 8), (int64_t)sm_count() * 4);
    return launch_dependent(k_xent_pack, dim3((unsigned)grid), 256, 0, st, g);
}

}  // namespace

size_t linear_xent_workspace_bytes(int64_t tokens, int64_t vocab, int64_t dim, bool backward)
{
    return (size_t)XentPlan(tokens, vocab, dim, backward).bytes;
}

int launch_linear_xent_fwd(const void *x, int64_t ldx, const void *w, int64_t ldw, const int32_t *target, int64_t tokens, int64_t vocab,
                           int64_t dim, float scale, float *loss, float *lse, void *workspace, int *status, cudaStream_t st)
{
    const XentPlan p(tokens, vocab, dim, false);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    XentArgs a{};
    int rc;
    const void *xp = x;
    int64_t ldxp = ldx, xrows = tokens;
    const int32_t *map = nullptr;
    a.target = target;
    if (packs(tokens, vocab, dim)) {
        PackArgs g{};
        g.loss = loss;
        g.lse = lse;
        g.row_target = reinterpret_cast<int32_t *>(ws + p.target);
        if ((rc = pack(p, ws, g, target, x, ldx, tokens, vocab, dim, status, st)) != FP8_OK) return rc;
        xp = ws + p.xp;
        ldxp = dim;
        xrows = p.rows;
        a.count = reinterpret_cast<int *>(ws + p.count);
        map = reinterpret_cast<int32_t *>(ws + p.map);
        a.target = g.row_target;
    }
    a.part = reinterpret_cast<float2 *>(ws + p.part);
    a.rows = p.rows;
    if (few(tokens, dim)) {
        rc = tokens == 1 ? run_few<1>(x, ldx, w, ldw, target, tokens, vocab, dim, scale, a.part, p, status, st)
             : tokens == 2 ? run_few<2>(x, ldx, w, ldw, target, tokens, vocab, dim, scale, a.part, p, status, st)
                           : run_few<4>(x, ldx, w, ldw, target, tokens, vocab, dim, scale, a.part, p, status, st);
    } else {
        Maps<XENT_LOSS> maps;
        a.box = x_box(tokens);
        if (!map_k(&maps.m[0], xp, dim, xrows, ldxp, a.box) || !map_k(&maps.m[1], w, dim, vocab, ldw)) return FP8_ERR_CUDA;
        maps.m[2] = maps.m[0];      // there is no matrix to write
        a.tokens = (int)tokens;
        a.vocab = a.vn = (int)vocab;
        a.dim = (int)dim;
        a.per_unit = p.per_unit;
        a.splits = 1;
        a.band = 16;
        a.scale = scale;
        a.status = status;
        rc = !single(tokens, vocab) ? run<XENT_LOSS, true, 256>(maps, a, st)
             : p.bn == 256   ? run<XENT_LOSS, false, 256>(maps, a, st)
                             : run<XENT_LOSS, false, 128>(maps, a, st);
    }
    if (rc != FP8_OK) return rc;
    JoinArgs j{};
    j.part = a.part;
    j.parts = p.parts;
    j.rows = p.rows;
    j.count = a.count;
    j.map = map;
    j.target = target;
    j.x = static_cast<const uint16_t *>(xp);
    j.w = static_cast<const uint16_t *>(w);
    j.ldx = ldxp;
    j.ldw = ldw;
    j.tokens = (int)tokens;
    j.vocab = (int)vocab;
    j.dim = (int)dim;
    j.scale = scale;
    j.loss = loss;
    j.lse = lse;
    j.status = status;
    return launch_dependent(k_xent_join, dim3((unsigned)tokens), kJoinThreads, 0, st, j);
}

int launch_linear_xent_bwd(const void *x, int64_t ldx, const void *w, int64_t ldw, const int32_t *target, const float *loss, const float *lse,
                           const float *dloss, const float *dlse, int64_t tokens, int64_t vocab, int64_t dim, float scale, void *dx, int64_t lddx,
                           void *dw, int dw_dtype, int64_t lddw, int accumulate, void *workspace, int *status, cudaStream_t st)
{
    const XentPlan p(tokens, vocab, dim, true);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (few_grad(tokens, dim)) {
        FewGradArgs a{};
        a.x = static_cast<const uint16_t *>(x);
        a.w = static_cast<const uint16_t *>(w);
        a.ldx = ldx;
        a.ldw = ldw;
        a.lddw = lddw;
        a.target = target;
        a.loss = loss;
        a.lse = lse;
        a.dloss = dloss;
        a.dlse = dlse;
        a.tokens = (int)tokens;
        a.vocab = (int)vocab;
        a.dim = (int)dim;
        a.scale = scale;
        a.dw = dw;
        a.part = reinterpret_cast<float *>(ws + p.xp);
        a.status = status;
        auto with = [&](auto t) {
            constexpr int T = decltype(t)::value;
            return dw_dtype != FP8_OUT_F32 ? run_few_grad<T, DW_BF16>(a, dx, lddx, st)
                   : accumulate            ? run_few_grad<T, DW_ADD>(a, dx, lddx, st)
                                           : run_few_grad<T, DW_F32>(a, dx, lddx, st);
        };
        return tokens == 1   ? with(std::integral_constant<int, 1>{})
               : tokens == 2 ? with(std::integral_constant<int, 2>{})
                             : with(std::integral_constant<int, 4>{});
    }
    PackArgs pk{};
    pk.dx = static_cast<uint16_t *>(dx);
    pk.lddx = lddx;
    pk.losses = loss;
    pk.lses = lse;
    pk.dloss = dloss;
    pk.dlse = dlse;
    pk.scale = scale;
    pk.norm = reinterpret_cast<float *>(ws + p.norm);
    pk.info = reinterpret_cast<float4 *>(ws + p.info);
    pk.xn = reinterpret_cast<uint16_t *>(ws + p.xn);
    int rc = FP8_OK;
    XentArgs a{};
    const bool packed = tokens > 128;       // else the first launch does it (100 x 8000 x 256: 18 us, 21 with a packing launch)
    if (packed) {
        if ((rc = pack(p, ws, pk, target, x, ldx, tokens, vocab, dim, status, st)) != FP8_OK) return rc;
        a.count = reinterpret_cast<int *>(ws + p.count);
        a.info = pk.info;
    } else {
        a.target = target;
        a.loss = loss;
        a.lse = lse;
        a.dloss = dloss;
        a.dlse = dlse;
        a.x = static_cast<const uint16_t *>(x);
        a.ldx = ldx;
        a.xn = pk.xn;
        a.norm = pk.norm;
    }
    a.tokens = (int)tokens;
    a.vocab = (int)vocab;
    a.dim = (int)dim;
    a.splits = p.splits;
    a.scale = scale;
    a.rows = p.rows;
    a.status = status;
    const void *xp = packed ? ws + p.xp : x;
    void *g = ws + p.g, *acc = ws + p.acc;
    a.dw_f32 = dw_dtype == FP8_OUT_F32;
    a.dw_add = accumulate;
    Maps<XENT_GRAD> grad;
    Maps<XENT_SUMS> sums;
    a.box = x_box(tokens);
    if (!map_k(&grad.m[0], xp, dim, packed ? p.rows : tokens, packed ? dim : ldx, a.box) || !map_k(&grad.m[1], w, dim, vocab, ldw) ||
        !map_out(&grad.m[2], g, false, p.piece, p.rows, p.piece) || !map_k(&sums.m[0], g, p.piece, p.rows, p.piece) ||
        !map_mn(&sums.m[1], w, dim, vocab, ldw) || !map_out(&sums.m[2], acc, true, dim, p.splits * p.rows, dim) ||
        !map_mn(&sums.m[3], g, p.piece, p.rows, p.piece) || !map_mn(&sums.m[4], pk.xn, dim, p.rows, dim) ||
        !map_out(&sums.m[5], dw, a.dw_f32, dim, vocab, lddw))
        return FP8_ERR_CUDA;
    // blocks of K in a unit of SUMS: tokens for dw, a part of the piece for dx
    const int64_t longest = std::max((tokens + kBK - 1) / kBK, (p.piece / kBK + p.splits - 1) / p.splits);
    for (int64_t v = 0; v < vocab; v += p.piece) {
        a.v0 = (int)v;
        a.vn = (int)std::min<int64_t>(p.piece, vocab - v);
        a.band = 16;
        rc = !single(tokens, vocab) ? run<XENT_GRAD, true, 256>(grad, a, st)
             : p.bn == 256   ? run<XENT_GRAD, false, 256>(grad, a, st)
                             : run<XENT_GRAD, false, 128>(grad, a, st);
        if (rc != FP8_OK) return rc;
        a.xn = nullptr;
        a.band = 8;
        a.dx_add = v > 0;
        rc = longest > kChunk ? run<XENT_SUMS, true, 256, true>(sums, a, st) : run<XENT_SUMS, true, 256, false>(sums, a, st);
        if (rc != FP8_OK) return rc;
    }
    // many parts means few columns: eight threads each (61 x 20674 x 192: 6 us, by one 13)
    auto join = [&](auto kernel, int lanes) {
        const int64_t blocks = std::min<int64_t>((tokens * (dim / 8) * lanes + kSumThreads - 1) / kSumThreads, (int64_t)sm_count() * 16);
        return launch_dependent(kernel, dim3((unsigned)blocks), kSumThreads, 0, st, static_cast<const float *>(acc), p.splits, p.rows, a.count, pk.map,
                                pk.norm, a.dim, static_cast<uint16_t *>(dx), lddx, a.tokens, status);
    };
    return p.splits >= 8 ? join(k_xent_dx_join<8>, 8) : join(k_xent_dx_join<1>, 1);
}

}  // namespace fp8fg
