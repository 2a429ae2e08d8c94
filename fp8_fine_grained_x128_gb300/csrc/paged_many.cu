// paged_many.cu -- attention over a paged cache when more than 16 rows (new
// tokens x query heads of a group) share a cache head: prompts, chunks and
// longer drafts (sm_103a).
//
// Bound: the tensor cores, in long series the rate that the power limit leaves
// them (32 query and 8 cache heads of 128: an 8192-token prompt 394 us, 1400
// TFLOP/s, 379 us in short bursts; 2048 tokens after 30720 E4M3 keys 679 and 648 us,
// 1570 and 1640).  With head_dim 64 an exponential stands for half the
// products, and the softmax chain sets the pace (about 1000 TFLOP/s).  A unit is 256 rows of one (sequence, cache head):
// two 128-row halves that share every 128-key tile of K and V.  S = Q K^T is a
// tcgen05.mma of 128 x 128 per half into tensor memory; the half's four
// softmax warps (one row a thread, no exchange between threads) read it, write
// P over it as 16-bit words, and O += P V takes P from tensor memory and
// accumulates there.  While one half's softmax runs, the other half's two
// products do.  Tensor memory: S0 S1 (128 columns each) O0 O1 (head_dim
// each).  The 512 columns and the shared memory allow one CTA per SM.
//
// All units' tiles stand in one line, cut into equal runs, one per CTA (as in
// paged_few.cu); a unit broken by a cut leaves its parts in the workspace,
// and k_attn_join adds them up in order.
//
// Warps: 0-3 and 4-7 the softmax of the two halves, 8 TMA, 9 MMA, 10 walks the
// run and hands its segments to the others ahead of time, 11 sees that a tile's
// operands have landed; with an FP8 cache 12-15 turn the code tiles into FP16
// operand tiles (exactly), and Q is scaled per row
// by a power of two to fit FP16, P by 2^6.
//
// With up to 128 rows one half is empty.  Giving its warps every second tile of
// the same rows (both chains joined at the unit's end) was built and measured: 110
// against 113 us for 32 sequences x 20 rows over 4000 BF16 keys, 129 against 118 for
// 64 rows over E4M3 keys.  The copies and conversions set the pace there, so it was left out.
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "paged.cuh"
#include "tmap.h"

namespace fp8fg {

constexpr int kUnitRows = 256;
constexpr int kTile = 128;            // keys of a tile
constexpr int kLoadWarp = 8, kMmaWarp = 9, kWalkWarp = 10, kGateWarp = 11, kConvWarp0 = 12;
constexpr int kUnitCost = 4;          // a unit's own time (Q, first scores, output) in tiles' times
constexpr int kSegs = 4;              // segments handed over ahead
constexpr int kSub = 128 * 128;       // bytes of 128 rows x 64 16-bit elements, 128-byte swizzle

template <int D, int FMT>
struct Many {
    static constexpr bool kFp8 = FMT != FP8_KV_BF16;
    static constexpr int kThreads = kFp8 ? 512 : 384;
    static constexpr int kTileB = (D / 64) * kSub;         // an operand tile
    static constexpr int kStages = D == 64 ? 6 : kFp8 ? 4 : 5;
    static_assert(kStages >= 3, "a segment's first tile holds two tiles of keys and one of values");
    static constexpr int kRawB = kFp8 ? kTile * D : 0;     // a tile of codes
    static constexpr int kRawStages = kFp8 ? (D == 64 ? 4 : 2) : 1;   // (BF16: an unused pair of barriers)
    static constexpr int kQ = 0;
    static constexpr int kKV = kQ + 2 * kTileB;
    static constexpr int kRaw = kKV + kStages * kTileB;
    static constexpr int kBar = kRaw + kRawStages * kRawB;
    static constexpr int kBars = 2 * kStages + 2 * kRawStages + 10 + 2 * kSegs + 1;
    static constexpr int kBytes = 1024 + kBar + kBars * 8;
    static constexpr float kOff = kFp8 ? 6.0f : 0.0f;      // P is kept as 2^kOff p
    // register split of the warpgroups (the launch has 128 a thread with an FP8 cache, 168 with a BF16 one)
    static constexpr int kSoftRegs = kFp8 ? 176 : 216, kMmaRegs = 72, kConvRegs = kFp8 ? 88 : 0;
    static constexpr int kLaunchRegs = 128 * (2 * kSoftRegs + kMmaRegs + kConvRegs);
    static_assert(kLaunchRegs <= kThreads * (kFp8 ? 128 : 168), "register split above what the block is launched with");
};

// A unit broken by the cut between two CTAs' runs, as its first CTA leaves it.
struct ManyJoin {
    int32_t rows;     // 0: this CTA starts no broken unit
    int32_t last;     // the last CTA with a part
    int32_t row0;     // first row of the unit in its sequence
    int32_t head;     // cache head
    int64_t first;    // first token of the sequence
};

constexpr int kPartFloats = kUnitRows * 128 + 3 * kUnitRows;   // o [D / 4][256] x 4, m [256], l [256], lp [256]

// The two products' instructions.  The descriptors' high words are constants
// and their low words (start address >> 4, leading offset) are put together
// here, so that no 64-bit descriptors stay live between instructions.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);   // stride 1024, version 1, 128-byte swizzle
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }

// D(tmem) (+)= A(smem) x B(smem)^T, 16-bit operands, FP32 accumulator.
__device__ __forceinline__ void tc_mma_16_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                             uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
        : "memory");
}
// D(tmem) (+)= A(tmem) x B(smem)
__device__ __forceinline__ void tc_mma_16_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc,
                                             uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
        : "memory");
}

// 32 lanes x 32 columns, registers -> tensor memory (thread i: lane base + i).
__device__ __forceinline__ void tc_st_32x32b_x32(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tc_st_32x32b_x16(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// 4-D tiled bulk tensor load (columns, row in page, head, page).
__device__ __forceinline__ void tma_load_4d(uint32_t smem_dst, const CUtensorMap *map, uint64_t *bar, int x, int y,
                                            int z, int w)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// Instruction descriptor of tcgen05.mma kind::f16: FP32 accumulator, both
// operands BF16 or both FP16, A K-major, B K-major or MN-major (bit 16).
__host__ __device__ constexpr uint32_t idesc_16(bool bf16, bool b_mn, int M, int N)
{
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// A segment: the tiles [tile0, tile1) of one unit; tile1 = 0 ends the run.
struct Segment {
    int32_t tile0, tile1;
    int32_t whole;         // all of the unit's tiles
    int32_t seq, first, len, pos0;
    int32_t head, row0, rows;   // first row of the unit in its sequence, its rows (<= 256)
};

// Whether the unit's first row sees fewer than kFineKeys keys.
__device__ __forceinline__ bool fine_unit(const Segment &q, int group) { return q.pos0 + q.row0 / group < kFineKeys; }

// The walk of one warp over its CTA's run of the line.  The line: sequence by
// sequence, in each head by head, in each unit by unit, in each kUnitCost
// places for the unit and one for every tile, so that equal runs take equal
// times.  Every member is the same in all lanes.
struct Walk {
    int64_t s, s_end;        // the run still to do
    int64_t unit0;           // the line's place where the current unit begins
    int64_t seq_end;         // and of the sequence's end
    int b, first, rows, len, pos0;   // pos0: position of the sequence's first new token
    int head, unit, nt;      // nt: tiles of the unit

    __device__ __forceinline__ int tiles_of(const AttnArgs &g, int u) const
    {
        const int last = (min(rows, (u + 1) * kUnitRows) - 1) / g.group;
        return max(1, (max(0, pos0 + last + 1) + kTile - 1) / kTile);
    }
    __device__ __forceinline__ int cost_of(const AttnArgs &g, int u) const { return kUnitCost + tiles_of(g, u); }
    __device__ __forceinline__ int units() const { return (rows + kUnitRows - 1) / kUnitRows; }

    // the sequence's places of one head (a sum over its units, lanes side by side)
    __device__ __forceinline__ int64_t load(const AttnArgs &g, int seq)
    {
        b = seq;
        rows = 0;
        if (b < g.b.seqs && !seq_lengths(g, b, first, rows, len)) set_status(g.status, FP8_ERR_INVALID_ARG);
        if (rows <= kFewRows) return 0;
        pos0 = len - rows / g.group;
        int64_t n = 0;
        for (int u = threadIdx.x & 31; u < units(); u += 32) n += cost_of(g, u);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        return n;
    }
    // the sequence that holds place s: the first at or after `seq` whose end lies past it
    __device__ __forceinline__ void seek(const AttnArgs &g, int seq, int64_t before)
    {
        int64_t per_head = load(g, seq);
        while (before + per_head * g.c.heads <= s) {
            before += per_head * g.c.heads;
            if (++seq >= g.b.seqs) {   // only if the lengths changed meanwhile
                s = s_end;
                return;
            }
            per_head = load(g, seq);
        }
        seq_end = before + per_head * g.c.heads;
        head = (int)((s - before) / per_head);
        unit0 = before + head * per_head;
        for (unit = 0;;) {   // 32 units a step
            const int u = unit + (int)(threadIdx.x & 31);
            const int n = u < units() ? cost_of(g, u) : 0;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if ((int)(threadIdx.x & 31) >= o) incl += v;
            }
            const unsigned past = __ballot_sync(0xffffffffu, unit0 + incl > s);
            if (past || unit + 32 >= units()) {
                const int at = past ? __ffs(past) - 1 : 0;
                unit += at;
                unit0 += __shfl_sync(0xffffffffu, incl - n, at);
                break;
            }
            unit += 32;
            unit0 += __shfl_sync(0xffffffffu, incl, 31);
        }
        nt = tiles_of(g, unit);
    }
    __device__ __forceinline__ bool valid() const { return s < s_end; }
    __device__ __forceinline__ Segment segment() const
    {
        Segment q;
        q.tile0 = (int)max((int64_t)0, s - unit0 - kUnitCost);
        q.tile1 = (int)min((int64_t)nt, s_end - unit0 - kUnitCost);   // <= tile0: none of its tiles in this run
        q.whole = q.tile0 == 0 && q.tile1 == nt;
        q.seq = b;
        q.first = first;
        q.len = len;
        q.pos0 = pos0;
        q.head = head;
        q.row0 = unit * kUnitRows;
        q.rows = min(kUnitRows, rows - q.row0);
        return q;
    }
    __device__ __forceinline__ void next(const AttnArgs &g)
    {
        unit0 += kUnitCost + nt;
        s = unit0;
        if (s >= s_end) return;
        if (s >= seq_end) {
            seek(g, b + 1, seq_end);
            return;
        }
        if (++unit == units()) {
            unit = 0;
            ++head;
        }
        nt = tiles_of(g, unit);
    }
};

template <int D, int FMT>
__global__ void __launch_bounds__(Many<D, FMT>::kThreads, 1)
    k_attn_many(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, AttnArgs g, int box_rows)
{
    using C = Many<D, FMT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBar);   // operand tiles
    uint64_t *empty = full + C::kStages;
    uint64_t *raw_full = empty + C::kStages;                         // code tiles
    uint64_t *raw_empty = raw_full + C::kRawStages;
    uint64_t *q_full = raw_empty + C::kRawStages;                    // per half
    uint64_t *s_full = q_full + 2;
    uint64_t *p_ready = s_full + 2;   // per half and 64 keys
    uint64_t *o_full = p_ready + 4;
    uint64_t *seg_full = o_full + 2;
    uint64_t *seg_empty = seg_full + kSegs;
    uint64_t *mma_done = seg_empty + kSegs;
    __shared__ Segment segs[kSegs];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    __shared__ int64_t s_total[C::kThreads / 32];
    volatile int *abort_flag = &abort_word;

    // (the shuffle tells the compiler that the role, and what follows from it, is the same in a whole warp)
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    constexpr int kWarps = C::kThreads / 32;

    dependents_launch();
    dependency_wait();
    // the line's length
    int64_t total = 0;
    for (int b = warp; b < g.b.seqs; b += kWarps) {
        Walk w;
        total += w.load(g, b) * g.c.heads;
    }
    if (lane == 0) s_total[warp] = total;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&full[i], C::kFp8 ? 4 : 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < C::kRawStages; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], 4);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&q_full[x], 4);
            mbar_init(&s_full[x], 1);
            mbar_init(&p_ready[2 * x], 4 + 1);   // and the gate
            mbar_init(&p_ready[2 * x + 1], 4);
            mbar_init(&o_full[x], 1);
        }
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(&seg_full[i], 1);
            mbar_init(&seg_empty[i], 8 + 3 + (C::kFp8 ? 4 : 0));   // the warps that read it
        }
        mbar_init(mma_done, 1);
        abort_word = 0;
        fence_barrier_init();
    }
    __syncthreads();
    total = 0;
    for (int i = 0; i < kWarps; ++i) total += s_total[i];
    ManyJoin *joins = static_cast<ManyJoin *>(g.many_joins);
    const int64_t ctas = min((int64_t)gridDim.x, total);
    if (blockIdx.x >= ctas) {
        if (threadIdx.x == 0) joins[blockIdx.x].rows = 0;
        return;
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // (uniform in the compiler's eyes, like everything the MMA warp's operands come from: operands that are
    // not took the issue 64 cycles an MMA instead of 33, and the kernel a tenth to a quarter longer)
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);

    // the n-th segment of the run, by a whole warp; false: the end, or an abort
    auto next_segment = [&](uint32_t n, Segment &q) {
        if (!warp_wait(&seg_full[n % kSegs], (n / kSegs) & 1, abort_flag, g.status)) return false;
        q = segs[n % kSegs];
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[n % kSegs]);
        return q.tile1 != 0;
    };

    if (warp < 8) {
        // -------------------------------------------------- softmax of half x
        regs_inc<C::kSoftRegs>();
        const int x = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tS = lanes + x * 128, tO = lanes + 256 + x * D;
        const float ks = g.c.k_scale ? *g.c.k_scale : 1.0f, vs = g.c.v_scale ? *g.c.v_scale : 1.0f;
        uint32_t it = 0, un = 0;
        bool ok = true;
        uint32_t nseg = 0;
        auto next_active = [&](Segment &q) {   // the next segment with rows of this half
            while (next_segment(nseg++, q))
                if (x * 128 < q.rows) return true;
            return false;
        };
        auto row_of = [&](const Segment &q) { return q.row0 + min(x * 128 + r, q.rows - 1); };
        auto q_row = [&](const Segment &q) {   // its token and query head
            const int row = row_of(q);
            return make_int2(q.first + row / g.group, q.head * g.group + row % g.group);
        };
        // The warp's 32 rows of Q into the swizzled operand tile, D / 8 lanes side by side on a row (a row
        // a lane met 32 lines an instruction: 3000 cycles); returns the factor from the lane's row's
        // products to log2 scores, which is positive, so that the largest product has the largest score: with
        // an FP8 cache Q takes the key scale's sign (or its NaN).
        auto load_q = [&](const Segment &q) {
            constexpr int kLanes = D / 8, kRows = 32 / kLanes;   // lanes of a row, rows an instruction
            const int2 at = q_row(q);
            const int64_t off = (int64_t)at.x * g.q_ld + (int64_t)at.y * D;
            float mul = fmaxf(g.scale * kLog2e * fabsf(ks), 1.17549435e-38f);
            uint4 v[D / 8];
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const int64_t o = __shfl_sync(0xffffffffu, off, i * kRows + lane / kLanes);
                v[i] = *reinterpret_cast<const uint4 *>(g.q + o + 8 * (lane % kLanes));
            }
            if (C::kFp8) {   // a power of two that brings each row's largest value into [2^14, 2^15)
                int mine = 0;
                const float sign = ks < 0.0f ? -1.0f : ks >= 0.0f ? 1.0f : ks;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    uint32_t m = absmax8(v[i]);
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                    const int e = min(max((int)(m >> 7), 15), 254) - 127;
                    const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23) * sign;
                    uint32_t h[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) h[k] = f16x2_rn(bf16_lo(h[k]) * up, bf16_hi(h[k]) * up);
                    v[i] = make_uint4(h[0], h[1], h[2], h[3]);
                    const int of_row = __shfl_sync(0xffffffffu, e, (lane % kRows) * kLanes);   // row i * kRows + lane % kRows
                    if (lane / kRows == i) mine = of_row;
                }
                mul = fmaxf(mul * __uint_as_float((uint32_t)(127 - 14 + mine) << 23), 1.17549435e-38f);
            }
            const int c = lane % kLanes;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const int row = (warp & 3) * 32 + i * kRows + lane / kLanes;
                *reinterpret_cast<uint4 *>(smem + C::kQ + x * C::kTileB + (c / 8) * kSub + row * 128 +
                                           (((c & 7) ^ (row & 7)) << 4)) = v[i];
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[x]);
            return mul;
        };
        Segment q;
        bool have = next_active(q);
        float mul = have ? load_q(q) : 0.0f;
        while (have) {
            const int tile0 = q.tile0, tile1 = q.tile1;
            const int pos = q.pos0 + row_of(q) / g.group;
            const bool fine = !C::kFp8 && fine_unit(q, g.group);
            const int pos_min = __shfl_sync(0xffffffffu, pos, 0);   // rows' positions do not decrease
            const float lazy = !C::kFp8 && pos_min < kExactKeys ? 0.0f : kLazy;
            // l: the sum of the exponentials, for the LSE.  lp: of P as it goes into the product, for the output:
            // with one BF16 term the largest of every 32 keys counts as it was rounded, so that a key that
            // carries a row's weight brings the same factor above and below the line.  (All keys as they were
            // rounded: 430 instead of 391 us for an 8192-token prompt.)
            float m = -INFINITY, l = 0.0f, lp = 0.0f;
            // (one loop with a branch on the number of P's terms inside was 15% slower)
            auto tiles = [&](auto two_terms) {
            constexpr bool FINE = decltype(two_terms)::value, ONE = !C::kFp8 && !FINE;   // ONE: one BF16 term
            for (int j = tile0; j < tile1; ++j, ++it) {
                if (!warp_wait(&s_full[x], it & 1, abort_flag, g.status)) { ok = false; break; }
                tc_fence_after();
                uint32_t s[4][32];
                uint64_t sum[2];
                float up = 1.0f;
                const bool masked = j * kTile + kTile - 1 > pos_min;   // keys past the row's position
                auto load = [&] {
#pragma unroll
                    for (int c = 0; c < 4; ++c) tc_ld_32x32b_x32(tS + 32 * c, s[c]);
                    tc_wait_ld();
                    if (masked) {
                        const int lim = pos - j * kTile;
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (32 * c + i > lim) s[c][i] = 0xFF800000u;   // -inf
                    }
                };
                float mx[4];   // of 32 keys each
                auto row_max = [&] {
                    mx[0] = mx[1] = mx[2] = mx[3] = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            mx[c] = max3(mx[c], __uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1]));
                    return max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
                };
                // P of 64 keys with the maximum m in use, packed into s[hf]
                auto exps = [&](int hf) {
                    const float base = m == -INFINITY ? 0.0f : C::kOff - m * mul;
                    const uint64_t mul2 = f2_pack(mul, mul), base2 = f2_pack(base, base);
#pragma unroll
                    for (int c = 2 * hf; c < 2 * hf + 2; ++c) {
                        uint32_t lo[16];
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float a, b;
                            f2_unpack(f2_fma_bits(s[c][i], s[c][i + 1], mul2, base2), a, b);
                            a = ex2_approx_ftz(a);
                            b = ex2_approx_ftz(b);
                            sum[(i >> 1) & 1] = f2_fma(f2_pack(a, b), f2_pack(1.0f, 1.0f), sum[(i >> 1) & 1]);
                            const uint32_t hi = C::kFp8 ? f16x2_rn(a, b) : bf16x2_rn(a, b);
                            if (FINE) lo[i / 2] = bf16x2_rn(a - bf16_lo(hi), b - bf16_hi(hi));
                            s[hf][(c & 1) * 16 + i / 2] = hi;
                        }
                        // the second term of P, in the upper half of S's columns
                        if (FINE) tc_st_32x32b_x16(tS + 64 + 16 * c, lo);
                    }
                };
                auto store = [&](int hf) {
                    tc_st_32x32b_x32(tS + 32 * hf, s[hf]);
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_ready[2 * x + hf]);
                };
                load();
                const float mt = row_max();
                // (with a BF16 cache no further than the weight so far: a key above that has p = 1)
                const float lag = C::kFp8 ? kLazy : fminf(lazy, __log2f(l));
                const bool grow = mt > m && (m == -INFINITY || (mt - m) * mul > lag);
                if (__any_sync(0xffffffffu, grow)) {
                    if (grow) {
                        up = ex2_approx_ftz((m - mt) * mul);
                        m = mt;
                    }
                    // the products so far are complete (S of this tile was issued after them): rescale them
                    if (j > tile0) {
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            tc_ld_32x32b_x16(tO + 16 * c, o);
                            tc_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * up);
                            tc_st_32x32b_x16(tO + 16 * c, o);
                        }
                    }
                }
                sum[0] = sum[1] = 0;
                exps(0);
                store(0);
                exps(1);
                store(1);
                float a, b, c, d;
                f2_unpack(sum[0], a, b);
                f2_unpack(sum[1], c, d);
                const float here = (a + b) + (c + d);
                l = l * up + here;
                if (ONE) {
                    const float base = m == -INFINITY ? 0.0f : C::kOff - m * mul;
                    float fix = 0.0f;
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        const float p0 = ex2_approx_ftz(fmaf(mx[i], mul, base)), p1 = ex2_approx_ftz(fmaf(mx[i + 1], mul, base));
                        const uint32_t w = bf16x2_rn(p0, p1);
                        fix += (bf16_lo(w) - p0) + (bf16_hi(w) - p1);
                    }
                    lp = lp * up + (here + fix);
                }
            }
            if (!ONE) lp = l;
            };
            if (fine)
                tiles(std::integral_constant<bool, !C::kFp8>());
            else
                tiles(std::false_type());
            if (!ok) break;
            // every product with this Q is complete (the last S was): the next one replaces it, and its
            // first scores are under way while this segment ends
            Segment next;
            const bool more = next_active(next);
            const float next_mul = more ? load_q(next) : 0.0f;
            if (!warp_wait(&o_full[x], un & 1, abort_flag, g.status)) break;
            ++un;
            tc_fence_after();
            const float inv = lp == 0.0f ? 0.0f : vs / lp;   // (a NaN stays one)
            const int lrow = x * 128 + r;
            const bool mine = lrow < q.rows;
            if (q.whole) {
                const int2 th = q_row(q);
                const int64_t off = mine ? (int64_t)th.x * g.out_ld + (int64_t)th.y * D : -1;
                // 16 rows x 64 columns a load: a lane holds columns 8j + 2 (lane % 4) + {0, 1} of rows lane / 4
                // and 8 more; four lanes turn their 4 x 4 words so that each stores 16 bytes of one row
                const int t4 = lane & 3;
#pragma unroll
                for (int lh = 0; lh < 2; ++lh) {
                    int64_t o2[2];
                    float inv2[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int from = 16 * lh + 8 * u + (lane >> 2);
                        o2[u] = __shfl_sync(0xffffffffu, off, from);
                        inv2[u] = __shfl_sync(0xffffffffu, inv, from);
                    }
#pragma unroll
                    for (int h = 0; h < D / 64; ++h) {
                        uint32_t o[32];
                        tc_ld_16x256b_x8(tO + ((uint32_t)(16 * lh) << 16) + 64 * h, o);
                        tc_wait_ld();
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                uint32_t w[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    w[k] = bf16x2_rn(__uint_as_float(o[4 * (4 * e + k) + 2 * u]) * inv2[u],
                                                     __uint_as_float(o[4 * (4 * e + k) + 2 * u + 1]) * inv2[u]);
#pragma unroll
                                for (int k = 0; k < 4; k += 2) {
                                    const uint32_t got = __shfl_xor_sync(0xffffffffu, (t4 & 1) ? w[k] : w[k + 1], 1);
                                    w[k] = (t4 & 1) ? got : w[k];
                                    w[k + 1] = (t4 & 1) ? w[k + 1] : got;
                                }
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const uint32_t got = __shfl_xor_sync(0xffffffffu, (t4 & 2) ? w[k] : w[k + 2], 2);
                                    w[k] = (t4 & 2) ? got : w[k];
                                    w[k + 2] = (t4 & 2) ? w[k + 2] : got;
                                }
                                const int64_t at = o2[u] + 64 * h + 32 * e + 8 * t4;
                                if (o2[u] >= 0 && dbg_span(at, 8, (g.tokens - 1) * g.out_ld + (int64_t)g.q_heads * D, g.status))
                                    *reinterpret_cast<uint4 *>(g.out + at) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                    }
                }
                if (mine && g.lse && dbg_lse(g, (int64_t)th.x * g.q_heads + th.y))
                    g.lse[(int64_t)th.x * g.q_heads + th.y] = l == 0.0f ? -INFINITY : (m * mul - C::kOff + log2f(l)) * kLn2;
            } else {
                float *part = g.many_parts + (int64_t)(2 * blockIdx.x + (tile0 == 0 ? 1 : 0)) * kPartFloats;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tc_ld_32x32b_x32(tO + 32 * c, o);
                    tc_wait_ld();
                    if (!mine) continue;
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        reinterpret_cast<uint4 *>(part)[(8 * c + i / 4) * kUnitRows + lrow] =
                            make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                }
                if (mine) {
                    part[kUnitRows * 128 + lrow] = m == -INFINITY ? -INFINITY : m * mul;
                    part[kUnitRows * 128 + kUnitRows + lrow] = l;
                    part[kUnitRows * 128 + 2 * kUnitRows + lrow] = lp;
                }
            }
            q = next;
            mul = next_mul;
            have = more;
        }
    } else if (warp < kConvWarp0) {
        regs_dec<C::kMmaRegs>();
        if (warp == kLoadWarp) {
            // ---------------------------------------------- TMA producer
            uint64_t *rfull = C::kFp8 ? raw_full : full, *rempty = C::kFp8 ? raw_empty : empty;
            constexpr int kRing = C::kFp8 ? C::kRawStages : C::kStages;
            const uint32_t ring = smem_u32(smem + (C::kFp8 ? C::kRaw : C::kKV));
            constexpr int kSlotB = C::kFp8 ? C::kRawB : C::kTileB;
            uint32_t it = 0;
            bool ok = true;
            Segment q;
            for (uint32_t n = 0; ok && next_segment(n, q); ++n) {
                const int32_t *table = g.b.page_table + q.seq * g.b.page_table_ld;
                const int tile0 = q.tile0, tile1 = q.tile1;
                // lane i loads the tile's i-th box of rows: its page, one tile ahead
                auto page_of = [&](int j) {
                    const int key = j * kTile + lane * box_rows;
                    if (j >= tile1 || lane * box_rows >= kTile || key >= q.len) return -1;
                    const int page = table[key / g.c.page_size];
                    if (page < 0 || page >= g.c.num_pages) set_status(g.status, FP8_ERR_INVALID_ARG);
                    return page;
                };
                int page = page_of(tile0);
                for (int j = tile0; j < tile1 && ok; ++j) {
                    const int next_page = page_of(j + 1);
                    const int keys = min(kTile, max(0, q.len - j * kTile));
                    const int boxes = (keys + box_rows - 1) / box_rows;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const int slot = it % kRing;
                        if (!warp_wait(&rempty[slot], ((it / kRing) & 1) ^ 1, abort_flag, g.status)) { ok = false; break; }
                        ++it;
                        if (lane == 0)   // a page out of range reads as zeros and still counts its bytes
                            mbar_arrive_expect_tx(&rfull[slot], boxes * box_rows * D * (C::kFp8 ? 1 : 2));
                        __syncwarp();
                        if (lane < boxes) {
                            const int rip = (j * kTile + lane * box_rows) & (g.c.page_size - 1);
                            const uint32_t dst = ring + slot * kSlotB;
                            const CUtensorMap *map = kv ? &tmV : &tmK;
                            if (C::kFp8) {
                                tma_load_4d(dst + lane * box_rows * D, map, &rfull[slot], 0, rip, q.head, page);
                            } else {
#pragma unroll
                                for (int sub = 0; sub < D / 64; ++sub)
                                    tma_load_4d(dst + sub * kSub + lane * box_rows * 128, map, &rfull[slot], 64 * sub, rip,
                                                q.head, page);
                            }
                        }
                    }
                    page = next_page;
                }
            }
            // no copy is in flight when the CTA ends
            const uint32_t from = it > (uint32_t)kRing ? it - kRing : 0;
            for (uint32_t i = from; i < it; ++i) mbar_wait_bounded(&rfull[i % kRing], (i / kRing) & 1, nullptr);
            __syncwarp();
        } else if (warp == kMmaWarp) {
            // ---------------------------------------------- MMA issuer
            // The whole warp walks along and one elected lane issues: the operands stay in
            // uniform registers.  (One lane alone in a branch took about 70 cycles to issue
            // an MMA of 64, so that no MMA was queued while it waited on a barrier.)
            constexpr uint32_t id_qk = idesc_16(!C::kFp8, false, 128, kTile);
            constexpr uint32_t id_pv = idesc_16(!C::kFp8, true, 128, D);
            const uint32_t sq = smem_u32(smem + C::kQ), skv = smem_u32(smem + C::kKV);
            uint32_t it = 0;             // tiles of the ring
            uint32_t done[2] = {0, 0};   // P tiles of each half
            uint32_t un[2] = {0, 0};     // units of each half
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                ok = ok && warp_wait(bar, parity, abort_flag, g.status);
                return ok;
            };
            auto wait_tile = [&](uint32_t i) { return wait(&full[i % C::kStages], (i / C::kStages) & 1); };
            auto qk = [&](int x, int slot) {
                const uint32_t qa = desc_lo(sq + x * C::kTileB, 16), kb = desc_lo(skv + slot * C::kTileB, 16);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = ((k / 4) * kSub + (k % 4) * 32) >> 4;
                        tc_mma_16_ss(tmem + x * 128, qa + off, kb + off, id_qk, k > 0);
                    }
                    tc_commit(&s_full[x]);
                }
                __syncwarp();
            };
            Segment q;
            for (uint32_t n = 0; ok; ++n) {
                if (!wait(&seg_full[n % kSegs], (n / kSegs) & 1)) break;
                q = segs[n % kSegs];
                __syncwarp();
                if (lane == 0) mbar_arrive(&seg_empty[n % kSegs]);
                if (q.tile1 == 0) break;
                const int tile0 = q.tile0, tile1 = q.tile1, halves = q.rows > 128 ? 2 : 1;
                const int terms = !C::kFp8 && fine_unit(q, g.group) ? 2 : 1;   // of P
                if (!wait_tile(it)) break;
                for (int x = 0; x < halves && ok; ++x) {
                    if (!wait(&q_full[x], un[x] & 1)) break;
                    ++un[x];
                    qk(x, it % C::kStages);
                }
                if (!ok) break;
                const int first_slot = it % C::kStages;
                ++it;
                for (int j = tile0; j < tile1; ++j) {
                    const int vslot = it % C::kStages, kslot = (it + 1) % C::kStages;
                    const bool more = j + 1 < tile1;
                    for (int x = 0; x < halves; ++x) {
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            if (!wait(&p_ready[2 * x + hf], done[x] & 1)) break;
                            tc_fence_after();
                            const uint32_t vb = desc_lo(skv + vslot * C::kTileB, kSub);
                            if (elect_one()) {
                                for (int e = 0; e < terms; ++e)
#pragma unroll
                                    for (int k = hf * kTile / 32; k < (hf + 1) * kTile / 32; ++k)
                                        tc_mma_16_ts(tmem + 256 + x * D, tmem + x * 128 + 64 * e + 8 * k, vb + k * 128,
                                                     id_pv, j > tile0 || k > 0 || e > 0);
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                        ++done[x];
                        if (more)
                            qk(x, kslot);
                        else if (elect_one())
                            tc_commit(&o_full[x]);
                    }
                    if (!ok) break;
                    if (elect_one()) {
                        if (j == tile0) tc_commit(&empty[first_slot]);   // (the gate has seen it: p_ready above)
                        tc_commit(&empty[vslot]);
                        if (more) tc_commit(&empty[kslot]);
                    }
                    __syncwarp();
                    it += more ? 2 : 1;
                }
            }
            if (elect_one()) {
                tc_commit(mma_done);
                mbar_wait_bounded(mma_done, 0, nullptr);
            }
            __syncwarp();
        } else if (warp == kGateWarp) {
            // ---------------------------------------------- gate: the operands of P V and the next Q K^T
            // Arrives on a tile's first p_ready once its values and the next tile's keys have landed,
            // so that the MMA warp has one barrier to wait on (each wait costs it about 100 cycles).
            // Value rows past the sequence's end may hold anything, and 0 x NaN is NaN: they are
            // zeroed here (the FP8 form's are when the codes are converted).
            // It sees every place of the ring in turn before the MMA warp can hand it back (which it does for all
            // of a tile's operands, and for the segment's first keys, after the gate's arrival for that tile):
            // were a slot filled again before the gate looked, the parity would be what it was, and the gate
            // would wait for ever.
            uint32_t it = 0, done[2] = {0, 0};
            bool ok = true;
            auto tile = [&](uint32_t i) { return warp_wait(&full[i % C::kStages], (i / C::kStages) & 1, abort_flag, g.status); };
            Segment q;
            for (uint32_t n = 0; ok && next_segment(n, q); ++n) {
                const int halves = q.rows > 128 ? 2 : 1;
                if (!(ok = tile(it))) break;   // the segment's first keys (the MMA warp waits for those itself)
                ++it;
                for (int j = q.tile0; j < q.tile1; ++j) {
                    const bool more = j + 1 < q.tile1;
                    if (!(ok = tile(it))) break;
                    if (!C::kFp8 && (j + 1) * kTile > q.len) {
                        uint8_t *v = smem + C::kKV + (it % C::kStages) * C::kTileB;
                        for (int c = max(0, q.len - j * kTile) * 8 + lane; c < kTile * 8; c += 32)
#pragma unroll
                            for (int sub = 0; sub < D / 64; ++sub)
                                *reinterpret_cast<uint4 *>(v + sub * kSub + c * 16) = make_uint4(0, 0, 0, 0);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (more && !(ok = tile(it + 1))) break;
                    it += more ? 2 : 1;
                    for (int x = 0; x < halves; ++x) {   // the last tile's phase first: one arrival each
                        if (done[x] > 0 && !(ok = warp_wait(&p_ready[2 * x], (done[x] - 1) & 1, abort_flag, g.status))) break;
                        ++done[x];
                        if (lane == 0) mbar_arrive(&p_ready[2 * x]);
                    }
                    if (!ok) break;
                }
            }
        } else if (warp == kWalkWarp) {
            // ---------------------------------------------- the run, segment by segment
            Walk w;
            w.s = blockIdx.x * total / ctas;
            w.s_end = (blockIdx.x + 1) * total / ctas;
            w.seek(g, 0, 0);
            ManyJoin j{};
            for (uint32_t n = 0;; ++n) {
                if (!warp_wait(&seg_empty[n % kSegs], ((n / kSegs) & 1) ^ 1, abort_flag, g.status)) break;
                Segment q{};
                while (w.valid()) {
                    q = w.segment();
                    if (q.tile1 > q.tile0) break;
                    w.next(g);
                }
                const bool more = w.valid();
                if (!more) q.tile1 = 0;
                if (lane == 0) {
                    segs[n % kSegs] = q;
                    mbar_arrive(&seg_full[n % kSegs]);
                }
                if (!more) break;
                if (!q.whole && q.tile0 == 0) {
                    j.rows = q.rows;
                    j.last = (int)(min(((w.unit0 + kUnitCost + w.nt) * ctas + total - 1) / total, ctas) - 1);
                    j.row0 = q.row0;
                    j.head = q.head;
                    j.first = q.first;
                }
                w.next(g);
            }
            if (lane == 0) joins[blockIdx.x] = j;
        }
    } else if (C::kFp8) {
        // -------------------------------------------------- codes to FP16 tiles
        regs_dec<C::kFp8 ? C::kConvRegs : 88>();
        constexpr int kChunks = D / 16;                // 16 codes each
        const int t = threadIdx.x & 127;
        const int c = t % kChunks, r0 = t / kChunks;   // a thread's chunk and its rows r0 + i * (128 / kChunks)
        uint32_t it = 0;
        bool ok = true;
        Segment q;
        for (uint32_t n = 0; ok && next_segment(n, q); ++n) {
            const int tile0 = q.tile0, tile1 = q.tile1;
            for (int j2 = 2 * tile0; j2 < 2 * tile1; ++j2, ++it) {
                const int keys = min(kTile, max(0, q.len - (j2 >> 1) * kTile));
                const int raw = it % C::kRawStages, slot = it % C::kStages;
                if (!warp_wait(&raw_full[raw], (it / C::kRawStages) & 1, abort_flag, g.status) ||
                    !warp_wait(&empty[slot], ((it / C::kStages) & 1) ^ 1, abort_flag, g.status)) {
                    ok = false;
                    break;
                }
                const uint32_t src = smem_u32(smem + C::kRaw + raw * C::kRawB) + t * 16;
                uint8_t *dst = smem + C::kKV + slot * C::kTileB + (c / 4) * kSub;
                // Four chunks at a time: their loads overlap, and the bursts beside the softmax warps stay short
                // (2048 tokens after 30720 keys: 643 us; all eight unrolled 675, two at a time 698).
#pragma unroll 1
                for (int i0 = 0; i0 < kChunks; i0 += 4) {
                    uint4 codes[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) codes[i] = lds128(src + (i0 + i) * 2048);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = r0 + (i0 + i) * (128 / kChunks);
                        uint4 v = codes[i];
                        if (r >= keys) v = make_uint4(0, 0, 0, 0);   // past the sequence's end
                        uint4 lo, hi;
                        fp8x4_f16<FMT>(v.x, lo.x, lo.y);
                        fp8x4_f16<FMT>(v.y, lo.z, lo.w);
                        fp8x4_f16<FMT>(v.z, hi.x, hi.y);
                        fp8x4_f16<FMT>(v.w, hi.z, hi.w);
                        // the two halves of the row's 128-byte lines in opposite order: no bank met twice
                        const int odd = (c >> 2) & 1;
                        const int c0 = 2 * (c & 3) + odd, c1 = c0 ^ 1;
                        *reinterpret_cast<uint4 *>(dst + r * 128 + ((c0 ^ (r & 7)) << 4)) = odd ? hi : lo;
                        *reinterpret_cast<uint4 *>(dst + r * 128 + ((c1 ^ (r & 7)) << 4)) = odd ? lo : hi;
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&raw_empty[raw]);
                    mbar_arrive(&full[slot]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The parts of the broken units added up: block (c, y) joins a slice of the
// rows of the unit that CTA c of k_attn_many started and did not finish.
constexpr int kJoinSlices = 16;

template <int D>
__global__ void __launch_bounds__(256) k_attn_join(AttnArgs g, float off)
{
    dependents_launch();
    dependency_wait();
    const ManyJoin j = static_cast<const ManyJoin *>(g.many_joins)[blockIdx.x];
    if (j.rows == 0) return;
    const int c0 = blockIdx.x;
    auto part = [&](int c) { return g.many_parts + (int64_t)(2 * c + (c == c0)) * kPartFloats; };
    const float vs = g.c.v_scale ? *g.c.v_scale : 1.0f;
    constexpr int kRows = kUnitRows / kJoinSlices;
#pragma unroll 1
    for (int e = threadIdx.x; e < kRows * (D / 4); e += 256) {
        const int lrow = blockIdx.y * kRows + e % kRows, d4 = e / kRows;
        if (lrow >= j.rows) continue;
        float m = -INFINITY, l = 0.0f, lp = 0.0f;
#pragma unroll 16
        for (int c = c0; c <= j.last; ++c) m = fmaxf(m, part(c)[kUnitRows * 128 + lrow]);
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int c = c0; c <= j.last; ++c) {
            const float *p = part(c);
            const float f = m == -INFINITY ? 0.0f : ex2_approx_ftz(p[kUnitRows * 128 + lrow] - m);
            const float4 v = reinterpret_cast<const float4 *>(p)[d4 * kUnitRows + lrow];
            a.x += f * v.x;
            a.y += f * v.y;
            a.z += f * v.z;
            a.w += f * v.w;
            l += f * p[kUnitRows * 128 + kUnitRows + lrow];
            lp += f * p[kUnitRows * 128 + 2 * kUnitRows + lrow];
        }
        const float inv = lp == 0.0f ? 0.0f : vs / lp;
        const int row = j.row0 + lrow;
        const int64_t tok = j.first + row / g.group;
        const int head = j.head * g.group + row % g.group;
        const int64_t at = tok * g.out_ld + (int64_t)head * D + 4 * d4;
        if (dbg_span(at, 4, (g.tokens - 1) * g.out_ld + (int64_t)g.q_heads * D, g.status))
            *reinterpret_cast<uint2 *>(g.out + at) = make_uint2(bf16x2_rn(a.x * inv, a.y * inv), bf16x2_rn(a.z * inv, a.w * inv));
        if (g.lse && d4 == 0 && dbg_lse(g, tok * g.q_heads + head)) g.lse[tok * g.q_heads + head] = l == 0.0f ? -INFINITY : (m - off + log2f(l)) * kLn2;
    }
}

size_t many_joins_bytes() { return (size_t)sm_count() * sizeof(ManyJoin); }
size_t many_parts_bytes() { return (size_t)sm_count() * 2 * kPartFloats * sizeof(float); }

template <int D, int FMT>
static int launch_many(const AttnArgs &g, cudaStream_t st)
{
    using C = Many<D, FMT>;
    static_assert(C::kBytes <= 227 * 1024, "dynamic shared memory above the per-CTA limit");
    static bool attr_done[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (!attr_done[dev & 63]) {
        // setmaxnreg re-splits the launch's registers: the block must hold them all
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, k_attn_many<D, FMT>) != cudaSuccess) return FP8_ERR_CUDA;
        if (fa.numRegs * C::kThreads < C::kLaunchRegs) return FP8_ERR_UNSUPPORTED;
        if (cudaFuncSetAttribute(k_attn_many<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes) !=
            cudaSuccess)
            return FP8_ERR_CUDA;
        attr_done[dev & 63] = true;
    }
    const int esz = C::kFp8 ? 1 : 2, box_rows = std::min(g.c.page_size, kTile);
    const CUtensorMapDataType type = C::kFp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUtensorMap mK, mV;
    if (!make_map_pages(&mK, type, g.c.k, D, g.c.page_size, g.c.heads, g.c.num_pages, g.c.k_row_stride * esz,
                        g.c.k_head_stride * esz, g.c.k_page_stride * esz, C::kFp8 ? D : 64, box_rows, !C::kFp8) ||
        !make_map_pages(&mV, type, g.c.v, D, g.c.page_size, g.c.heads, g.c.num_pages, g.c.v_row_stride * esz,
                        g.c.v_head_stride * esz, g.c.v_page_stride * esz, C::kFp8 ? D : 64, box_rows, !C::kFp8))
        return FP8_ERR_CUDA;
    const int rc = launch_dependent(k_attn_many<D, FMT>, dim3(sm_count()), C::kThreads, C::kBytes, st, mK, mV, g, box_rows);
    if (rc != FP8_OK) return rc;
    return launch_dependent(k_attn_join<D>, dim3(sm_count(), kJoinSlices), 256, 0, st, g, C::kOff);
}

int run_many(const AttnArgs &g, cudaStream_t st)
{
    if (g.c.head_dim == 128) {
        if (g.c.format == FP8_KV_BF16) return launch_many<128, FP8_KV_BF16>(g, st);
        if (g.c.format == FP8_KV_E5M2) return launch_many<128, FP8_KV_E5M2>(g, st);
        return launch_many<128, FP8_KV_E4M3>(g, st);
    }
    if (g.c.format == FP8_KV_BF16) return launch_many<64, FP8_KV_BF16>(g, st);
    if (g.c.format == FP8_KV_E5M2) return launch_many<64, FP8_KV_E5M2>(g, st);
    return launch_many<64, FP8_KV_E4M3>(g, st);
}

}  // namespace fp8fg
