// paged.cuh -- device helpers shared by the paged key/value cache kernels.
#pragma once

#include "common.cuh"

namespace fp8fg {

// The sequence that owns new token t: the number of offsets <= t, less one
// (offsets[0 .. seqs] non-decreasing; the whole warp calls with one t).  -1 or
// seqs: t belongs to none.  The offsets are read side by side, 32 a step, so
// the latency is one load's for up to 32 sequences rather than a search's.
__device__ __forceinline__ int seq_of_token(const int32_t *__restrict__ offsets, int seqs, int64_t t, int lane)
{
    int n = 0;
    for (int i = lane; i - lane <= seqs; i += 32) {
        const bool le = i <= seqs && offsets[i] <= t;
        n += __popc(__ballot_sync(0xffffffffu, le));
    }
    return n - 1;
}

// Whether a sequence's values in the batch's arrays are within their ranges: its
// new tokens are rows [first, next) of `tokens`, len its tokens in the cache.  A
// sequence without new tokens takes no part, and its length is not looked at.
__device__ __forceinline__ bool seq_rows_ok(const fp8_paged_batch_t &b, int64_t tokens, int first, int next)
{
    return next == first || (first >= 0 && next > first && next <= tokens && next - first <= b.max_new);
}
__device__ __forceinline__ bool seq_len_ok(const fp8_paged_batch_t &b, int page_size, int len)
{
    return len >= 0 && len <= (int64_t)b.pages_per_seq * page_size;
}

struct AttnArgs {
    fp8_paged_kv_t c;
    fp8_paged_batch_t b;
    int64_t tokens, q_ld, out_ld;
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    float scale;   // softmax scale
    int q_heads, group;
    int *few_count;      // workspace: one counter a CTA of k_attn_few,
    void *few_parts;     // its parts of broken pairs,
    void *many_joins;    // k_attn_many's records of broken units
    float *many_parts;   // and their parts
    int *status;
};

// Rows of a sequence (new tokens x group) that k_attn_few takes: up to kFewRows
// from any batch, up to kFewMost if the whole batch keeps to that.
constexpr int kFewRows = 16, kFewMost = 32;
constexpr int kDirectParts = 12;   // up to so many parts of a pair k_attn_few joins without finding the maxima first

// The maximum in use may lag behind the true one by 2^kLazy before the sums
// are rescaled: no result depends on it but through roundings.
constexpr float kLazy = 8.0f;
// With a BF16 cache P is rounded to BF16 (unit roundoff 2^-8).  A row's error
// averages out over the keys that carry its weight, so where there may be few of
// them more is done: below kFineKeys keys P is the sum of two BF16 terms (an error
// of 2^-17, and a second product with V), and the key that carries most has p = 1,
// which is exact: k_attn_few's maximum never lags, nor k_attn_many's below kExactKeys,
// and beyond that it lags by less than would let a key outweigh all before it.
// k_attn_many's sum that divides the output then counts the heaviest keys as they were
// rounded.  (k_attn_few without a lag: 118 instead of 114 us for 32 sequences x 5 tokens
// over 4000 keys, no other case measured longer.  k_attn_many, an 8192-token prompt: 388
// with neither the limit nor that sum, 395 with both, 419 without a lag.)
constexpr int kFineKeys = 128, kExactKeys = 2048;
constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

// Debug build: a token's LSE of one head lies inside the output.
__device__ __forceinline__ bool dbg_lse(const AttnArgs &g, int64_t at) { return dbg_span(at, 1, g.tokens * g.q_heads, g.status); }

// Sequence b: its first row of q, its rows (new tokens x group; 0: none, or not
// to be read) and its length.  false: a value outside its range.
__device__ __forceinline__ bool seq_lengths(const AttnArgs &g, int b, int &first, int &rows, int &len)
{
    first = g.b.q_offsets[b];
    const int next = g.b.q_offsets[b + 1];
    len = g.b.kv_lens[b];
    rows = 0;
    if (next == first) return true;
    if (!seq_rows_ok(g.b, g.tokens, first, next)) return false;
    rows = (next - first) * g.group;
    if (!seq_len_ok(g.b, g.c.page_size, len)) {
        len = 0;
        return false;
    }
    return true;
}

// The four FP8 codes of w as two pairs of FP16 values, exactly.
template <int FMT>
__device__ __forceinline__ void fp8x4_f16(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    if (FMT == FP8_KV_E4M3)
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(w));
    else   // an E5M2 code is an FP16 number's upper byte
        lo = __byte_perm(w, 0, 0x1404), hi = __byte_perm(w, 0, 0x3424);
}

__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
// Programmatic dependent launch: the kernels of this family let the next kernel
// of the stream be set up while they run, and wait, before they touch memory, for
// the one before them to be complete (about 1 us less between two short calls).
__device__ __forceinline__ void dependents_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
inline int launch_dependent(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t st, A... args)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

// a / b for a >= 0, b > 0: in 32 bits where both fit (a 64-bit division takes hundreds of cycles).
__device__ __forceinline__ int64_t div_short(int64_t a, int64_t b)
{
    return (uint64_t)(a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// Inclusive sum over the CTA's threads; `total` = the last thread's.
__device__ __forceinline__ int64_t cta_scan(int64_t v, int64_t *warp_sums, int64_t &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    total = 0;
    int64_t before = 0;
    for (int i = 0; i < nw; ++i) {
        if (i < warp) before += warp_sums[i];
        total += warp_sums[i];
    }
    return v + before;
}

// Bounded wait on an mbarrier phase for roles that hand over many times a
// microsecond: the clock is read only after 256 polls (reading it at once, as
// mbar_wait_bounded does, put about 1 us on every wait that had to wait).
__device__ __forceinline__ bool wait_slow(uint32_t addr, uint32_t parity, volatile int *abort_flag, int *status)
{
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait_a(addr, parity)) return true;
        if ((i & 255u) != 0u) continue;
        if (*abort_flag) return false;
        const uint64_t t = globaltimer_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > kWaitTimeoutNs) {
            if (!*abort_flag) {
                *abort_flag = 1;
                set_status(status, FP8_ERR_TIMEOUT);
            }
            return false;
        }
    }
}
__device__ __forceinline__ bool thread_wait(uint32_t addr, uint32_t parity, volatile int *abort_flag, int *status)
{
    return mbar_try_wait_a(addr, parity) || wait_slow(addr, parity, abort_flag, status);
}
// The same for a whole warp, which stays converged.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *status)
{
    return __all_sync(0xffffffffu, thread_wait(smem_u32(bar), parity, abort_flag, status));
}

// paged_few.cu, paged_many.cu
size_t few_parts_bytes();
int few_grid();
int run_few(const AttnArgs &g, int rows, cudaStream_t st);   // sequences of up to `rows` (<= kFewMost) rows
size_t many_joins_bytes();
size_t many_parts_bytes();
int run_many(const AttnArgs &g, cudaStream_t st);

}  // namespace fp8fg
