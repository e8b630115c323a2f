// prompt_tc.cu -- the causal mixer core over packed ragged prompts on the
// sm_100a tensor cores (bf16 activations, headdim 64, d_state 128).
//
// Operation (Mamba-2 recurrence, d_conv = 4; the cache entry of "Fixed state,
// long reach: constant-size caches in large-scale block diffusion"), for each
// prompt from its pool entry's state and tail (or zeros), per head:
//     u_t = SiLU(bias + sum_j w_j raw_{t-3+j})        (x, B and C channels)
//     h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t^T,   y_t = h_t C_t + D x_t
//
// Chunked form (chunks of 128 tokens from the prompt's own start; c_t =
// inclusive prefix sum of dt A in the chunk, S = state entering it):
//     G       = C B^T
//     M[t,s]  = G[t,s] exp(c_t - c_s) dt_s  (s < t),  G[t,t] dt_t + D  (s = t)
//     Y       = exp(c_t) (C S^T) + M X
//     S      <- exp(c_last) S + (w o X)^T B,    w_s = exp(c_last - c_s) dt_s
//
// Precision.  y is to be as exact as fp32 sums rounded once to bf16: 1.7e-3
// from 64 bits in the 2-norm (2.9e-3, and 3.4e-3 on long prompts, when M, X,
// C and the state entered as bf16).  So X, M (with D on its diagonal), C and
// the copy of S in C S^T are fp16 operands, 2^-12 each, times powers of two that
// keep them inside fp16's range: X kXUnit (a channel whose values do not fit
// that in a chunk one of its own, see repair), M one a row from bounds of its
// factors, C one a token, S one a head from a bound that is carried along (a row
// far from the others its own).  B and C in G are bf16: they touch only the part
// of y that stays within the chunk.  The state is kept and handed on in fp32
// over any number of tokens, so its update is not rounded to 16 bits: w o X and
// B enter as two bf16 halves each
// (value = hi + lo to 2^-17) and three products, hi hi + lo hi + hi lo; the
// conv, SiLU and decays before them are fp32, exp(c_last - c_s) comes from
// suffix sums (no cancellation where it matters), a slow decay is applied as
// S + S expm1(c_last), and a chunk's products are summed on their own and
// added once, rounding to nearest (the tensor core's sums drop what falls
// below the accumulator's last bit: onto the state itself, thousands of such
// steps were off by 2e-5 after 32768 tokens).  So no error adds up with the
// number of chunks.  A value below 2^-29 of its scale keeps fewer than 11 bits:
// an activation below 2^-24 beside larger ones of its head in a chunk, or far
// below its channel's largest where that is past 2^8.  The conv makes X times
// kXUnit (the state's weights are divided by it), so that a sum from 2^120 on is
// an infinity: the unit after it would be one more product a value.
//
// A token's infinity or NaN must not reach the rows before it, but in M X it
// meets their zeros (0 inf = NaN): such values enter X as zeros, and the rows
// from their token on are set to NaN when they are stored (repair, stage_rows).
//
// Kernels of one call:
//   1. plan + conv of B and C: per 128-token chunk the operand rows
//      [B hi | B lo | C | C in fp16] and their exponents (zeros behind the
//      prompt's end, so that a neighbour never enters a product), and, by one
//      CTA, the table of walks.  All of it latency (10 us for 74 chunks of 11
//      prompts, alone): short loops, few scans.
//   2. only where a prompt may be long against the GPU's share of the work
//      (segment_chunks): prompts above that are cut into equal segments; a
//      state-only walk of each segment but the last, then
//   3. the states that enter the segments, chained over them.
//   4. one walk per (segment, head pair): all products on tcgen05, their sums
//      in tensor memory, the state in registers.
//
// Bounds of the walk, per chunk and head pair: 56 MMAs of 65 cycles (8 G, 8
// C S^T, 16 M X, 24 state) = 3.6K cycles, about 20K warp instructions (conv
// and SiLU, operand splitting, M, state and output scaling) = 5K cycles of
// the four schedulers, and HBM 66 KB = 1.5K cycles at the SM's share.  It
// takes 9.0K: the chain from one chunk's state product to the next's (copy of
// the state, C S^T, scaled rows, M X, G), of which the latencies of the
// products and the hand-offs are half.  Issuing the next state product ahead
// of G or M X, or freeing (w o X)^T a quarter at a time, gains nothing: the
// conv, M and the row work then wait for the same issue slots.  A walk's
// beginning and end take about 13 us besides.
// Measured, 64 heads, calls one after another on the same buffers, three cards:
// 8 prompts of 4096 tokens 374..386 us, one of 32768 534..552, 11 ragged ones of
// 8126 in all 136..139, 37 tokens 22.5 (18 of them the host's call).  On one card
// in turn with the form whose operands were all bf16: 371 for 338, 515 for 502,
// 138 for 127.
#include "common.cuh"
#include "dispatch.h"
#include "tc_ptx.cuh"

#include <algorithm>
#include <cuda.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

namespace bimamba {

namespace {

constexpr int kQ = 128;            // tokens per chunk
constexpr int kP = 64, kN = 128;   // headdim and d_state of this path
constexpr int kPP = 2 * kP;        // x channels of a head pair
constexpr int kAct = 4 * kN;       // operand row: B hi | B lo | C | C in fp16, scaled
constexpr int kXUnit = 256;        // what X^T is multiplied by, see the top
constexpr float kFltMax = 3.402823466e38f;
constexpr int kRawRows = kQ + 3;   // raw x rows of a chunk with the conv halo
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// One walk: `chunks` chunks of prompt `seq` from chunk `chunk`, whose operand
// rows start at chunk `act` of the operand array.
struct __align__(16) Walk {
    int seq, chunk, chunks, act;
    int begin, len;    // the prompt's rows
    int entry;         // its pool entry
    int resume;        // whether it continues from that
    int slot;          // entering state's slot (prompts in segments), or -1
    int last;          // the prompt's last segment
    int pad0, pad1;
};

struct PlanHeader {
    int inner, total;  // walks that are not their prompt's last; all walks
    int cuts;          // prompts in segments
    int pad;
};

struct PromptParams {
    const __nv_bfloat16 *xbc, *dt;
    const float *A, *D, *conv_w, *conv_b;
    const int *cu, *slots, *resume;
    float *state;            // pool
    __nv_bfloat16 *tail;     // pool
    __nv_bfloat16 *y, *act;
    uint8_t *b_exp, *c_exp;  // per operand row: biased exponent of the largest of its B; of what its fp16 C is to be multiplied by
    PlanHeader *head;
    Walk *walks;
    int4 *cuts;              // per prompt in segments: prompt, first slot, segments
    float *seg_state;        // [slot][H][kP][kN]
    float *seg_dec;          // [slot][H], log2 of the segment's decay before it
    int *status;
    int batch, len, H, ch, pool;
    int max_chunks;          // chunks of the operand array
    int cut_over;            // prompts of more chunks are cut
    int seg_chunks;          // into pieces of at most this many
};

// Prompt s as the plan sees it: its chunks, or none where its slot or range
// is not usable (`bad`: to be reported).
struct Prompt {
    int begin, len, chunks;
    bool ok, bad;
    bool back;   // its range runs backwards: others may overlap
};
__device__ __forceinline__ Prompt read_prompt(const PromptParams &p, int s)
{
    Prompt r{0, 0, 0, false, false, false};
    if (s >= p.batch) return r;
    const int slot = p.slots[s];
    r.begin = p.cu[s];
    const int end = p.cu[s + 1];
    r.ok = slot >= 0 && slot < p.pool && r.begin >= 0 && end >= r.begin && end <= p.len;
    r.bad = !r.ok && slot >= 0;
    r.back = end < r.begin;
    if (r.ok) {
        r.len = end - r.begin;
        r.chunks = (r.len + kQ - 1) / kQ;
    }
    return r;
}

constexpr int kPrepThreads = 512, kPrepCtas = 2;   // CTAs per chunk

// Exclusive prefix sum over the CTA's threads, and the total.
template <typename T> __device__ __forceinline__ T block_scan(T v, T *total)
{
    __shared__ T part[kPrepThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T run = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T t = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += t;
    }
    __syncthreads();
    if (lane == 31) part[warp] = run;
    __syncthreads();
    T before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPrepThreads / 32; ++w) {
        if (w < warp) before += part[w];
        all += part[w];
    }
    *total = all;
    return before + run - v;
}

__device__ __forceinline__ float rcp_approx(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// a sigmoid(a) of two values, off by a few 2^-23 (the hardware tanh's 2^-11
// would do for y but not for the state).
// kUnit: a and the result are kUnit times what they stand for.
template <int kUnit = 1> __device__ __forceinline__ float2 silu2(float2 a)
{
    const float2 t = tc::mul2(a, make_float2(-kLog2e / kUnit, -kLog2e / kUnit));
    const float2 d = tc::fma2(make_float2(tc::exp2_approx(t.x), tc::exp2_approx(t.y)), make_float2(1.0f, 1.0f),
                              make_float2(1.0f, 1.0f));
    return tc::mul2(a, make_float2(rcp_approx(d.x), rcp_approx(d.y)));
}

__device__ __forceinline__ float2 unpack2(uint32_t v)
{
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// hi = the bf16 nearest to v, lo = the bf16 nearest to v - hi, for two values.
__device__ __forceinline__ void split2(float2 v, uint32_t &hi, uint32_t &lo)
{
    hi = tc::pack_bf16x2(v.x, v.y);
    const float2 rest = tc::fma2(unpack2(hi), make_float2(-1.0f, -1.0f), v);
    lo = tc::pack_bf16x2(rest.x, rest.y);
}

// What brings values of at most 2^128 below 2^15, as fp16 operands (11 bits,
// and below 2^-29 of the largest one a fixed grain): the power of two for
// values whose largest has biased exponent `e` (kLeastExp at least, so that
// both factors are normal numbers), and the biased exponent of its inverse.
constexpr uint32_t kLeastExp = 15, kMostExp = 187;
__device__ __forceinline__ float fp16_scale(uint32_t e) { return __uint_as_float((268u - e) << 23); }
__device__ __forceinline__ uint32_t fp16_unscale_exp(uint32_t e) { return e - 14u; }

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float log2_approx(float v)
{
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// The largest of three magnitudes (a NaN does not count).
__device__ __forceinline__ float max_abs3(float a, float b, float c)
{
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 4 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr) : "memory");
}

// Store 4 consecutive 32-bit columns of this thread's TMEM lane (no wait).
__device__ __forceinline__ void tmem_st4_nw(uint32_t taddr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};"
                 ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}

}  // namespace

// Plan (the last CTA) and B/C operand rows (two CTAs per chunk of the operand
// array).  A thread convolves 4 channels of 8 tokens.
__global__ void __launch_bounds__(kPrepThreads)
prompt_prep_kernel(const PromptParams p)
{
    // the walk kernel behind this one may start its set-up
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x;
    const int me = blockIdx.x / kPrepCtas;
    if (me == p.max_chunks) {
        // ---- the table of walks.  First the walks that are not a prompt's
        // last segment (the state-only walks take exactly these), then the
        // last ones, longer before shorter in four classes, so that the long
        // walks start first.
        int inner = 0, chunks = 0;
        int cls[4] = {0, 0, 0, 0};
        auto shape = [&](const Prompt &r, int &nseg, int &seg) {
            nseg = r.chunks > p.cut_over ? (r.chunks + p.seg_chunks - 1) / p.seg_chunks : 1;
            seg = nseg > 1 ? (r.chunks + nseg - 1) / nseg : r.chunks;
            if (nseg > 1) nseg = (r.chunks + seg - 1) / seg;
        };
        // The tables hold what any prompts of p.len rows together can need.
        // Prompts of more (ranges that overlap, which takes one that runs
        // backwards) are reported from the first on that is too many.
        bool back = false;
        long long rows = 0;
        auto fits = [&](const Prompt &r, int at) {
            back = __syncthreads_or(back || r.back);
            if (back) {
                long long all;
                const long long before = rows + block_scan((long long)r.len, &all);
                rows += all;
                if (before + r.len > p.len) return false;
            }
            return at + r.chunks <= p.max_chunks;
        };
        auto class_of = [&](int n) { return min(3, 4 * n / (p.cut_over + 1)); };
        for (int s0 = 0; s0 < p.batch; s0 += kPrepThreads) {
            Prompt r = read_prompt(p, s0 + tid);
            if (r.bad) record_error(p.status, kStatusBadSlot);
            int all, nseg, seg;
            const int at = chunks + block_scan(r.chunks, &all);
            // (ranges that overlap may have any number of chunks together)
            chunks = min(chunks + all, p.max_chunks + 1);
            if (!fits(r, at) && r.ok) {
                r.ok = false;
                record_error(p.status, kStatusBadSlot);
            }
            shape(r, nseg, seg);
            block_scan(r.ok ? nseg - 1 : 0, &all);
            inner += all;
            const int c = class_of(r.chunks - (nseg - 1) * seg);
            unsigned long long four;   // 16 bits each
            block_scan(r.ok ? 1ull << 16 * c : 0ull, &four);
#pragma unroll
            for (int q = 0; q < 4; ++q) cls[q] += (int)(four >> 16 * q & 0xffffu);
        }
        int next[4];   // first walk of each class
        next[3] = inner;
        next[2] = next[3] + cls[3];
        next[1] = next[2] + cls[2];
        next[0] = next[1] + cls[1];
        int inner_at = 0, cut_at = 0;
        const int walks = next[0] + cls[0];
        chunks = 0;
        back = false;
        rows = 0;
        for (int s0 = 0; s0 < p.batch; s0 += kPrepThreads) {
            const int s = s0 + tid;
            Prompt r = read_prompt(p, s);
            int all, nseg, seg;
            const int at = chunks + block_scan(r.chunks, &all);
            chunks = min(chunks + all, p.max_chunks + 1);
            if (!fits(r, at)) r.ok = false;
            shape(r, nseg, seg);
            const bool cut = r.ok && nseg > 1;
            const int wi = inner_at + block_scan(cut ? nseg - 1 : 0, &all);
            inner_at += all;
            const int ci = cut_at + block_scan((int)cut, &all);
            cut_at += all;
            const int slot = wi + ci;   // (a cut prompt has a slot more than inner walks)
            const int tail_chunks = r.chunks - (nseg - 1) * seg;
            const int c = class_of(tail_chunks);
            unsigned long long four;
            const unsigned long long before = block_scan(r.ok ? 1ull << 16 * c : 0ull, &four);
            int wl = (int)(before >> 16 * c & 0xffffu);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (c == q) wl += next[q];
                next[q] += (int)(four >> 16 * q & 0xffffu);
            }
            if (cut) p.cuts[ci] = make_int4(s, slot, nseg, 0);
            if (!r.ok) continue;
            const int entry = p.slots[s], resume = p.resume && p.resume[s] != 0;
            for (int i = 0; i < nseg - 1; ++i)
                p.walks[wi + i] = Walk{s, i * seg, seg, at + i * seg, r.begin, r.len, entry, resume, slot + i, 0, 0, 0};
            const int first = (nseg - 1) * seg;
            p.walks[wl] = Walk{s,      first, tail_chunks, at + first, r.begin, r.len, entry,
                               resume, cut ? slot + nseg - 1 : -1, 1, 0, 0};
        }
        if (tid == 0) *p.head = PlanHeader{inner, walks, cut_at, 0};
        return;
    }

    // ---- which prompt's chunk is chunk `me` of the operand array
    __shared__ int4 found;   // prompt, chunk in it, begin, len
    if (tid == 0) found = make_int4(-1, 0, 0, 0);
    int chunks = 0;
    for (int s0 = 0; s0 < p.batch && chunks <= me; s0 += kPrepThreads) {
        const Prompt r = read_prompt(p, s0 + tid);
        int all;
        const int at = chunks + block_scan(r.chunks, &all);
        chunks += all;
        if (r.ok && at <= me && me < at + r.chunks && at + r.chunks <= p.max_chunks)
            found = make_int4(s0 + tid, me - at, r.begin, r.len);
    }
    __syncthreads();
    const int4 f = found;
    if (f.x < 0) return;
    const int n0 = 4 * (tid & 63);             // channels n0 .. n0 + 3 of [B | C]
    const int c = p.H * kP + n0;
    const int i0 = (blockIdx.x % kPrepCtas) * (kQ / kPrepCtas) + 8 * (tid >> 6);   // first token of this thread
    const int t0 = f.y * kQ + i0;              // in the chunk and in the prompt
    const __nv_bfloat16 *raw = p.xbc + (size_t)f.z * p.ch + c;
    const bool resume = p.resume && p.resume[f.x] != 0;
    const __nv_bfloat16 *tail = p.tail + (size_t)p.slots[f.x] * 4 * p.ch + c;
    auto at = [&](int t) -> uint2 {
        if (t >= f.w) return make_uint2(0u, 0u);
        if (t >= 0) return *reinterpret_cast<const uint2 *>(raw + (size_t)t * p.ch);
        return resume ? *reinterpret_cast<const uint2 *>(tail + (size_t)(4 + t) * p.ch) : make_uint2(0u, 0u);
    };
    uint2 rows[11];
#pragma unroll
    for (int i = 0; i < 11; ++i) rows[i] = at(t0 - 3 + i);
    float w[4][4], bias[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float4 t = *reinterpret_cast<const float4 *>(p.conv_w + (size_t)(c + q) * 4);
        w[q][0] = t.x; w[q][1] = t.y; w[q][2] = t.z; w[q][3] = t.w;
        bias[q] = p.conv_b ? p.conv_b[c + q] : 0.0f;
    }
    __nv_bfloat16 *out = p.act + ((size_t)me * kQ + i0) * kAct;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = bias[q];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v0 = unpack2(rows[i + j].x), v1 = unpack2(rows[i + j].y);
            o[0] = fmaf(w[0][j], v0.x, o[0]);
            o[1] = fmaf(w[1][j], v0.y, o[1]);
            o[2] = fmaf(w[2][j], v1.x, o[2]);
            o[3] = fmaf(w[3][j], v1.y, o[3]);
        }
        uint2 hi, lo;
        const bool in = t0 + i < f.w;
        const float2 zero = make_float2(0.0f, 0.0f);
        const float2 a0 = in ? silu2(make_float2(o[0], o[1])) : zero, a1 = in ? silu2(make_float2(o[2], o[3])) : zero;
        split2(a0, hi.x, lo.x);
        split2(a1, hi.y, lo.y);
        __nv_bfloat16 *row = out + (size_t)i * kAct;
        // (a token's B, and its C, is a warp's)
        const uint32_t big = __float_as_uint(fmaxf(fmaxf(fabsf(a0.x), fabsf(a0.y)), fmaxf(fabsf(a1.x), fabsf(a1.y))));
        const uint32_t e = max(__reduce_max_sync(0xffffffffu, big) >> 23, kLeastExp);
        if (n0 < kN) {
            *reinterpret_cast<uint2 *>(row + n0) = hi;
            *reinterpret_cast<uint2 *>(row + kN + n0) = lo;
            if (n0 == 0) p.b_exp[(size_t)me * kQ + i0 + i] = (uint8_t)e;
        } else {
            *reinterpret_cast<uint2 *>(row + kN + n0) = hi;
            const float2 s2 = make_float2(fp16_scale(e), fp16_scale(e));
            const float2 c0 = tc::mul2(a0, s2), c1 = tc::mul2(a1, s2);
            *reinterpret_cast<uint2 *>(row + 2 * kN + n0) = make_uint2(pack_f16x2(c0.x, c0.y), pack_f16x2(c1.x, c1.y));
            if (n0 == kN) p.c_exp[(size_t)me * kQ + i0 + i] = (uint8_t)fp16_unscale_exp(e);
        }
    }
}

// The states entering each segment of a cut prompt, over its slots in order:
// slot i holds the end state from zero of segment i - 1 (and its decay) and
// gets E_i, E_0 = the prompt's initial state, E_i = 2^dec E_{i-1} + S_{i-1}.
__global__ void __launch_bounds__(256)
prompt_chain_kernel(const PromptParams p)
{
    // (a programmatic launch; the walks behind it may start once the state-only
    // ones are done: before that they would take their places)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.y >= p.head->cuts) return;
    const int4 cut = p.cuts[blockIdx.y];
    const int s = cut.x;
    const int e = blockIdx.x * 256 + threadIdx.x;   // float4 of the state
    const int per = p.H * kP * kN / 4;
    if (e >= per) return;
    const int h = e / (kP * kN / 4);
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (p.resume && p.resume[s] != 0)
        v = reinterpret_cast<const float4 *>(p.state)[(size_t)p.slots[s] * per + e];
    float4 *st = reinterpret_cast<float4 *>(p.seg_state) + (size_t)cut.y * per + e;
    *st = v;
    for (int i = 1; i < cut.z; ++i) {
        st += per;
        const float a = exp2f(p.seg_dec[(size_t)(cut.y + i) * p.H + h]);
        const float4 q = *st;
        v.x = fmaf(a, v.x, q.x);
        v.y = fmaf(a, v.y, q.y);
        v.z = fmaf(a, v.z, q.z);
        v.w = fmaf(a, v.w, q.w);
        *st = v;
    }
}

namespace {

// ---- the walk kernel's shared memory (bytes from a 1024-aligned base)
constexpr uint32_t kTile = 32768;                   // 128 x 128 bf16: two 64-wide swizzled blocks
constexpr uint32_t kOffC = 0;                       // C  [t][n]: bf16 for G, then fp16 for C S^T
constexpr uint32_t kOffBh = kOffC + kTile;          // B hi [s][n]
constexpr uint32_t kOffBl = kOffBh + kTile;         // B lo [s][n], then the fp16 copy of the state [p'][n]
constexpr uint32_t kOffX0 = kOffBl + kTile;         // X^T [p'][s], then the finished rows: even chunks
constexpr uint32_t kOffX1 = kOffX0 + kTile;         // odd chunks
constexpr uint32_t kOffRaw1 = kOffX1;               // raw x [131][128] of odd chunks (state-only walk: no X^T)
constexpr uint32_t kOffRaw = kOffX1 + kTile + 1024; // of even ones (of all, in the other walk)
constexpr uint32_t kRawBytes = kRawRows * kPP * 2;
static_assert(kOffRaw1 + kRawBytes <= kOffRaw, "raw buffers");
constexpr uint32_t kOffFac = kOffRaw + kRawBytes;   // per-slot factors, f32 [2 parity][2 head][128] each:
constexpr uint32_t kFac = 2 * 2 * kQ * 4;
constexpr uint32_t kOffCum = kOffFac;               //   prefix sums of dt A, log2 units
constexpr uint32_t kOffDt = kOffCum + kFac;         //   dt
constexpr uint32_t kOffFB = kOffDt + kFac;          //   exp(c_R - c_s) dt_s, R = end of s's 32-slot block
constexpr uint32_t kOffF4 = kOffFB + kFac;          //   exp(c_R4 - c_s) dt_s, R4 = s | 3
constexpr uint32_t kOffWgt = kOffF4 + kFac;         //   w_s / kXUnit
constexpr uint32_t kOffColF = kOffWgt + kFac;       // float [128]: what takes a state row's own scale from a column of C S^T
constexpr uint32_t kOffSMax = kOffColF + kPP * 4;   // float [2][128]: largest of a state row's halves
constexpr uint32_t kOffCExp = kOffSMax + 8 * kPP;   // u8 [2 parity][128]: c_exp
constexpr uint32_t kOffMUnit = kOffCExp + 2 * kQ;   // float [2 parity][2 head][128]: what M's rows are multiplied by
constexpr uint32_t kOffXFac = kOffMUnit + kFac;     // float [2 parity][128]: what channels of X^T are multiplied by besides, see repair
constexpr uint32_t kOffGrow = kOffXFac + 2 * kPP * 4;   // float [2 parity][2 head]: what the chunk adds to the state for |x| = 1 at most
constexpr uint32_t kOffXRow = kOffGrow + 16;        // fp16 [2 parity][part][128]: largest of X^T's magnitudes, of a thread
constexpr int kParts = 5;                           // of a chunk's units: 3 x 4 (X group), 2 x 2 (M group)
constexpr uint32_t kOffXHead = kOffXRow + 2 * kParts * kPP * 2;   // u32 [2 parity][2 head]: the same of a head, zeros between
constexpr uint32_t kOffXMost = kOffXHead + 16;      // float [2 parity][2 head]: bound of the head's finite |x|
constexpr uint32_t kOffMOff = kOffXMost + 16;        // int: the M group's share of X^T is not as it should be
constexpr uint32_t kOffAgain = kOffMOff + 4;        // int: X^T has to be made again
constexpr uint32_t kOffWMax = kOffAgain + 12;       // float [2 head][4]: largest of a Y warp's state values
constexpr uint32_t kOffHeadF = kOffWMax + 32;       // float [2 head]: what takes the state copy's scale from C S^T
constexpr uint32_t kOffRowwise = kOffHeadF + 8;     // int [2 head], see choose_scale
constexpr uint32_t kOffScale = kOffRowwise + 8;     // float2 [2 parity][2 head]: see next_state
constexpr uint32_t kOffBad = kOffScale + 32;        // u8 [2 parity][3][128]: first token of X not finite (128: none), see repair
constexpr uint32_t kOffAnyBad = kOffBad + 6 * kPP;  // int [2 parity]: there is one; int [2 parity]: kOffXFac is not all 1
constexpr uint32_t kOffDtBuf = kOffAnyBad + 16;     // [2][128] bf16x2: dt of both heads
constexpr uint32_t kOffTaps = kOffDtBuf + 2 * kQ * 4;   // float4 [128] conv taps, float [128] biases, float [2] D, float [3][128] halo
constexpr uint32_t kOffMbar = kOffTaps + kPP * 20 + 8 + 3 * kPP * 4;
constexpr uint32_t kOffTmem = kOffMbar + 192;
constexpr uint32_t kStateRow = kN * 4 + 16;         // a row of the last state on its way out: 16-byte stores of
static_assert(kPP * kStateRow <= 3 * kTile, "state rows");   // 8 threads' rows meet no bank twice

constexpr uint32_t kSmemBytes = kOffTmem + 16 + 1024;   // + alignment slack
static_assert(kOffRaw % 1024 == 0 && kOffFac % 16 == 0 && kOffColF % 16 == 0 && kOffCExp % 4 == 0 && kOffMUnit % 16 == 0 &&
                  kOffXFac % 4 == 0 && kOffXRow % 4 == 0 && kOffXHead % 4 == 0 && kOffWMax % 16 == 0 &&
                  kOffScale % 8 == 0 && kOffAnyBad % 4 == 0 && kOffDtBuf % 16 == 0 && kOffTaps % 16 == 0 && kOffMbar % 8 == 0 &&
                  kOffTmem % 4 == 0 && kSmemBytes <= 227 * 1024, "shared memory");

// ---- tensor memory columns
constexpr uint32_t kColG = 0;      // G, then in place [M_0 | M_1] per 16 tokens (8 + 8 columns of bf16 pairs)
constexpr uint32_t kColY = 128;    // Y, 64 columns per head
constexpr uint32_t kColW = 256;    // (w o X)^T, A operand: 64 columns hi, 64 columns lo
constexpr uint32_t kColS = 384;    // a chunk's (w o X)^T B [p' = lane][n], fp32

// ---- warps: groups of 8, 8 and 12 and 4 single ones (the register shares
// below are given to whole sets of 4 warps)
constexpr int kMGroup = 256, kYGroup = 256, kXGroup = 384;   // threads
constexpr int kYWarp = 8, kXWarp = 16, kProducerWarp = 28, kHelperWarp = 29, kPublisherWarp = 30, kTailWarp = 31;
constexpr int kThreads = 32 * 32;
// registers a thread: 1024 threads are launched with 64; the Y group holds
// the state (64 values a thread)
constexpr int kRegsLaunch = 64, kRegsM = 56, kRegsY = 96, kRegsX = 56, kRegsOne = 40;
static_assert(kRegsM * kMGroup + kRegsY * kYGroup + kRegsX * kXGroup + kRegsOne * 128 <= kRegsLaunch * kThreads, "register shares");

template <int kRegs> __device__ __forceinline__ void take_registers()
{
    if constexpr (kRegs > kRegsLaunch)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Bounded wait for phase `parity` of `bar`: false after kWaitTries tries (a
// try that finds the phase incomplete takes some tens of cycles: half a second
// and more, where the longest wait of a walk is tens of microseconds).  Three
// instructions a try: the waiting threads poll beside the warps that compute.
constexpr uint32_t kWaitTries = 1u << 24;

__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 n;\n\t"
        "mov.b32 n, %3;\n\t"
        "TRY:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE;\n\t"
        "sub.u32 n, n, 1;\n\t"
        "setp.ne.u32 q, n, 0;\n\t"
        "@q bra TRY;\n\t"
        "DONE:\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity), "n"(kWaitTries) : "memory");
    return ok != 0;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// Barriers over a group's threads (named barrier `id`).
template <int kCount> __device__ __forceinline__ void grp_sync(int id)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kCount) : "memory");
}

template <int kCount> __device__ __forceinline__ bool grp_or(int id, bool pred)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %2, 0;\n\t"
        "bar.red.or.pred q, %1, %3, p;\n\t"
        "selp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"(id), "r"((uint32_t)pred), "n"(kCount) : "memory");
    return r != 0;
}

template <int kCount> __device__ __forceinline__ bool grp_and(int id, bool pred)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %2, 0;\n\t"
        "bar.red.and.pred q, %1, %3, p;\n\t"
        "selp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"(id), "r"((uint32_t)pred), "n"(kCount) : "memory");
    return r != 0;
}

}  // namespace

// One walk of one head pair.  kStateOnly: from a zero state, writing the end
// state and decay of a segment, no outputs.
//
// Warp roles (hand-offs through mbarriers, every wait bounded; [k] = once
// per chunk):
//   warps 0..7   M group: M(k) in place over G(k); a quarter of the X group's
//                work on chunk k + 1.
//   warps 8..15  Y group: the state (in registers) and its bf16 copy; the rows
//                of C S^T scaled by exp(c_t) in place, ready for M X to be
//                added; the finished rows over the chunk's X^T.
//   warps 16..27 X group: conv + SiLU of the chunk's raw rows, X^T and both
//                halves of (w o X)^T (the largest share of the instructions,
//                so the largest group).
//   warp 28      producer: every MMA, the B/C tile loads.
//   warp 29      helper: dt copies, prefix sums and factors, two chunks ahead.
//   warp 30      publisher: finished rows to y.
//   warp 31      the new tail of the prompt's entry (behind the others' loops
//                in the code: there it costs them no registers).
template <bool kStateOnly>
__global__ void __launch_bounds__(kThreads, 1)
prompt_walk_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_bc,
                   const __grid_constant__ CUtensorMap tm_y, const PromptParams p)
{
    extern __shared__ uint8_t smem_raw[];
    // (an offset, not a cast of the rounded address: so the compiler still
    // knows the space, and addresses are 32 bits)
    uint8_t *sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = tc::smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int H = p.H, ch = p.ch, HP = H / 2;
    const int hp = blockIdx.x % HP;
    const int wi = blockIdx.x / HP;
    float *cum = reinterpret_cast<float *>(sm + kOffCum);
    float *dts = reinterpret_cast<float *>(sm + kOffDt);
    float *fB = reinterpret_cast<float *>(sm + kOffFB);
    float *f4 = reinterpret_cast<float *>(sm + kOffF4);
    float *wgt = reinterpret_cast<float *>(sm + kOffWgt);
    float2 *scl = reinterpret_cast<float2 *>(sm + kOffScale);
    uint8_t *bad_at = sm + kOffBad;
    int *any_bad = reinterpret_cast<int *>(sm + kOffAnyBad);
    const uint32_t mb = sbase + kOffMbar;
    const uint32_t mb_bc = mb;            // [k] B/C tiles landed (state-only: even chunks, odd ones at mb_g)
    const uint32_t mb_x = mb + 8;         // [k] raw x landed (state-only: even chunks, odd ones at mb_cs)
    const uint32_t mb_cs = mb + 16;       // [k] the copy of the state entering it ready
    const uint32_t mb_g = mb + 24;        // [k] G done
    const uint32_t mb_m = mb + 32;        // [k] M ready
    const uint32_t mb_s = mb + 40;        // [k] kColS free (the last chunk's products taken)
    const uint32_t mb_yo = mb + 48;       // [k] C S^T done
    const uint32_t mb_ys = mb + 56;       // [k] its rows scaled
    const uint32_t mb_e = mb + 64;        // [k] M X done
    const uint32_t mb_st = mb + 72;       // [k] rows staged, Y columns free
    // the rest one for even and one for odd chunks (+8): a wait may come
    // after the next chunk's phase has completed, never after the next but one
    const uint32_t mb_w0 = mb + 80;       // X^T and (w o X)^T ready
    const uint32_t mb_sd0 = mb + 96;      // state product done
    const uint32_t mb_dt0 = mb + 112;     // factors ready
    const uint32_t mb_free0 = mb + 128;   // their buffer free
    const uint32_t mb_xf0 = mb + 144;     // X^T's buffer free (the rows over it stored)
    const uint32_t mb_c16 = mb + 160;     // [k] fp16 C landed
    const uint32_t mb_mc = mb + 168;      // [k] the M group's share of X^T ready
    const uint32_t mb_end = mb + 176;     // MMAs done, after a wait that gave up
    auto of = [](uint32_t pair, int k) { return pair + 8 * (k & 1); };
    auto phase = [](int k) -> uint32_t { return (k >> 1) & 1; };   // of a pair's barrier
    auto xbuf = [](int k) { return (k & 1) ? kOffX1 : kOffX0; };
    // ---- set-up: first what no kernel before this one has written (a
    // programmatic launch: this may run beside the end of that one)
    float4 *taps = reinterpret_cast<float4 *>(sm + kOffTaps);
    float *biases = reinterpret_cast<float *>(sm + kOffTaps + kPP * 16);   // then D of both heads
    float4 my_taps = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float my_bias = 0.0f, A0 = 0.0f, A1 = 0.0f;
    if (tid < kPP) {
        my_taps = *reinterpret_cast<const float4 *>(p.conv_w + (size_t)(hp * kPP + tid) * 4);
        my_bias = p.conv_b ? p.conv_b[hp * kPP + tid] : 0.0f;
    }
    if (warp == kHelperWarp) {
        A0 = p.A[2 * hp] * kLog2e;
        A1 = p.A[2 * hp + 1] * kLog2e;
    }
    if (tid == 32 * kProducerWarp) {
        tc::prefetch_tmap(&tm_x);
        tc::prefetch_tmap(&tm_bc);
        if (!kStateOnly) tc::prefetch_tmap(&tm_y);
        tc::mbar_init(mb_bc, kStateOnly ? 2 : 3);
        tc::mbar_init(mb_g, kStateOnly ? 2 : 1);
        for (uint32_t b = mb_x; b < mb_dt0; b += 8)
            if (b != mb_g && b != mb_w0 && b != mb_w0 + 8) tc::mbar_init(b, 1);
        tc::mbar_init(mb_w0, 2);       // the X and the M group
        tc::mbar_init(mb_w0 + 8, 2);
        tc::mbar_init(mb_c16, 1);
        tc::mbar_init(mb_mc, 1);
        tc::mbar_init(mb_end, 1);
        tc::mbar_init(mb_xf0, 1);
        tc::mbar_init(mb_xf0 + 8, 1);
        tc::mbar_init(mb_dt0, 32);
        tc::mbar_init(mb_dt0 + 8, 32);
        tc::mbar_init(mb_free0, 3);
        tc::mbar_init(mb_free0 + 8, 3);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (kStateOnly) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Walk wk = p.walks[wi];   // (requested beside the table's length: the table has an entry for every CTA)
    if (wi >= (kStateOnly ? p.head->inner : p.head->total)) return;
    const int slot = wk.entry, begin = wk.begin, len = wk.len;
    const bool resume = wk.resume != 0;
    const int nk = wk.chunks;
    __nv_bfloat16 *tail = p.tail + (size_t)slot * 4 * ch;
    // chunk k's rows in the prompt
    const int left = len - wk.chunk * kQ, row0 = begin + wk.chunk * kQ;
    auto tokens = [&](int k) { return min(kQ, left - k * kQ); };
    auto first_row = [&](int k) { return row0 + k * kQ; };

    // (the state-only walk has two raw buffers)
    auto raw_off = [](int k) { return kStateOnly && (k & 1) ? kOffRaw1 : kOffRaw; };
    auto x_bar = [&](int k) { return kStateOnly && (k & 1) ? mb_cs : mb_x; };
    struct { uint32_t x, bc, c16; } loads = {0, 0, 0};   // requests so far, of the thread that makes them
    auto issue_x = [&](int k) {
        ++loads.x;
        tc::mbar_expect_tx(x_bar(k), kRawBytes);
        tc::tma_load_3d(sbase + raw_off(k), &tm_x, hp * kPP, first_row(k) - 3, 0, x_bar(k));
    };
    // B hi, B lo and C tiles of chunk k: three arrivals of mb_bc's phase (two
    // in the state-only walk, which has two B buffers: odd chunks in the C and
    // X tiles, on mb_g).
    auto bh_off = [](int k) { return kStateOnly && (k & 1) ? kOffC : kOffBh; };
    auto bl_off = [](int k) { return kStateOnly && (k & 1) ? kOffX0 : kOffBl; };
    auto b_bar = [&](int k) { return kStateOnly && (k & 1) ? mb_g : mb_bc; };
    auto issue_tile = [&](int k, uint32_t off, int col, uint32_t bar) {
        const int row = (wk.act + k) * kQ;
        tc::mbar_expect_tx(bar, kTile);
        tc::tma_load_3d(sbase + off, &tm_bc, col, row, 0, bar);
        tc::tma_load_3d(sbase + off + kTile / 2, &tm_bc, col + 64, row, 0, bar);
    };
    auto issue_bh = [&](int k) { ++loads.bc; issue_tile(k, bh_off(k), 0, b_bar(k)); };
    auto issue_bl = [&](int k) { ++loads.bc; issue_tile(k, bl_off(k), kN, b_bar(k)); };
    auto issue_c = [&](int k) { ++loads.bc; issue_tile(k, kOffC, 2 * kN, mb_bc); };
    auto issue_c16 = [&](int k) { ++loads.c16; issue_tile(k, kOffC, 3 * kN, mb_c16); };

    // helper warp: dt of both heads (adjacent: one 4-byte copy per token)
    auto load_dt_async = [&](int k) {
        const int cnt = tokens(k);
        uint32_t *dst = reinterpret_cast<uint32_t *>(sm + kOffDtBuf) + (k & 1) * kQ;
        const __nv_bfloat16 *src = p.dt + (size_t)first_row(k) * H + 2 * hp;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = 4 * lane + i;
            if (j < cnt)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;"
                             ::"r"(tc::smem_u32(dst + j)), "l"(src + (size_t)j * H) : "memory");
            else
                dst[j] = 0u;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    if (tid == 32 * kProducerWarp) {
        if (nk > 0) {
            issue_x(0);
            issue_bh(0);
            issue_bl(0);
            if (!kStateOnly) issue_c(0);
        }
        if (kStateOnly && nk > 1) {
            issue_x(1);
            issue_bh(1);
            issue_bl(1);
        }
    }
    if (warp == kHelperWarp) {
        if (nk > 0) load_dt_async(0);
        if (nk > 1) load_dt_async(1);
    }
    if (warp == 0) tc::tmem_alloc(sbase + kOffTmem, 512);
    if (tid < kPP) {
        taps[tid] = make_float4(kXUnit * my_taps.x, kXUnit * my_taps.y, kXUnit * my_taps.z, kXUnit * my_taps.w);
        biases[tid] = kXUnit * my_bias;
    }
    if (tid < 2) biases[kPP + tid] = p.D[2 * hp + tid];
    if (tid < 4) reinterpret_cast<uint32_t *>(sm + kOffXHead)[tid] = 0u;
    if (tid < 2) reinterpret_cast<int *>(sm + kOffRowwise)[tid] = 0;
    // the 3 tokens before the walk's first chunk where they are not in the raw
    // tile: the prompt's entry's tail, or zeros
    const bool starts = wk.chunk == 0;
    float *halo = biases + kPP + 2;   // [3][128]
    if (starts && tid < 3 * kPP)
        halo[tid] = resume ? __bfloat162float(tail[(1 + tid / kPP) * ch + hp * kPP + tid % kPP]) : 0.0f;
    // an entry that two prompts name belongs to neither
    bool twice = false;
    if (!kStateOnly)
        for (int r = tid; r < p.batch; r += kThreads) twice |= r != wk.seq && p.slots[r] == slot;
    tc::fence_before_sync();
    twice = __syncthreads_or(twice);
    tc::fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sm + kOffTmem);
    if (!kStateOnly && twice) {
        // (the copies on their way land first)
        if (tid == 32 * kProducerWarp) {
            if (nk > 0 && !(mbar_wait(mb_x, 0) && mbar_wait(mb_bc, 0))) record_error(p.status, kStatusTimeout);
            if (hp == 0 && wk.last) record_error(p.status, kStatusBadSlot);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        if (warp == 0) tc::tmem_dealloc(tmem, 512);
        return;
    }

    // conv + SiLU of channel p' = pr, units ua .. ub - 1 (8 tokens each) of
    // chunk k: X^T to shared memory, both halves of (w o X)^T to tensor
    // memory (lane = channel, so that a thread's tokens are consecutive:
    // 16-byte stores of X^T, and the A operand's layout).  Returns whether a
    // value is not finite, in X^T's fp16 with kXUnit at least.
    auto conv_units = [&](int k, int pr, int ua, int ub, int part) -> bool {
        const int par = k & 1;
        const float4 w4 = taps[pr];
        const float bias = biases[pr];
        const uint8_t *raw = sm + raw_off(k) + 2 * pr;
        auto ld = [&](int i) -> float {   // row i of the tile: token i - 3 of the chunk
            return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(raw + i * (kPP * 2))) << 16);
        };
        const int rows = tokens(k) + 3;   // rows past these are a neighbour's
        float v0 = ld(8 * ua), v1 = ld(8 * ua + 1), v2 = ld(8 * ua + 2);
        if (ua == 0 && k == 0 && starts) {
            v0 = halo[pr];
            v1 = halo[kPP + pr];
            v2 = halo[2 * kPP + pr];
        } else {
            if (8 * ua >= rows) v0 = 0.0f;
            if (8 * ua + 1 >= rows) v1 = 0.0f;
            if (8 * ua + 2 >= rows) v2 = 0.0f;
        }
        const float *ws = wgt + (par * 2 + (pr >> 6)) * kQ;
        const uint32_t wcol = tmem + (static_cast<uint32_t>(pr & 96) << 16) + kColW - (kStateOnly && par ? kColW : 0u);
        uint8_t *xt = sm + xbuf(k);
        const float2 wa = make_float2(w4.x, w4.x), wc = make_float2(w4.z, w4.z), b2 = make_float2(bias, bias);
        // unit u's 16 bytes of X^T's row
        auto piece = [&](int u) { return (u >> 3) * (kTile / 2) + tc::sw128(pr, u & 7); };
        [[maybe_unused]] uint32_t largest = 0u;   // of X^T's magnitudes, the words of an fp16 pair
#pragma unroll 2
        for (int u = ua; u < ub; ++u) {
            float v[11];
            v[0] = v0; v[1] = v1; v[2] = v2;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[3 + i] = ld(8 * u + 3 + i);
            if (8 * u + 11 > rows) {
                // a neighbour's rows: zeros (what the conv makes of them meets
                // dt = 0 and M = 0)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (8 * u + 3 + i >= rows) v[3 + i] = 0.0f;
            }
            v0 = v[8]; v1 = v[9]; v2 = v[10];
            const float4 w01 = *reinterpret_cast<const float4 *>(ws + 8 * u);
            const float4 w23 = *reinterpret_cast<const float4 *>(ws + 8 * u + 4);
            uint32_t hi[4], lo[4];
            [[maybe_unused]] uint32_t xp[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // tokens 2 j, 2 j + 1 of the unit: taps 0 and 2 as packed pairs
                float2 a = tc::fma2(wa, make_float2(v[2 * j], v[2 * j + 1]), b2);
                a = tc::fma2(wc, make_float2(v[2 * j + 2], v[2 * j + 3]), a);
                a.x = fmaf(w4.y, v[2 * j + 1], a.x);
                a.y = fmaf(w4.y, v[2 * j + 2], a.y);
                a.x = fmaf(w4.w, v[2 * j + 3], a.x);
                a.y = fmaf(w4.w, v[2 * j + 4], a.y);
                const float2 x = silu2<kXUnit>(a);
                if constexpr (!kStateOnly) {
                    xp[j] = pack_f16x2(x.x, x.y);
                    if (j & 1) largest = __vimax3_u16x2(largest, xp[j - 1] & 0x7fff7fffu, xp[j] & 0x7fff7fffu);
                }
                const float2 w = j == 0 ? make_float2(w01.x, w01.y) : j == 1 ? make_float2(w01.z, w01.w)
                               : j == 2 ? make_float2(w23.x, w23.y) : make_float2(w23.z, w23.w);
                split2(tc::mul2(x, w), hi[j], lo[j]);
            }
            if constexpr (!kStateOnly)
                *reinterpret_cast<uint4 *>(xt + piece(u)) = make_uint4(xp[0], xp[1], xp[2], xp[3]);
            tmem_st4_nw(wcol + 4 * u, hi);
            tmem_st4_nw(wcol + 64 + 4 * u, lo);
        }
        if constexpr (!kStateOnly) {
            largest = max(largest >> 16, largest & 0xffffu);
            reinterpret_cast<uint16_t *>(sm + kOffXRow)[(par * kParts + part) * kPP + pr] = (uint16_t)largest;
            const uint32_t all = __reduce_max_sync(0xffffffffu, largest);
            if (lane == 0) atomicMax(reinterpret_cast<uint32_t *>(sm + kOffXHead) + 2 * par + (pr >> 6), all);
        }
        tc::tmem_wait_st();
        if constexpr (!kStateOnly) tc::fence_proxy_async();   // X^T, for the tensor core
        tc::fence_before_sync();
        return !kStateOnly && largest >= 0x7c00u;
    };
    // X^T of chunk k once more (rare), by the X group, all 16 units of 8 tokens
    // from the raw rows: values that are not finite as zeros, the first such
    // token of a channel noted in bad_at; a channel whose largest value is past
    // fp16's range or near its small end times a power of two of its own.  (8
    // prompts of 4096 tokens whose every chunk has activations past 2^8: 828 us
    // for 380.)
    float *xfac = reinterpret_cast<float *>(sm + kOffXFac);
    auto repair = [&](int k, int third, int pr) {
        const int par = k & 1;
        const float4 w4 = taps[pr];
        const float bias = biases[pr];
        const int rows = tokens(k) + 3;
        const uint16_t *raw = reinterpret_cast<const uint16_t *>(sm + raw_off(k)) + pr;
        auto row = [&](int t) -> float {   // as in conv_units
            return t < rows ? __uint_as_float(static_cast<uint32_t>(raw[t * kPP]) << 16) : 0.0f;
        };
        // this thread's third of the tokens, in order: f(token, activation), in
        // the same steps as there
        auto each = [&](auto f) {
            constexpr int kThird = (kQ + 2) / 3;
            const int i0 = kThird * third, i1 = min(i0 + kThird, kQ);
            const bool in_halo = i0 == 0 && k == 0 && starts;
            float v0 = in_halo ? halo[pr] : row(i0), v1 = in_halo ? halo[kPP + pr] : row(i0 + 1);
            float v2 = in_halo ? halo[2 * kPP + pr] : row(i0 + 2);
#pragma unroll 4
            for (int i = i0; i < i1; ++i) {
                const float v3 = row(i + 3);
                const float a = fmaf(w4.w, v3, fmaf(w4.y, v1, fmaf(w4.z, v2, fmaf(w4.x, v0, bias))));
                f(i, silu2<kXUnit>(make_float2(a, a)).x);
                v0 = v1;
                v1 = v2;
                v2 = v3;
            }
        };
        uint32_t *most = reinterpret_cast<uint32_t *>(xfac + par * kPP + pr);   // (of the channel, until its factor is known)
        float big = 0.0f;
        int at = kQ;
        if (third == 0) *most = 0u;
        grp_sync<kXGroup>(3);
        each([&](int i, float x) {
            const float v = fabsf(x);
            if (v <= kFltMax) big = fmaxf(big, v);
            else at = min(at, i);
        });
        bad_at[(par * 3 + third) * kPP + pr] = (uint8_t)at;
        if (at < kQ) any_bad[par] = 1;
        atomicMax(most, __float_as_uint(big));
        atomicMax(reinterpret_cast<uint32_t *>(sm + kOffXMost) + 2 * par + (pr >> 6), __float_as_uint(big * (1.0f / kXUnit)));
        grp_sync<kXGroup>(3);
        big = __uint_as_float(*most);
        const bool own = big >= 65504.0f || (big < 0x1p-12f && big != 0.0f);
        const float f = own ? __uint_as_float(min(max(268u - (__float_as_uint(big) >> 23), 127u - 113u), 127u + 40u) << 23) : 1.0f;
        if (own) any_bad[2 + par] = 1;
        grp_sync<kXGroup>(3);
        if (third == 0) xfac[par * kPP + pr] = f;
        __half *xt = reinterpret_cast<__half *>(sm + xbuf(k));
        each([&](int i, float x) {
            xt[(i >> 6) * (kTile / 4) + tc::sw128(pr, i >> 3 & 7) / 2 + (i & 7)] = __float2half_rn(fabsf(x) <= kFltMax ? f * x : 0.0f);
        });
        tc::fence_proxy_async();
        grp_sync<kXGroup>(3);
    };
    // One thread's waits (after one that gave up, the rest are not tried).
    auto wait = [&](bool ok, uint32_t bar, uint32_t parity) -> bool {
        return ok && mbar_wait(bar, parity);
    };
    // What conv_units(k) waits for: the raw rows, the factors, X^T's buffer
    // (the rows of the chunk before last stored) and (w o X)^T's columns (the
    // last chunk's product done; the state-only walk has two sets of them).
    // One lane each of a group's first four warps waits for one of these.
    auto x_ready = [&](int k, int first) -> bool {
        const int w = tid - first;
        if (w == 0) return wait(true, of(mb_dt0, k), phase(k));
        if (w == 32) return wait(true, x_bar(k), kStateOnly ? phase(k) : k & 1);
        if (kStateOnly) {
            if (w == 64 && k > 1) return wait(true, of(mb_sd0, k - 2), phase(k - 2));
        } else {
            if (w == 64 && k > 0) return wait(true, of(mb_sd0, k - 1), phase(k - 1));
            if (w == 96 && k > 1) return wait(true, of(mb_xf0, k - 2), phase(k - 2));
        }
        return true;
    };

    if (warp >= kProducerWarp) take_registers<kRegsOne>();
    if (warp == kProducerWarp) {
        // the whole warp follows the loop, one elected lane issues: what the
        // MMAs take then stays in uniform registers.  (Rolled loops of MMAs: half
        // the instructions to fetch beside the other groups', 378 -> 364 us on 8
        // prompts of 4096 tokens.)
        const bool issuer = elect_one();
        const uint64_t dC = tc::smem_desc(sbase + kOffC, 16, 1024);    // K-major A
        const uint64_t dBk = tc::smem_desc(sbase + kOffBh, 16, 1024);  // K-major B (G)
        const uint64_t dS = tc::smem_desc(sbase + kOffBl, 16, 1024);   // K-major B (C S^T)
        constexpr uint32_t idG = tc::idesc_bf16(128, 128, 0, 0);
        constexpr uint32_t idS = tc::idesc_bf16(128, 128, 0, 1);
        constexpr uint32_t idC = tc::idesc_f16(128, 128, 0, 0);
        constexpr uint32_t idY = tc::idesc_f16(128, 64, 0, 0);
        loads.x = nk > 1 && kStateOnly ? 2 : nk > 0 ? 1 : 0;   // (in the set-up, maybe by another lane)
        loads.bc = kStateOnly ? 2 * loads.x : 3 * loads.x;
        bool ok = true;
        auto take = [&](uint32_t bar, uint32_t parity) { ok = wait(ok, bar, parity); };
        // a wait that gave up in one lane gives up in all
        auto all_ok = [&]() { return ok = __all_sync(0xffffffffu, ok); };
        auto koff = [](int ks) -> uint32_t { return (ks >> 2) * (kTile / 2) + (ks & 3) * 32; };   // K-major step
        auto issue_g = [&]() {
            if (issuer) {
#pragma unroll 1
                for (int ks = 0; ks < kN / 16; ++ks)
                    tc::mma_bf16(tmem + kColG, tc::desc_add(dC, koff(ks)), tc::desc_add(dBk, koff(ks)), idG, ks > 0);
                tc::mma_commit(mb_g);
            }
            __syncwarp();
        };
        if (!kStateOnly && nk > 0) {
            take(mb_bc, 0);
            if (all_ok()) {
                tc::fence_after_sync();
                issue_g();
            }
        }
        for (int k = 0; k < nk && ok; ++k) {
            const uint32_t par = k & 1;
            // (w o X)^T B: hi hi, lo hi, hi lo
            if (kStateOnly) {
                take(b_bar(k), phase(k));
            } else {
                take(mb_g, par);   // (G has read C: its fp16 form may come)
                if (!all_ok()) break;
                if (issuer) issue_c16(k);
            }
            take(mb_s, par);
            take(of(mb_w0, k), phase(k));
            if (!all_ok()) break;
            constexpr int ahead = kStateOnly ? 2 : 1;
            if (issuer && k + ahead < nk) issue_x(k + ahead);   // (the raw rows have been read)
            tc::fence_after_sync();
            if (issuer) {
                const uint64_t dBh = tc::smem_desc(sbase + bh_off(k), kTile / 2, 1024);   // MN-major B
                const uint64_t dBl = tc::smem_desc(sbase + bl_off(k), kTile / 2, 1024);
                const uint32_t w = tmem + kColW - (kStateOnly && (k & 1) ? kColW : 0u);
#pragma unroll 1
                for (int ks = 0; ks < kQ / 16; ++ks) {
                    tc::mma_bf16_tmemA(tmem + kColS, w + 8 * ks, tc::desc_add(dBh, ks * 2048), idS, ks > 0);
                    tc::mma_bf16_tmemA(tmem + kColS, w + 64 + 8 * ks, tc::desc_add(dBh, ks * 2048), idS, 1);
                    tc::mma_bf16_tmemA(tmem + kColS, w + 8 * ks, tc::desc_add(dBl, ks * 2048), idS, 1);
                }
                tc::mma_commit(of(mb_sd0, k));
            }
            __syncwarp();
            if constexpr (kStateOnly) {
                if (k + 2 < nk) {
                    take(of(mb_sd0, k), phase(k));
                    if (!all_ok()) break;
                    if (issuer) {
                        issue_bh(k + 2);
                        issue_bl(k + 2);
                    }
                }
            } else {
                if (k + 1 < nk) {
                    take(of(mb_sd0, k), phase(k));
                    if (!all_ok()) break;
                    if (issuer) issue_bh(k + 1);
                }
                // Y = C S^T once the copy of S is in the B lo tile and the last
                // chunk's rows are out of Y's columns
                take(mb_c16, par);
                take(mb_cs, par);
                if (k > 0) take(mb_st, (k - 1) & 1);
                if (!all_ok()) break;
                tc::fence_after_sync();
                if (issuer) {
#pragma unroll 1
                    for (int ks = 0; ks < kN / 16; ++ks)
                        tc::mma_bf16(tmem + kColY, tc::desc_add(dC, koff(ks)), tc::desc_add(dS, koff(ks)), idC, ks > 0);
                    tc::mma_commit(mb_yo);
                }
                __syncwarp();
                if (k + 1 < nk) {
                    take(mb_yo, par);
                    if (!all_ok()) break;
                    if (issuer) {
                        issue_c(k + 1);
                        issue_bl(k + 1);
                    }
                }
                take(mb_ys, par);
                take(mb_m, par);
                if (!all_ok()) break;
                tc::fence_after_sync();
                // Y_h += M_h X_h
                if (issuer) {
                    const uint64_t d0 = tc::smem_desc(sbase + xbuf(k), 16, 1024);
#pragma unroll 1
                    for (int ks = 0; ks < kQ / 16; ++ks) {
                        tc::mma_bf16_tmemA(tmem + kColY, tmem + kColG + 16 * ks, tc::desc_add(d0, koff(ks)), idY, 1);
                        tc::mma_bf16_tmemA(tmem + kColY + 64, tmem + kColG + 16 * ks + 8,
                                           tc::desc_add(d0, koff(ks) + 64 * 128), idY, 1);
                    }
                    tc::mma_commit(mb_e);
                }
                __syncwarp();
                if (k + 1 < nk) {
                    take(mb_e, par);
                    take(mb_bc, (k + 1) & 1);
                    if (!all_ok()) break;
                    tc::fence_after_sync();
                    issue_g();
                }
            }
        }
        if (!ok) {
            // what this warp has under way ends before the CTA does: shared memory
            // and tensor memory are another's then.  (The B and C tiles of a chunk
            // share a phase: the arrivals of those not requested yet are given to it.)
            if (issuer) {
                record_error(p.status, kStatusTimeout);
                tc::mma_commit(mb_end);
                mbar_wait(mb_end, 0);
                if constexpr (kStateOnly) {
                    for (uint32_t b = 0; b < 2; ++b) {
                        if (loads.x > b) mbar_wait(x_bar(loads.x - 1 - b), phase(loads.x - 1 - b));
                        if (loads.bc > 2 * b) mbar_wait(b_bar(loads.bc / 2 - 1 - b), phase(loads.bc / 2 - 1 - b));
                    }
                } else {
                    for (; loads.bc % 3 != 0; ++loads.bc) tc::mbar_arrive(mb_bc);
                    if (loads.x > 0) mbar_wait(mb_x, (loads.x - 1) & 1);
                    if (loads.bc > 0) mbar_wait(mb_bc, (loads.bc / 3 - 1) & 1);
                    if (loads.c16 > 0) mbar_wait(mb_c16, (loads.c16 - 1) & 1);
                }
            }
        }
        __syncwarp();
    } else if (warp == kHelperWarp) {
        // Slots 4 lane .. 4 lane + 3, one head after the other, all in registers:
        // the first head's factors are there when their buffer comes free.
        bool ok = true;
        for (int k = 0; k < nk && ok; ++k) {
            const int b = k & 1;
            uint32_t b_exp = 0u, c_exp = 0u;
            if constexpr (!kStateOnly) {
                b_exp = *reinterpret_cast<const uint32_t *>(p.b_exp + (size_t)(wk.act + k) * kQ + 4 * lane);
                c_exp = *reinterpret_cast<const uint32_t *>(p.c_exp + (size_t)(wk.act + k) * kQ + 4 * lane);
            }
            // |B[s, n]| < 2^(its b_exp - 126), and for all s of the chunk
            const uint32_t b_top = __reduce_max_sync(0xffffffffu, __vmaxu4(__vmaxu4(b_exp, b_exp >> 16), __vmaxu4(b_exp, b_exp >> 16) >> 8) & 255u);
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const uint4 src = *(reinterpret_cast<const uint4 *>(sm + kOffDtBuf) + b * (kQ / 4) + lane);
                const uint32_t up = h ? 0u : 16u;   // (head 0 in the lower halves)
                const float d[4] = {__uint_as_float((src.x << up) & 0xffff0000u), __uint_as_float((src.y << up) & 0xffff0000u),
                                    __uint_as_float((src.z << up) & 0xffff0000u), __uint_as_float((src.w << up) & 0xffff0000u)};
                // prefix sums c and, for w, suffix sums c_last - c (from the end, so
                // that the factors that matter, near the end, come from short sums;
                // shifted between lanes, not subtracted: a lane's own may be large)
                const float Aw = h ? A1 : A0;
                const float x0 = d[0] * Aw, x1 = d[1] * Aw, x2 = d[2] * Aw, x3 = d[3] * Aw;
                float pre = (x0 + x1) + (x2 + x3), suf = pre;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float u = __shfl_up_sync(0xffffffffu, pre, o);
                    const float v = __shfl_down_sync(0xffffffffu, suf, o);
                    if (lane >= o) pre += u;
                    if (lane + o < 32) suf += v;
                }
                const float all = __shfl_sync(0xffffffffu, suf, 0);
                pre = __shfl_up_sync(0xffffffffu, pre, 1);
                suf = __shfl_down_sync(0xffffffffu, suf, 1);
                if (lane == 0) pre = 0.0f;
                if (lane == 31) suf = 0.0f;
                const float c[4] = {pre + x0, (pre + x0) + x1, ((pre + x0) + x1) + x2, (((pre + x0) + x1) + x2) + x3};
                float w[4] = {((suf + x3) + x2) + x1, (suf + x3) + x2, suf + x3, suf};
                const float cR = __shfl_sync(0xffffffffu, c[3], lane | 7);   // end of the 32-slot block
                [[maybe_unused]] float unit[4];
                if constexpr (!kStateOnly) {
                    // A row's unit: the power of two that takes a bound of M[t, s] to
                    // 2^13..2^14.  |G[t, s]| <= 128 max |C_t| max |B_s|; in log2, with the
                    // decay, over all s <= t: max(log2 |B_s| dt_s - c_s) + c_t + log2 128
                    // |C_t|; and D.  (So a token's infinity or large value leaves the rows
                    // before it alone.)
                    float q = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        q = fmaxf(q, static_cast<float>(b_exp >> 8 * i & 255u) + log2_approx(fabsf(d[i])) - c[i]);
                        unit[i] = q;
                    }
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const float u = __shfl_up_sync(0xffffffffu, q, o);
                        if (lane >= o) q = fmaxf(q, u);
                    }
                    q = __shfl_up_sync(0xffffffffu, q, 1);
                    if (lane == 0) q = -INFINITY;
                    const float lD = log2_approx(fabsf(biases[kPP + h]));
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float e = fmaxf(fmaxf(q, unit[i]) + c[i] + static_cast<float>(c_exp >> 8 * i & 255u) + (7.0f + 14.0f - 2 * 126.0f), lD);
                        unit[i] = __int_as_float((127 + static_cast<int>(fmaxf(fminf(floorf(13.0f - e), 20.0f), -36.0f))) << 23);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[i] = tc::exp2_approx(w[i]) * (d[i] * (1.0f / kXUnit));
                }
                // |what the chunk adds to the state| <= sum of w |x| |B|
                [[maybe_unused]] float sum = (fabsf(w[0]) + fabsf(w[1])) + (fabsf(w[2]) + fabsf(w[3]));
                if constexpr (!kStateOnly) {
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                }
                // exp(c_last) S as S f + (S or 0): f = exp - 1 for slow decays
                const float f = all > -1.0f ? expm1f(all * kLn2) : exp2f(all);
                if (h == 0 && k >= 2) {
                    if (lane == 0) ok = mbar_wait(mb_free0 + 8 * b, ((k >> 1) - 1) & 1);
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                }
                const int e = (b * 2 + h) * kQ + 4 * lane;
                *reinterpret_cast<float4 *>(wgt + e) = make_float4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<float4 *>(cum + e) = make_float4(c[0], c[1], c[2], c[3]);
                if (lane == 0) scl[b * 2 + h] = make_float2(f, all);
                if constexpr (!kStateOnly) {
                    *reinterpret_cast<float4 *>(dts + e) = make_float4(d[0], d[1], d[2], d[3]);
                    *reinterpret_cast<float4 *>(fB + e) = make_float4(tc::exp2_approx(cR - c[0]) * d[0], tc::exp2_approx(cR - c[1]) * d[1],
                                                                      tc::exp2_approx(cR - c[2]) * d[2], tc::exp2_approx(cR - c[3]) * d[3]);
                    *reinterpret_cast<float4 *>(f4 + e) = make_float4(tc::exp2_approx(c[3] - c[0]) * d[0], tc::exp2_approx(c[3] - c[1]) * d[1],
                                                                      tc::exp2_approx(c[3] - c[2]) * d[2], d[3]);
                    *reinterpret_cast<float4 *>(reinterpret_cast<float *>(sm + kOffMUnit) + e) = make_float4(unit[0], unit[1], unit[2], unit[3]);
                    if (lane == 0)
                        reinterpret_cast<float *>(sm + kOffGrow)[2 * b + h] =
                            1.01f * kXUnit * sum * __uint_as_float(min(b_top + 1u, 254u) << 23);
                    if (h == 0) *reinterpret_cast<uint32_t *>(sm + kOffCExp + b * kQ + 4 * lane) = c_exp;
                }
            }
            if (!ok) break;
            if (k + 2 < nk) load_dt_async(k + 2);
            tc::mbar_arrive(mb_dt0 + 8 * b);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (lane == 0 && !ok) record_error(p.status, kStatusTimeout);
    } else if (warp == kPublisherWarp) {
        if constexpr (!kStateOnly) {
            bool ok = true;
            for (int k = 0; k < nk; ++k) {
                if (lane == 0) ok = mbar_wait(mb_st, k & 1);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                const int cnt = tokens(k), row = first_row(k);
                if (cnt == kQ) {
                    if (lane == 0) {
                        const uint32_t st = sbase + xbuf(k);
                        tc::tma_store_3d(&tm_y, st, hp * kPP, row, 0);
                        tc::tma_store_3d(&tm_y, st + kTile / 2, hp * kPP + kP, row, 0);
                        tc::bulk_commit();
                        tc::bulk_wait_read0();   // the rows have been read
                        tc::mbar_arrive(of(mb_xf0, k));
                    }
                } else {
                    // the prompt's end (always its walk's last chunk): its rows
                    // only, 16 bytes a lane; the next rows are another prompt's
                    const uint8_t *box = sm + xbuf(k);
                    for (int e = lane; e < cnt * 16; e += 32) {
                        const int r = e >> 4, h = (e >> 3) & 1, piece = e & 7;
                        *reinterpret_cast<uint4 *>(p.y + (size_t)(row + r) * H * kP + hp * kPP + h * kP + piece * 8) =
                            *reinterpret_cast<const uint4 *>(box + h * (kTile / 2) + tc::sw128(r, piece));
                    }
                }
            }
            if (lane == 0) {
                tc::bulk_wait0();
                if (!ok) record_error(p.status, kStatusTimeout);
            }
            __syncwarp();
        }
    } else if (warp < kYWarp) {
        // ================= M group, in place over G: the 16 G columns of unit
        // U (tokens 16 U .. 16 U + 15) become [M_0 | M_1] (8 columns of bf16
        // pairs each).  Thread: row t, both heads; the two warps h of a
        // quarter's rows share its units: the `quad` units h quad ..
        // h quad + quad - 1 below its diagonal block and unit 2 quad + h of
        // that block (past it: zeros).
        // Between two Ms, while G is made: its share of the next chunk's conv.
        take_registers<kRegsM>();
        const int h = warp >> 2, quad = warp & 3, row = tid & 127;
        const uint32_t gcol = tmem + (static_cast<uint32_t>(32 * quad) << 16) + kColG;
        bool ok = true;
        for (int k = -1; k < nk; ++k) {
            if (!kStateOnly && k >= 0) {
                const int par = k & 1;
                ok = grp_and<kMGroup>(1, tid != 0 || wait(true, mb_g, par));
                if (!ok) break;
                tc::fence_after_sync();
                const float *c0 = cum + 2 * par * kQ;   // this chunk's factors, head 0 (head 1: + kQ)
                uint32_t g[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) g[i] = 0u;
#pragma unroll 1
                for (int U = 2 * quad + 2 + h; U < 8; U += 2) tc::tmem_st16_nw(gcol + 16 * U, g);
#pragma unroll 1
                for (int i = 0; i < quad; ++i) {
                    // below the diagonal block: exp(c_t - c_R) exp(c_R - c_s), both <= 1
                    const int U = h * quad + i;
                    tc::tmem_ld16_nw(gcol + 16 * U, g);
                    tc::tmem_wait_ld16(g);
#pragma unroll 1
                    for (int hd = 0; hd < 2; ++hd) {
                        const float *cm = c0 + hd * kQ;
                        const float et = tc::exp2_approx(cm[row] - cm[16 * U | 31]) * cm[(kOffMUnit - kOffCum) / 4 + row];
                        const float2 et2 = make_float2(et, et);
                        const float4 *fb = reinterpret_cast<const float4 *>(cm + (kOffFB - kOffCum) / 4 + 16 * U);
                        uint32_t out[8];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 f = fb[j];
                            const float2 a = tc::mul2(tc::mul2(make_float2(__uint_as_float(g[4 * j]), __uint_as_float(g[4 * j + 1])), et2),
                                                      make_float2(f.x, f.y));
                            const float2 b = tc::mul2(tc::mul2(make_float2(__uint_as_float(g[4 * j + 2]), __uint_as_float(g[4 * j + 3])), et2),
                                                      make_float2(f.z, f.w));
                            out[2 * j] = pack_f16x2(a.x, a.y);
                            out[2 * j + 1] = pack_f16x2(b.x, b.y);
                        }
                        tc::tmem_st8_nw(gcol + 16 * U + 8 * hd, out);
                    }
                }
                tc::tmem_ld16_nw(gcol + 16 * (2 * quad + h), g);
                tc::tmem_wait_ld16(g);
                // the diagonal block's unit: column s = 16 h + i against row r of the block
                const int r = (row & 31) - 16 * h;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (i > r) g[i] = 0u;
#pragma unroll 1
                for (int hd = 0; hd < 2; ++hd) {
                    const float *cb = c0 + hd * kQ + 32 * quad;   // the block's
                    const float *cm = cb + 16 * h;                // the unit's
                    const float ct = cb[row & 31], unit = cb[(kOffMUnit - kOffCum) / 4 + (row & 31)], Dh = unit * biases[kPP + hd];
                    uint32_t out[8];
                    if (cb[0] - cb[31] <= 60.0f) {   // warp-uniform
                        // through 4-token blocks: exp(c_t - c_R4) exp(c_R4 - c_s);
                        // with the whole block's decay at most 2^60 the row
                        // factor (>= 1 inside t's own) is finite
                        const float4 *f4h = reinterpret_cast<const float4 *>(cm + (kOffF4 - kOffCum) / 4);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float rf = unit * tc::exp2_approx(ct - cm[4 * j + 3]);
                            const float2 rf2 = make_float2(rf, rf);
                            const float4 f = f4h[j];
                            const float2 a = tc::fma2(tc::mul2(make_float2(__uint_as_float(g[4 * j]), __uint_as_float(g[4 * j + 1])), rf2),
                                                      make_float2(f.x, f.y),
                                                      make_float2(4 * j == r ? Dh : 0.0f, 4 * j + 1 == r ? Dh : 0.0f));
                            const float2 b = tc::fma2(tc::mul2(make_float2(__uint_as_float(g[4 * j + 2]), __uint_as_float(g[4 * j + 3])), rf2),
                                                      make_float2(f.z, f.w),
                                                      make_float2(4 * j + 2 == r ? Dh : 0.0f, 4 * j + 3 == r ? Dh : 0.0f));
                            out[2 * j] = pack_f16x2(a.x, a.y);
                            out[2 * j + 1] = pack_f16x2(b.x, b.y);
                        }
                    } else {
                        // steep decays (or a dt that is not finite, whose
                        // factors must not meet the zeros): one exponential per
                        // element, each <= 1
                        const float *dh = cm + (kOffDt - kOffCum) / 4;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float v[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int i = 2 * j + e;
                                const float ex = unit * tc::exp2_approx(fminf(ct - cm[i], 0.0f));
                                const float x = fmaf(__uint_as_float(g[i]) * ex, dh[i], i == r ? Dh : 0.0f);
                                v[e] = i <= r ? x : 0.0f;
                            }
                            out[j] = pack_f16x2(v[0], v[1]);
                        }
                    }
                    tc::tmem_st8_nw(gcol + 16 * (2 * quad + h) + 8 * hd, out);
                }
                tc::tmem_wait_st();
                tc::fence_before_sync();
                grp_sync<kMGroup>(1);
                if (tid == 0) {
                    tc::mbar_arrive(mb_m);
                    tc::mbar_arrive(of(mb_free0, k));
                }
            }
            if (k + 1 < nk) {
                ok = grp_and<kMGroup>(1, x_ready(k + 1, 0));
                if (!ok) break;
                tc::fence_after_sync();
                const bool off = grp_or<kMGroup>(1, conv_units(k + 1, row, 12 + 2 * h, 14 + 2 * h, 3 + h));
                if (tid == 0) {
                    if constexpr (!kStateOnly) {
                        *reinterpret_cast<int *>(sm + kOffMOff) = off;
                        tc::mbar_arrive(mb_mc);
                    }
                    tc::mbar_arrive(of(mb_w0, k + 1));
                    if (kStateOnly) tc::mbar_arrive(of(mb_free0, k + 1));
                }
            }
        }
        if (!ok && tid == 0) record_error(p.status, kStatusTimeout);
    } else if (warp < kXWarp) {
        // ================= Y group.  State: thread (p' = row, half of n), its
        // 64 values in registers.  Rows: thread (t = row, head).
        take_registers<kRegsY>();
        const int tb = tid - 32 * kYWarp;
        const int hf = tb >> 7, quad = warp & 3;
        const uint32_t lane_base = static_cast<uint32_t>(32 * quad) << 16;
        const int prow = tb & 127;
        // this thread's values of the pair's state, [head][p][n] in memory
        const size_t pair_off = (size_t)hp * kPP * kN + (size_t)prow * kN + 64 * hf;
        const uint32_t scol = tmem + lane_base + kColS + 64 * hf;
        float2 st[32];
        {
            const float *from = nullptr;
            if (!kStateOnly) {
                if (wk.slot >= 0)
                    from = p.seg_state + (size_t)wk.slot * H * kP * kN + pair_off;
                else if (resume)
                    from = p.state + (size_t)slot * H * kP * kN + pair_off;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float4 v = from ? *reinterpret_cast<const float4 *>(from + 4 * i)
                                      : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                st[2 * i] = make_float2(v.x, v.y);
                st[2 * i + 1] = make_float2(v.z, v.w);
            }
        }
        float dec = 0.0f;   // state-only: log2 of the walk's decay (this thread's head)
        // Bounds of the magnitudes of this thread's row of the state and of its
        // head's, for copy_state: found here, then carried over a chunk with what it
        // can add: sum of w, times the largest |B|, times the row's largest |x| (a
        // bound that is too large only costs some of fp16's 29 octaves of full
        // precision: 8 or so, and 2 more over the chunks between two findings).
        float row_most = 0.0f, head_most = 0.0f;
        auto find_bounds = [&]() {
            uint32_t *rmax = reinterpret_cast<uint32_t *>(sm + kOffSMax);
            uint32_t *wmax = reinterpret_cast<uint32_t *>(sm + kOffWMax) + 4 * (quad >> 1);
            float big = 0.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i) big = max_abs3(big, st[i].x, st[i].y);
            const uint32_t all = __reduce_max_sync(0xffffffffu, big <= kFltMax ? __float_as_uint(big) : 0u);
            rmax[hf * kPP + prow] = __float_as_uint(big);
            if (lane == 0) wmax[2 * hf + (quad & 1)] = all;
            grp_sync<kYGroup>(2);
            row_most = __uint_as_float(max(rmax[prow], rmax[kPP + prow]));
            head_most = __uint_as_float(max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3])));
        };
        // S <- exp(c_last) S + chunk k's products
        auto next_state = [&](int k) {
            const float2 f = scl[(k & 1) * 2 + (quad >> 1)];
            const bool slow = f.y > -1.0f;
            const float2 f2 = make_float2(f.x, f.x), zero = make_float2(0.0f, 0.0f), one = make_float2(1.0f, 1.0f);
            if constexpr (kStateOnly) dec += f.y;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t r[16];
                tc::tmem_ld16_nw(scol + 16 * q, r);
                tc::tmem_wait_ld16(r);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float2 &v = st[8 * q + i];
                    v = tc::fma2(v, f2, slow ? v : zero);
                    v = tc::fma2(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), one, v);
                }
            }
        };
        // the fp16 copy of the state (operand of C S^T), times a power of two
        // whose inverse C S^T is multiplied by: one for the head, and for rows
        // whose largest value is below 2^-16 of its (or above 2^60) their own, which
        // (rare) takes another pass over C S^T's columns (8 prompts of 4096 tokens,
        // such rows in every head and chunk: 464 us for 380)
        float *colf = reinterpret_cast<float *>(sm + kOffColF), *headf = reinterpret_cast<float *>(sm + kOffHeadF);
        int *rowwise = reinterpret_cast<int *>(sm + kOffRowwise);   // [head]: last chunk + 1 with such rows
        float copy_scale = 1.0f;
        auto choose_scale = [&](int k) {   // for chunk k's
            const uint32_t head = min(max(__float_as_uint(head_most) >> 23, kLeastExp), kMostExp);
            uint32_t row = __float_as_uint(row_most) >> 23;
            const bool own = row < 255u && (row > head || (row + 16u < head && row >= kLeastExp));
            row = own ? max(row + 120u, head) - 120u : head;
            if (hf == 0) {
                colf[prow] = __uint_as_float((row + 127u - head) << 23);
                if (own) rowwise[quad >> 1] = k + 1;
                if (lane == 0) headf[quad >> 1] = __uint_as_float(fp16_unscale_exp(head) << 23);
            }
            copy_scale = fp16_scale(row);
        };
        auto copy_state = [&]() {
            const float2 s2 = make_float2(copy_scale, copy_scale);
#pragma unroll
            for (int pc = 0; pc < 8; ++pc) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = tc::mul2(st[4 * pc + i], s2);
                    w[i] = pack_f16x2(v.x, v.y);
                }
                *reinterpret_cast<uint4 *>(sm + kOffBl + hf * (kTile / 2) + tc::sw128(prow, pc)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        };
        const uint32_t ycol = tmem + lane_base + kColY + 64 * hf;
        // a row's factor (asked for before the wait for C S^T)
        auto row_factor = [&](int k, float unit) {
            return tc::exp2_approx(cum[((k & 1) * 2 + hf) * kQ + prow]) * unit * headf[hf] *
                   __uint_as_float((uint32_t)sm[kOffCExp + (k & 1) * kQ + prow] << 23);
        };
        auto scale_rows = [&](int k, float et) {
            const float2 et2 = make_float2(et, et);
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                uint32_t r[16];
                tc::tmem_ld16_nw(ycol + 16 * q, r);
                tc::tmem_wait_ld16(r);
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float2 o = tc::mul2(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), et2);
                    r[i] = __float_as_uint(o.x);
                    r[i + 1] = __float_as_uint(o.y);
                }
                tc::tmem_st16_nw(ycol + 16 * q, r);
            }
            const bool own_x = any_bad[2 + (k & 1)] != 0;
            if (rowwise[hf] == k + 1 || own_x) {   // (rare)
                tc::tmem_wait_st();
                const float *f = xfac + (k & 1) * kPP + 64 * hf;
#pragma unroll 1
                for (int c = 0; c < 64; c += 4) {
                    uint32_t r[4];
                    tmem_ld4(ycol + c, r);
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * colf[64 * hf + c + i] * (own_x ? f[c + i] : 1.0f));
                    tmem_st4_nw(ycol + c, r);
                }
            }
        };
        // chunk k's rows as two TMA store boxes (one per head: 128-byte rows,
        // 16-byte piece j of row t at j ^ (t & 7)) in its x buffer
        auto stage_rows = [&](int k, float unit) {
            const int row = tc::no_hoist(prow);
            uint8_t *box = sm + xbuf(k) + hf * (kTile / 2);
            const float one = __uint_as_float(0x7f000000u - __float_as_uint(unit));   // 1 / unit
            if (any_bad[2 + (k & 1)]) {   // (rare)
                const float *f = xfac + (k & 1) * kPP + 64 * hf;
#pragma unroll 1
                for (int c = 0; c < 64; c += 4) {
                    uint32_t r[4];
                    tmem_ld4(ycol + c, r);
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * __uint_as_float(0x7f000000u - __float_as_uint(f[c + i])));
                    tmem_st4_nw(ycol + c, r);
                }
                tc::tmem_wait_st();
            }
            const bool bad = any_bad[k & 1] != 0;   // (rare: see the top)
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                uint32_t r[16];
                tc::tmem_ld16_nw(ycol + 16 * q, r);
                tc::tmem_wait_ld16(r);
                if (bad) {
                    const uint8_t *b = bad_at + (k & 1) * 3 * kPP + 64 * hf + 16 * q;
#pragma unroll 1
                    for (int part = 0; part < 3; ++part)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (row >= b[part * kPP + i]) r[i] = 0x7fffffffu;
                }
#pragma unroll
                for (int pc = 0; pc < 2; ++pc) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 v = tc::mul2(make_float2(__uint_as_float(r[8 * pc + 2 * i]), __uint_as_float(r[8 * pc + 2 * i + 1])),
                                                  make_float2(one, one));
                        w[i] = tc::pack_bf16x2(v.x, v.y);
                    }
                    *reinterpret_cast<uint4 *>(box + tc::sw128(row, 2 * q + pc)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        };
        bool ok = true;
        if constexpr (!kStateOnly) {
            find_bounds();
            choose_scale(0);
        }
        if (tb == 0) tc::mbar_arrive(mb_s);   // chunk 0's products may start
        for (int k = 0; k < nk; ++k) {
            const int par = k & 1;
            // the products done: kColS, and the B lo tile is free
            ok = grp_and<kYGroup>(2, tb != 0 || wait(wait(true, of(mb_dt0, k), phase(k)), of(mb_sd0, k), phase(k)));
            if (!ok) break;
            tc::fence_after_sync();
            if constexpr (!kStateOnly) {
                copy_state();
                tc::fence_proxy_async();   // the copy, for the tensor core
                grp_sync<kYGroup>(2);
                if (tb == 0) tc::mbar_arrive(mb_cs);
            }
            next_state(k);
            tc::fence_before_sync();   // the reads of kColS before the next products
            grp_sync<kYGroup>(2);
            if (tb == 0) {
                tc::mbar_arrive(mb_s);
                if (kStateOnly) tc::mbar_arrive(of(mb_free0, k));
            }
            if constexpr (!kStateOnly) {
                // what M X's row is multiplied by (read here: from mb_free0 on it is the next but one's)
                const float unit = kXUnit * cum[(kOffMUnit - kOffCum) / 4 + (2 * par + hf) * kQ + prow];
                const float et = row_factor(k, unit);
                // what is left of the state's bounds after the chunk, and what it adds
                const float2 f = scl[par * 2 + (quad >> 1)];
                const float keep = f.y > -1.0f ? 1.0f + f.x : f.x;
                const float grow = reinterpret_cast<const float *>(sm + kOffGrow)[2 * par + (quad >> 1)];
                const float more = grow * reinterpret_cast<const float *>(sm + kOffXMost)[2 * par + (quad >> 1)];
                const uint16_t *xr = reinterpret_cast<const uint16_t *>(sm + kOffXRow) + par * kParts * kPP + prow;
                const uint32_t x_row = max(max(max((uint32_t)xr[0], (uint32_t)xr[kPP]), (uint32_t)xr[2 * kPP]), max((uint32_t)xr[3 * kPP], (uint32_t)xr[4 * kPP]));
                float more_row = grow * ((1.0f / kXUnit) * __half2float(__ushort_as_half((uint16_t)min(x_row, 0x7bffu))));
                if (any_bad[2 + par] && xfac[par * kPP + prow] != 1.0f)   // (rare)
                    more_row = grow * ((65504.0f / kXUnit) * __uint_as_float(0x7f000000u - __float_as_uint(xfac[par * kPP + prow])));
                ok = grp_and<kYGroup>(2, tb != 0 || wait(true, mb_yo, par));
                if (!ok) break;
                tc::fence_after_sync();
                scale_rows(k, et);
                tc::tmem_wait_st();
                tc::fence_before_sync();
                grp_sync<kYGroup>(2);
                if (tb == 0) {
                    tc::mbar_arrive(mb_ys);
                    tc::mbar_arrive(of(mb_free0, k));
                }
                // (here, while M X is made)
                if ((k & 15) == 15) {
                    find_bounds();
                } else {
                    row_most = fmaf(row_most, keep, more_row);
                    head_most = fmaf(head_most, keep, more);
                }
                ok = grp_and<kYGroup>(2, tb != 0 || wait(true, mb_e, par));
                if (!ok) break;
                tc::fence_after_sync();
                choose_scale(k + 1);
                stage_rows(k, unit);
                tc::fence_proxy_async();   // the rows, for the TMA store
                tc::fence_before_sync();   // TMEM reads before the next product writes
                grp_sync<kYGroup>(2);
                if (tb == 0) tc::mbar_arrive(mb_st);
            }
        }
        // the state after the walk (an empty prompt that resumes keeps its
        // entry).  Its place is looked up again: not a register is spared for
        // it through the loop.
        const Walk end = p.walks[blockIdx.x / HP];
        if (ok && (kStateOnly || end.last) && (nk > 0 || !end.resume)) {
            // through the B and C tiles, which nothing reads or loads any
            // more, and 512-byte copies (a thread's own 16-byte stores, 512
            // bytes apart in a warp, took 4 us)
            uint8_t *rows = sm + kOffC + prow * kStateRow;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                *reinterpret_cast<float4 *>(rows + 256 * hf + 16 * i) =
                    make_float4(st[2 * i].x, st[2 * i].y, st[2 * i + 1].x, st[2 * i + 1].y);
            tc::fence_proxy_async();
            grp_sync<kYGroup>(2);
            if (hf == 0) {
                float *to = (kStateOnly ? p.seg_state + (size_t)(end.slot + 1) * H * kP * kN
                                        : p.state + (size_t)end.entry * H * kP * kN) +
                            (size_t)hp * kPP * kN + (size_t)prow * kN;
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                             ::"l"(to), "r"(tc::smem_u32(rows)), "n"(kN * 4) : "memory");
                tc::bulk_commit();
                tc::bulk_wait_read0();   // (shared memory must outlive the reads; the grid's end the writes)
                if (kStateOnly && (prow & 63) == 0)
                    p.seg_dec[(size_t)(end.slot + 1) * H + 2 * hp + (prow >> 6)] = dec;
            }
        }
        if (!ok && tb == 0) record_error(p.status, kStatusTimeout);
    } else if (warp < kProducerWarp) {
        // ================= X group: thread (channel p' = lane of its quarter,
        // a third of the tokens)
        take_registers<kRegsX>();
        const int tx = tid - 32 * kXWarp;
        const int third = tx >> 7, pr = tx & 127;   // units 4 third .. 4 third + 3
        bool ok = true;
        for (int k = 0; k < nk; ++k) {
            ok = grp_and<kXGroup>(3, x_ready(k, 32 * kXWarp));
            if (!ok) break;
            tc::fence_after_sync();
            const bool off = grp_or<kXGroup>(3, conv_units(k, pr, 4 * third, 4 * third + 4, third));
            if constexpr (kStateOnly) {
                if (tx == 0) {
                    tc::mbar_arrive(of(mb_w0, k));
                    tc::mbar_arrive(of(mb_free0, k));
                }
            } else {
                volatile int *again = reinterpret_cast<volatile int *>(sm + kOffAgain);
                if (tx == 0) {
                    // whether X^T's values, the M group's too, are finite and fit kXUnit
                    const int par = k & 1;
                    any_bad[par] = any_bad[2 + par] = 0;
                    ok = wait(true, mb_mc, par);
                    volatile uint32_t *xh = reinterpret_cast<volatile uint32_t *>(sm + kOffXHead) + 2 * par;
                    const uint32_t x0 = xh[0], x1 = xh[1];
                    xh[0] = xh[1] = 0u;
                    auto small = [](uint32_t x) { return x - 1u < 0x0c00u - 1u; };   // (below 2^-12, not 0)
                    const bool other = off || *reinterpret_cast<volatile int *>(sm + kOffMOff) != 0 || small(x0) || small(x1);
                    float *xm = reinterpret_cast<float *>(sm + kOffXMost) + 2 * par;
                    xm[0] = other ? 0.0f : __half2float(__ushort_as_half((uint16_t)x0)) * (1.0f / kXUnit);
                    xm[1] = other ? 0.0f : __half2float(__ushort_as_half((uint16_t)x1)) * (1.0f / kXUnit);
                    if (!other) {
                        tc::mbar_arrive(of(mb_w0, k));
                        tc::mbar_arrive(of(mb_free0, k));
                    }
                    *again = other;
                }
                ok = grp_and<kXGroup>(3, ok);
                if (!ok) break;
                if (*again) {
                    repair(k, third, pr);
                    if (tx == 0) {
                        tc::mbar_arrive(of(mb_w0, k));
                        tc::mbar_arrive(of(mb_free0, k));
                    }
                }
            }
        }
        if (!ok && tx == 0) record_error(p.status, kStatusTimeout);
    }
    if constexpr (!kStateOnly) {
        // the new tail: by the prompt's first walk (the only one that read the
        // old x channels, in its set-up; the old B and C channels were read by
        // the prep kernel)
        if (starts && warp == kTailWarp) {
            const Walk end = p.walks[blockIdx.x / HP];
            const bool again = end.resume != 0;
            const int from = end.begin, n = end.len;
            __nv_bfloat16 *entry = p.tail + (size_t)end.entry * 4 * ch;
            auto commit = [&](int cc) {
                __nv_bfloat16 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = n - 4 + i;
                    v[i] = t >= 0 ? p.xbc[(size_t)(from + t) * ch + cc]
                                  : again ? entry[(size_t)(4 + t) * ch + cc] : __float2bfloat16_rn(0.0f);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) entry[(size_t)i * ch + cc] = v[i];
            };
#pragma unroll 1
            for (int i = lane; i < kPP + (hp == 0 ? 2 * kN : 0); i += 32) commit(i < kPP ? hp * kPP + i : H * kP + i - kPP);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

bool prompt_tc_supported(const bimamba_dims &d)
{
    return d.dtype == BIMAMBA_BF16 && d.headdim == kP && d.d_state == kN && d.ngroups == 1 && d.d_conv == 4 &&
           d.heads % 2 == 0;
}

namespace {

constexpr int kSMs = 148;

struct Layout {
    int max_chunks, cut_over, seg_chunks, max_inner, max_walks, max_slots, max_cuts;
    size_t head, walks, cuts, act, b_exp, c_exp, dec, state, bytes;
};

// How prompts are cut.  The pieces are as long as is best for one prompt of
// all the rows: n pieces take ceil(n pairs / SMs) rounds of a piece's chunks
// and about 3 chunks' time to begin and end, after state-only walks of the
// first n - 1 at half of that.  A prompt is cut once its walk would take
// longer than these do: a piece's state-only walk, three chunks' time for two
// more launches, and the GPU's share of the call (a fifth added: walks do not
// fill it evenly).  1311, 1, 640, 129, 0, 2777, 63, 1024, 517, 1536 and 128
// tokens in 64 heads: 138 us, with the 2777 in two pieces 166.  (The host knows
// the rows that there is room for, not the prompts' lengths: a call with room for
// many rows does not cut a prompt that few of them make.)
void cut_of(long long chunks, int pairs, int &cut_over, int &seg_chunks)
{
    const long long share = (chunks * pairs + kSMs - 1) / kSMs;
    long long best = 1ll << 60, piece = chunks;
    for (long long n = 2; n <= 16 && n <= chunks; ++n) {
        const long long seg = (chunks + n - 1) / n;
        const long long cost = (seg + 3) * (2 * ((n * pairs + kSMs - 1) / kSMs) + ((n - 1) * pairs + kSMs - 1) / kSMs);
        if (cost < best) {
            best = cost;
            piece = seg;
        }
    }
    cut_over = (int)(std::max(piece, (share * 6 + 4) / 5) + piece / 2 + 3);
    seg_chunks = (int)std::max<long long>(1, std::min<long long>(piece, cut_over));
}

// Sizes that hold for any lengths of `batch` prompts in `len` rows.  A prompt of
// L tokens has at most (L - 1) / 128 + 1 chunks.  Only prompts of more than
// cut_over are cut, and one of c chunks into at most (c - 1) / seg_chunks + 1
// pieces: their number goes by the rows, not by the other prompts.
// `fewer`: that fit calls of fewer rows, too, for which the rule may cut more
// (14976 rows in 64 heads take 6 pieces, 15104 take 4).  Every count of chunks
// is tried up to kTried (a millisecond, in the size query alone); of more, a
// piece has a 16th of the rows at least and a prompt that is cut 1.5 of that,
// so that there are at most 16 and 10.
Layout layout_of(const bimamba_dims &d, bool fewer)
{
    Layout l{};
    const long long chunks = (long long)d.len / kQ + std::min(d.batch, d.len);
    l.max_chunks = (int)chunks;
    auto cuts_of = [&](long long rows) {
        cut_of(rows / kQ, d.heads / 2, l.cut_over, l.seg_chunks);
        const int cuts = (int)std::min<long long>(d.batch, rows / (l.cut_over * (long long)kQ + 1));
        l.max_cuts = std::max(l.max_cuts, cuts);
        if (cuts > 0) l.max_inner = std::max(l.max_inner, (int)(rows / kQ / l.seg_chunks));
    };
    if (fewer) {
        constexpr int kTried = 4096;
        for (int c = std::min(d.len / kQ, kTried); c >= 0; --c) cuts_of((long long)c * kQ + kQ - 1);
        if (d.len / kQ > kTried) {
            l.max_cuts = std::max(l.max_cuts, std::min(d.batch, 10));
            l.max_inner = std::max(l.max_inner, 16);
        }
    } else {
        cuts_of(d.len);
    }
    l.max_walks = l.max_inner + d.batch;
    l.max_slots = l.max_inner + l.max_cuts;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) & ~(size_t)255;
        return here;
    };
    l.head = take(sizeof(PlanHeader));
    l.walks = take(sizeof(Walk) * (size_t)l.max_walks);
    l.cuts = take(sizeof(int4) * (size_t)l.max_cuts);
    l.act = take((size_t)l.max_chunks * kQ * kAct * 2);
    l.b_exp = take((size_t)l.max_chunks * kQ);
    l.c_exp = take((size_t)l.max_chunks * kQ);
    l.dec = take((size_t)l.max_slots * d.heads * 4);
    l.state = take((size_t)l.max_slots * d.heads * kP * kN * 4);
    l.bytes = at;
    return l;
}

// 3-D bf16 tensor map over a (rows, cols) matrix: boxes of box0 columns x box1 rows.
bool make_map(CUtensorMap *m, const void *base, uint64_t cols, uint64_t rows, uint32_t box0, uint32_t box1,
              bool swizzle)
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        cudaDriverEntryPointQueryResult q;
        void *f = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return false;
        fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }
    const cuuint64_t dims[3] = {cols, rows, 1};
    const cuuint64_t strides[2] = {cols * 2, cols * rows * 2};
    const cuuint32_t box[3] = {box0, box1, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t prompt_tc_ws_bytes(const bimamba_dims &d, bool fewer) { return layout_of(d, fewer).bytes; }

cudaError_t launch_prompt_tc(const PromptProblem &q, cudaStream_t stream)
{
    const bimamba_dims &d = q.dims;
    const Layout l = layout_of(d, false);
    char *ws = static_cast<char *>(q.workspace);
    PromptParams p{};
    p.xbc = static_cast<const __nv_bfloat16 *>(q.xbc);
    p.dt = static_cast<const __nv_bfloat16 *>(q.dt);
    p.A = q.A; p.D = q.D; p.conv_w = q.conv_w; p.conv_b = q.conv_b;
    p.cu = q.cu_seqlens; p.slots = q.slots; p.resume = q.resume;
    p.state = q.state;
    p.tail = static_cast<__nv_bfloat16 *>(q.tail);
    p.y = static_cast<__nv_bfloat16 *>(q.y);
    p.head = reinterpret_cast<PlanHeader *>(ws + l.head);
    p.walks = reinterpret_cast<Walk *>(ws + l.walks);
    p.cuts = reinterpret_cast<int4 *>(ws + l.cuts);
    p.act = reinterpret_cast<__nv_bfloat16 *>(ws + l.act);
    p.c_exp = reinterpret_cast<uint8_t *>(ws + l.c_exp);
    p.b_exp = reinterpret_cast<uint8_t *>(ws + l.b_exp);
    p.seg_dec = reinterpret_cast<float *>(ws + l.dec);
    p.seg_state = reinterpret_cast<float *>(ws + l.state);
    p.status = q.status;
    p.batch = d.batch; p.len = d.len; p.H = d.heads; p.ch = d.heads * kP + 2 * kN; p.pool = q.pool;
    p.max_chunks = l.max_chunks;
    p.cut_over = l.cut_over;
    p.seg_chunks = l.seg_chunks;

    CUtensorMap tm_x, tm_bc, tm_y;
    // (no rows at all: the walks load nothing; the maps are placeholders)
    const bool rows = d.len > 0;
    const void *any = p.walks;
    if (!make_map(&tm_x, rows ? q.xbc : any, p.ch, rows ? d.len : 1, kPP, kRawRows, false) ||
        !make_map(&tm_bc, rows ? p.act : any, kAct, rows ? (uint64_t)l.max_chunks * kQ : 1, 64, kQ, true) ||
        !make_map(&tm_y, rows ? q.y : any, (uint64_t)d.heads * kP, rows ? d.len : 1, kP, kQ, true))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(prompt_walk_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmemBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(prompt_walk_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    const int pairs = d.heads / 2;
    prompt_prep_kernel<<<l.max_chunks * kPrepCtas + 1, kPrepThreads, 0, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    count_launch();
    // programmatic launches: set-up and launch beside the end of the kernel before
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (l.max_inner > 0) {
        cfg.gridDim = dim3((unsigned)pairs * l.max_inner);
        if ((e = cudaLaunchKernelEx(&cfg, prompt_walk_kernel<true>, tm_x, tm_bc, tm_y, p)) != cudaSuccess) return e;
        cudaLaunchConfig_t chain = {};
        chain.gridDim = dim3(d.heads * kP * kN / 4 / 256, l.max_cuts);
        chain.blockDim = dim3(256);
        chain.stream = stream;
        chain.attrs = attr;
        chain.numAttrs = 1;
        if ((e = cudaLaunchKernelEx(&chain, prompt_chain_kernel, p)) != cudaSuccess) return e;
        count_launch(2);
    }
    cfg.gridDim = dim3((unsigned)pairs * l.max_walks);
    if ((e = cudaLaunchKernelEx(&cfg, prompt_walk_kernel<false>, tm_x, tm_bc, tm_y, p)) != cudaSuccess) return e;
    count_launch();
    return cudaSuccess;
}

}  // namespace bimamba
