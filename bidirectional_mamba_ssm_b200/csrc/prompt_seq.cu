// prompt_seq.cu -- the causal mixer core over packed ragged prompts on the
// CUDA cores, in fp32: fp32 activations (bf16 operands could not hold their
// bound) and the head shapes without a tensor-core kernel.
//
// Operation (Mamba-2 recurrence, d_conv = 4; the cache entry of "Fixed state,
// long reach: constant-size caches in large-scale block diffusion"), for each
// prompt from its pool entry's state and tail (or zeros), per head:
//     u_t = SiLU(bias + sum_j w_j raw_{t-3+j})        (x, B and C channels)
//     h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t^T,   y_t = h_t C_t + D x_t
//
// Bound by FP32 issue: 5 P N flops per token and head.  Two kernels:
//   1. B and C of every row, activated, in fp32 (all heads read them).
//   2. one CTA per (prompt, head, slice of state rows): the rows of a state
//      are independent, so a head's 64 rows are walked by several CTAs and a
//      few prompts still fill the SMs.  Two compute warps: a thread holds 4
//      rows x 8 columns in registers; the dot products with C over the kLpr
//      threads of a row are summed for 4 tokens at a time by a transposing
//      reduction (each shuffle halves the number of values: 15 shuffles for
//      16 sums, not 64).  A third warp convolves x and loads dt of the next
//      16 tokens, and stores the rows of the last 16, meanwhile; B and C come
//      by asynchronous copies.
// (One CTA per head with conv of B and C inside each: 664 us for prompts of
// 1024, 517, 1 and 300 tokens at 64 heads of 64 x 128.)
#include "common.cuh"
#include "dispatch.h"
#include "tc_ptx.cuh"

namespace bimamba {

namespace {

constexpr int kTok = 16;          // tokens per staged chunk
constexpr int kBatch = 4;         // tokens per reduction
constexpr int kRp = 4;            // state rows per compute thread
constexpr int kCompute = 64;      // compute threads: kSlice * N / 32
constexpr int kThreads = kCompute + 32;
constexpr int kActRows = 32;      // rows per CTA of the first kernel
constexpr int kActThreads = 256;

// State rows per CTA, so that its 64 compute threads hold 32 values each.
template <int kLpr> constexpr int kSlice = kCompute / kLpr * kRp;

// Sums v[0..V) over the kLanes threads of an aligned group; thread l of the
// group ends with max(1, V / kLanes) of the totals in v[0..), the first being
// index transpose_base(l) (threads share one where there are fewer totals).
template <int V, int kLanes>
__device__ __forceinline__ void transpose_sum(float (&v)[V], int lane)
{
    int have = V;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
        if (have == 1) {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
            continue;
        }
        const bool upper = lane & o;
        have /= 2;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            if (i < have) {
                const float keep = upper ? v[i + have] : v[i];
                const float send = upper ? v[i] : v[i + have];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
        }
    }
}
template <int V, int kLanes> __device__ __forceinline__ int transpose_base(int lane)
{
    int base = 0, half = V / 2;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1, half /= 2)
        if (lane & o) base += half;
    return base;
}

// Prompt s: whether it is walked (`bad`: to be reported where it is not).
struct Range {
    int begin, len, slot;
    bool ok, bad;
};
__device__ __forceinline__ Range read_range(const PromptProblem &q, int s)
{
    Range r;
    r.slot = q.slots[s];
    r.begin = q.cu_seqlens[s];
    const int end = q.cu_seqlens[s + 1];
    r.len = end - r.begin;
    r.ok = r.slot >= 0 && r.slot < q.pool && r.begin >= 0 && end >= r.begin && end <= q.dims.len;
    r.bad = !r.ok && r.slot >= 0;
    return r;
}

__device__ __forceinline__ void cp_async16(float *dst, const float *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}

}  // namespace

// act[row][B | C]: conv + SiLU of the B and C channels of 32 packed rows,
// which any number of prompts may share.
template <typename T>
__global__ void __launch_bounds__(kActThreads)
prompt_act_kernel(const PromptProblem q, float *__restrict__ act)
{
    __shared__ int owner[kActRows];   // each row's prompt, or -1
    const int tid = threadIdx.x;
    const int r0 = blockIdx.x * kActRows;
    const int n2 = 2 * q.dims.d_state, HP = q.dims.heads * q.dims.headdim, ch = HP + n2;
    if (tid < kActRows) owner[tid] = -1;
    __syncthreads();
    for (int s = tid; s < q.dims.batch; s += kActThreads) {
        const Range r = read_range(q, s);
        if (!r.ok) continue;
        for (int i = max(r.begin - r0, 0); i < min(r.begin + r.len - r0, kActRows); ++i) owner[i] = s;
    }
    __syncthreads();
    for (int e = tid; e < n2 * (kActRows / 8); e += kActThreads) {
        // one channel of 8 rows, their raw values requested together
        const int c = HP + e % n2, i0 = e / n2 * 8;
        const float4 w = *reinterpret_cast<const float4 *>(q.conv_w + (size_t)c * 4);
        const float bias = q.conv_b ? q.conv_b[c] : 0.0f;
        float raw[11];
#pragma unroll
        for (int i = 0; i < 11; ++i) {
            const int row = r0 + i0 + i - 3;
            raw[i] = row >= 0 && row < q.dims.len ? Elem<T>::load(static_cast<const T *>(q.xbc) + (size_t)row * ch + c) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int s = owner[i0 + i];
            if (s < 0) continue;
            const int t = r0 + i0 + i - q.cu_seqlens[s];
            float v[4] = {raw[i], raw[i + 1], raw[i + 2], raw[i + 3]};
            if (t < 3) {   // tokens before the prompt: its entry's tail, or zeros
                const bool resume = q.resume && q.resume[s] != 0;
                const T *tail = static_cast<const T *>(q.tail) + (size_t)q.slots[s] * 4 * ch + c;
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    if (t - 3 + j < 0) v[j] = resume ? Elem<T>::load(tail + (size_t)(4 + t - 3 + j) * ch) : 0.0f;
            }
            float a = bias;
            a = fmaf(w.x, v[0], a);
            a = fmaf(w.y, v[1], a);
            a = fmaf(w.z, v[2], a);
            a = fmaf(w.w, v[3], a);
            act[(size_t)(r0 + i0 + i) * n2 + (c - HP)] = silu_f(a);
        }
    }
}

template <typename T, int kLpr>
__global__ void __launch_bounds__(kThreads)
prompt_seq_kernel(const PromptProblem q, const float *__restrict__ act)
{
    constexpr int N = 8 * kLpr, kRows = kSlice<kLpr>;
    constexpr int V = kBatch * kRp, kOwn = V > kLpr ? V / kLpr : 1;
    extern __shared__ __align__(16) float smem[];
    // two buffers each: B | C rows, x rows (and dt, decay, the chunk's decay
    // correction), y rows
    float *bc = smem;                                  // [2][kTok][2 N]
    float *xs = bc + 2 * kTok * 2 * N;                 // [2][kTok][kRows]
    float *ys = xs + 2 * kTok * kRows;                 // [2][kTok][kRows]
    float *ds = ys + 2 * kTok * kRows;                 // [2][2 kTok + 4]
    const int P = q.dims.headdim, H = q.dims.heads, ch = H * P + 2 * N;
    const int slices = (P + kRows - 1) / kRows;
    const int h = blockIdx.x / slices, p0 = blockIdx.x % slices * kRows, seq = blockIdx.y, tid = threadIdx.x;
    const int rows = min(kRows, P - p0);   // (a multiple of 8)

    const Range r = read_range(q, seq);
    // a prompt whose slot is another's too belongs to neither
    bool twice = false;
    if (r.slot >= 0)
        for (int s = tid; s < q.dims.batch; s += kThreads) twice |= s != seq && q.slots[s] == r.slot;
    twice = __syncthreads_or(twice);
    if (!r.ok || twice) {
        if (r.slot >= 0 && blockIdx.x == 0 && tid == 0) record_error(q.status, kStatusBadSlot);
        return;
    }
    const int len = r.len;
    const bool resume = q.resume && q.resume[seq] != 0;
    const int nchunks = (len + kTok - 1) / kTok;
    float *state = q.state + (((size_t)r.slot * H + h) * P + p0) * N;
    T *tail = static_cast<T *>(q.tail) + (size_t)r.slot * 4 * ch;
    const T *raw = static_cast<const T *>(q.xbc) + (size_t)r.begin * ch;

    // every thread: chunk k's B and C rows (contiguous) into buffer k % 2
    auto copy_bc = [&](int k) {
        if (k < nchunks) {
            const int vecs = min(kTok, len - k * kTok) * (2 * N / 4);
            float *dst = bc + (k & 1) * kTok * 2 * N;
            const float *src = act + (size_t)(r.begin + k * kTok) * 2 * N;
            for (int e = tid; e < vecs; e += kThreads) cp_async16(dst + 4 * e, src + 4 * e);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto copied = [&]() { asm volatile("cp.async.wait_all;" ::: "memory"); };

    if (tid >= kCompute) {
        // ---- third warp: x, dt and decays of chunk k; y rows of chunk k - 2
        const int st = tid - kCompute;
        const T *dtp = static_cast<const T *>(q.dt) + (size_t)r.begin * H + h;
        T *y = static_cast<T *>(q.y) + ((size_t)r.begin * H + h) * P + p0;
        const float A = q.A[h];
        for (int k = 0; k <= nchunks + 1; ++k) {
            copy_bc(k);
            if (k < nchunks) {
                const int s0 = k * kTok, cnt = min(kTok, len - s0);
                float *x = xs + (k & 1) * kTok * kRows;
                for (int e = st; e < rows * (kTok / 8); e += 32) {
                    // one channel of 8 tokens, their raw values requested together
                    const int p = e % rows, i0 = e / rows * 8, c = h * P + p0 + p;
                    const float4 w = *reinterpret_cast<const float4 *>(q.conv_w + (size_t)c * 4);
                    float v[11];
#pragma unroll
                    for (int i = 0; i < 11; ++i) {
                        const int t = s0 + i0 + i - 3;
                        v[i] = t >= len ? 0.0f
                               : t >= 0 ? Elem<T>::load(raw + (size_t)t * ch + c)
                               : resume ? Elem<T>::load(tail + (size_t)(4 + t) * ch + c) : 0.0f;
                    }
                    const float bias = q.conv_b ? q.conv_b[c] : 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float a = bias;
                        a = fmaf(w.x, v[i], a);
                        a = fmaf(w.y, v[i + 1], a);
                        a = fmaf(w.z, v[i + 2], a);
                        a = fmaf(w.w, v[i + 3], a);
                        x[(i0 + i) * kRows + p] = i0 + i < cnt ? silu_f(a) : 0.0f;
                    }
                }
                // past the end: dt = 0 and decay = 1 leave the state as it is
                float *d2 = ds + (k & 1) * (2 * kTok + 4);
                const float d = st < cnt ? Elem<T>::load(dtp + (size_t)(s0 + st) * H) : 0.0f;
                const float a = st < cnt ? expf(d * A) : 1.0f;
                // Slow decays: what rounding took from a is up to half a step
                // of 2^-24 each token, alike for alike dt, which thousands of
                // tokens would add up; the relative rest (from expm1, whose
                // error is relative to 1 - a) is summed over the chunk and
                // given back to the state once.
                float rest = st < kTok && a >= 0.5f ? (expm1f(d * A) - (a - 1.0f)) / a : 0.0f;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
                if (st < kTok) {
                    d2[st] = d;
                    d2[kTok + st] = a;
                }
                if (st == 0) d2[2 * kTok] = rest;
                // rows of B and C past the end are read by a batch that ends
                // past it, with dt = 0: zeros, not what was there
                float *b = bc + (k & 1) * kTok * 2 * N;
                for (int e = cnt * 2 * N + st; e < kTok * 2 * N; e += 32) b[e] = 0.0f;
            }
            if (k >= 2) {
                const int s0 = (k - 2) * kTok, cnt = min(kTok, len - s0);
                const float *yk = ys + (k & 1) * kTok * kRows;
                for (int e = st; e < cnt * rows; e += 32) {
                    const int i = e / rows, p = e - i * rows;
                    Elem<T>::store(y + (size_t)(s0 + i) * H * P + p, yk[i * kRows + p]);
                }
            }
            copied();
            __syncthreads();
        }
    } else {
        // ---- compute warps: rows kRp g .. kRp g + kRp - 1 of the slice,
        // columns 4 lane + 4 kLpr j + e, as packed pairs
        const int lane = tid % kLpr, g = tid / kLpr;
        const bool in = kRp * g < rows;   // (a thread's rows are all in or all out)
        const int pr = in ? kRp * g : 0;  // (rows past P compute on row 0's inputs and are not stored)
        const float D = q.D[h];
        float2 s[kRp][4];
#pragma unroll
        for (int i = 0; i < kRp; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (in && resume)
                    v = *reinterpret_cast<const float4 *>(state + (size_t)(pr + i) * N + 4 * lane + 4 * kLpr * j);
                s[i][2 * j] = make_float2(v.x, v.y);
                s[i][2 * j + 1] = make_float2(v.z, v.w);
            }
        const int base = transpose_base<V, kLpr>(lane);
        for (int k = 0; k <= nchunks + 1; ++k) {
            copy_bc(k);
            if (k >= 1 && k <= nchunks) {
                const int b = (k - 1) & 1, cnt = min(kTok, len - (k - 1) * kTok);
                const float *bk = bc + b * kTok * 2 * N, *xk = xs + b * kTok * kRows, *dk = ds + b * (2 * kTok + 4);
                float *yk = ys + b * kTok * kRows;
                for (int t0 = 0; t0 < cnt; t0 += kBatch) {
                    float acc[V];
#pragma unroll
                    for (int t = 0; t < kBatch; ++t) {
                        const int i = t0 + t;
                        float2 B[4], C[4];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float4 b4 = *reinterpret_cast<const float4 *>(bk + i * 2 * N + 4 * lane + 4 * kLpr * j);
                            const float4 c4 = *reinterpret_cast<const float4 *>(bk + i * 2 * N + N + 4 * lane + 4 * kLpr * j);
                            B[2 * j] = make_float2(b4.x, b4.y);
                            B[2 * j + 1] = make_float2(b4.z, b4.w);
                            C[2 * j] = make_float2(c4.x, c4.y);
                            C[2 * j + 1] = make_float2(c4.z, c4.w);
                        }
                        const float4 x4 = *reinterpret_cast<const float4 *>(xk + i * kRows + pr);
                        const float x[kRp] = {x4.x, x4.y, x4.z, x4.w};
                        const float dt = dk[i], a = dk[kTok + i];
                        const float2 a2 = make_float2(a, a);
#pragma unroll
                        for (int e = 0; e < kRp; ++e) {
                            const float dx = dt * x[e];
                            const float2 dx2 = make_float2(dx, dx);
                            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                s[e][j] = tc::fma2(a2, s[e][j], tc::mul2(dx2, B[j]));
                                sum = tc::fma2(s[e][j], C[j], sum);
                            }
                            acc[t * kRp + e] = (lane == 0 ? D * x[e] : 0.0f) + (sum.x + sum.y);
                        }
                    }
                    transpose_sum<V, kLpr>(acc, lane);
#pragma unroll
                    for (int e = 0; e < kOwn; ++e) {
                        const int i = t0 + (base + e) / kRp, p = pr + (base + e) % kRp;
                        if (in) yk[i * kRows + p] = acc[e];
                    }
                }
                const float rest = dk[2 * kTok];
                const float2 rest2 = make_float2(rest, rest);
#pragma unroll
                for (int i = 0; i < kRp; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[i][j] = tc::fma2(s[i][j], rest2, s[i][j]);
            }
            copied();
            __syncthreads();
        }
        if (in) {
#pragma unroll
            for (int i = 0; i < kRp; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    *reinterpret_cast<float4 *>(state + (size_t)(pr + i) * N + 4 * lane + 4 * kLpr * j) =
                        make_float4(s[i][2 * j].x, s[i][2 * j].y, s[i][2 * j + 1].x, s[i][2 * j + 1].y);
        }
    }
    __syncthreads();
    // the new tail: this CTA's x channels (nobody else reads them); the first
    // CTA the B and C channels too (read by the kernel before)
    auto commit = [&](int c) {
        T v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = len - 4 + i;
            v[i] = t >= 0 ? raw[(size_t)t * ch + c] : resume ? tail[(size_t)(4 + t) * ch + c] : static_cast<T>(0.0f);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) tail[(size_t)i * ch + c] = v[i];
    };
    for (int p = tid; p < rows; p += kThreads) commit(h * P + p0 + p);
    if (blockIdx.x == 0)
        for (int c = H * P + tid; c < ch; c += kThreads) commit(c);
}

template <typename T, int kLpr>
static cudaError_t launch_one(const PromptProblem &q, const float *act, cudaStream_t stream)
{
    constexpr int N = 8 * kLpr, kRows = kSlice<kLpr>;
    const int P = q.dims.headdim;
    constexpr size_t smem = sizeof(float) * 2 * (kTok * (size_t)(2 * N + 2 * kRows) + 2 * kTok + 4);
    cudaError_t e = cudaFuncSetAttribute(prompt_seq_kernel<T, kLpr>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    prompt_seq_kernel<T, kLpr><<<dim3(q.dims.heads * ((P + kRows - 1) / kRows), q.dims.batch), kThreads, smem, stream>>>(
        q, act);
    return cudaGetLastError();
}

size_t prompt_seq_ws_bytes(const bimamba_dims &d) { return (size_t)d.len * 2 * d.d_state * sizeof(float); }

template <typename T>
cudaError_t launch_prompt_seq(const PromptProblem &q, cudaStream_t stream)
{
    float *act = static_cast<float *>(q.workspace);
    cudaError_t e = cudaSuccess;
    if (q.dims.len > 0) {
        prompt_act_kernel<T><<<(q.dims.len + kActRows - 1) / kActRows, kActThreads, 0, stream>>>(q, act);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        count_launch();
    }
    switch (q.dims.d_state) {
    case 8: e = launch_one<T, 1>(q, act, stream); break;
    case 16: e = launch_one<T, 2>(q, act, stream); break;
    case 32: e = launch_one<T, 4>(q, act, stream); break;
    case 64: e = launch_one<T, 8>(q, act, stream); break;
    case 128: e = launch_one<T, 16>(q, act, stream); break;
    case 256: e = launch_one<T, 32>(q, act, stream); break;
    default: return cudaErrorInvalidValue;
    }
    if (e == cudaSuccess) count_launch();
    return e;
}

template cudaError_t launch_prompt_seq<float>(const PromptProblem &, cudaStream_t);
template cudaError_t launch_prompt_seq<__nv_bfloat16>(const PromptProblem &, cudaStream_t);

}  // namespace bimamba
