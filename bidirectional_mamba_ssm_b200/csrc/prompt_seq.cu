// prompt_seq.cu -- the causal mixer core over packed ragged prompts on the
// CUDA cores, in fp32: fp32 activations (the tensor-core kernel's y is made for
// bf16; its 16-bit operands would need two halves each throughout, as its state's
// have) and the head shapes without a tensor-core kernel.
//
// Operation (Mamba-2 recurrence, d_conv = 4; the cache entry of "Fixed state,
// long reach: constant-size caches in large-scale block diffusion"), for each
// prompt from its pool entry's state and tail (or zeros), per head:
//     u_t = SiLU(bias + sum_j w_j raw_{t-3+j})        (x, B and C channels)
//     h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t^T,   y_t = h_t C_t + D x_t
//
// Bound by FP32 issue: 5 P N flops per token and head.  1842 tokens in four
// prompts (1024, 517, 1 and 300), 64 heads of 64 x 128: 305 us, where the
// flops take 65; the longest prompt alone takes 183 (a warp's 16 fused
// operations a row and token are half of its cycles, the rest latencies).
// Two kernels:
//   1. every channel activated, and each head's dt and decays, in fp32: what
//      the walks read.  30 us of the above.  (Done inside the walks, by a warp
//      beside two that compute, the conv and its exponentials bound them: 370
//      us in all.)
//   2. one CTA per (prompt, head, slice of state rows): the rows of a state
//      are independent, so a head's 64 rows are walked by several CTAs and a
//      few prompts still fill the SMs.  A thread holds 4 rows x 8 columns in
//      registers (2 rows: 285 us above, but 16 prompts of 100 tokens 250 us
//      for 180); the dot products with C over the kLpr threads of a row are
//      summed for 4 tokens at a time by a transposing reduction (each shuffle
//      halves the number of values: 15 shuffles for 16 sums, not 64).  The
//      next 16 tokens come by asynchronous copies.
#include "common.cuh"
#include "dispatch.h"
#include "tc_ptx.cuh"

namespace bimamba {

namespace {

constexpr int kTok = 16;          // tokens per staged chunk
constexpr int kBatch = 4;         // tokens per reduction
constexpr int kRp = 4;            // state rows per compute thread
constexpr int kCompute = 64;      // threads of a walk: kSlice * N / 32
constexpr int kActRows = 32;      // rows per CTA of the first kernel
constexpr int kActThreads = 256;  // channels per CTA

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

// act[row][channel] = conv + SiLU of 32 packed rows, which any number of
// prompts may share, and (first CTAs) dec[row][head] = (dt, exp(dt A), what
// rounding took from it relative to it, 0).
template <typename T>
__global__ void __launch_bounds__(kActThreads)
prompt_act_kernel(const PromptProblem q, float *__restrict__ act, float4 *__restrict__ dec)
{
    __shared__ int owner[kActRows], token[kActRows];   // each row's prompt, or -1, and its token there
    const int tid = threadIdx.x;
    const int r0 = blockIdx.x * kActRows;
    const int H = q.dims.heads, ch = H * q.dims.headdim + 2 * q.dims.d_state;
    if (tid < kActRows) owner[tid] = -1;
    __syncthreads();
    for (int s = tid; s < q.dims.batch; s += kActThreads) {
        const Range r = read_range(q, s);
        if (!r.ok) continue;
        for (int i = max(r.begin - r0, 0); i < min(r.begin + r.len - r0, kActRows); ++i) {
            owner[i] = s;
            token[i] = r0 + i - r.begin;
        }
    }
    __syncthreads();
    const int c = blockIdx.y * kActThreads + tid;
    if (c < ch) {
        const float4 w = *reinterpret_cast<const float4 *>(q.conv_w + (size_t)c * 4);
        const float bias = q.conv_b ? q.conv_b[c] : 0.0f;
        const T *src = static_cast<const T *>(q.xbc) + ((size_t)r0 * ch + c);
        float *dst = act + ((size_t)r0 * ch + c);
        for (int i0 = 0; i0 < kActRows; i0 += 8, src += (size_t)8 * ch, dst += (size_t)8 * ch) {
            float raw[11];   // requested together
#pragma unroll
            for (int i = 0; i < 11; ++i) {
                const int row = r0 + i0 + i - 3;
                raw[i] = row >= 0 && row < q.dims.len ? Elem<T>::load(src + (long long)(i - 3) * ch) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int s = owner[i0 + i];
                if (s < 0) continue;
                const int t = token[i0 + i];
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
                dst[(size_t)i * ch] = silu_f(a);
            }
        }
    }
    if (blockIdx.y == 0) {
        for (int e = tid; e < min(kActRows, q.dims.len - r0) * H; e += kActThreads) {
            const int i = e / H, h = e - i * H;
            const float d = Elem<T>::load(static_cast<const T *>(q.dt) + (size_t)(r0 + i) * H + h);
            const float v = d * q.A[h], a = expf(v);
            // Slow decays: what rounding takes from a is up to half a step of
            // 2^-24 each token, alike for alike dt, which thousands of tokens
            // would add up; the relative rest (from expm1, whose error is
            // relative to 1 - a) is given back to the state once a chunk.
            dec[(size_t)(r0 + i) * H + h] = make_float4(d, a, a >= 0.5f ? (expm1f(v) - (a - 1.0f)) / a : 0.0f, 0.0f);
        }
    }
}

template <typename T, int kLpr>
__global__ void __launch_bounds__(kCompute)
prompt_seq_kernel(const PromptProblem q, const float *__restrict__ act, const float4 *__restrict__ dec)
{
    constexpr int N = 8 * kLpr, kRows = kSlice<kLpr>;
    constexpr int V = kBatch * kRp, kOwn = V > kLpr ? V / kLpr : 1;
    extern __shared__ __align__(16) float smem[];
    // two buffers each: rows of B | C, of x, and (dt, decay, rest, 0)
    float *bc = smem;                                  // [2][kTok][2 N]
    float *xs = bc + 2 * kTok * 2 * N;                 // [2][kTok][kRows]
    float *ds = xs + 2 * kTok * kRows;                 // [2][kTok][4]
    const int P = q.dims.headdim, H = q.dims.heads, ch = H * P + 2 * N;
    const int slices = (P + kRows - 1) / kRows;
    const int h = blockIdx.x / slices, p0 = blockIdx.x % slices * kRows, seq = blockIdx.y, tid = threadIdx.x;
    const int rows = min(kRows, P - p0);   // (a multiple of 8)

    const Range r = read_range(q, seq);
    // a prompt whose slot is another's too belongs to neither
    bool twice = false;
    if (r.slot >= 0)
        for (int s = tid; s < q.dims.batch; s += kCompute) twice |= s != seq && q.slots[s] == r.slot;
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
    T *y = static_cast<T *>(q.y) + ((size_t)r.begin * H + h) * P + p0;

    // chunk k's rows into buffer k % 2; tokens past the end: x = B = C = 0,
    // dt = 0 and decay = 1 (they leave the state as it is)
    auto copy = [&](int k) {
        if (k < nchunks) {
            const int cnt = min(kTok, len - k * kTok), b = k & 1;
            const float *src = act + (size_t)(r.begin + k * kTok) * ch;
            float *db = bc + b * kTok * 2 * N, *dx = xs + b * kTok * kRows, *dd = ds + b * kTok * 4;
            for (int e = tid; e < kTok * (N / 2); e += kCompute) {
                const int i = e / (N / 2), v = e % (N / 2) * 4;
                if (i < cnt) cp_async16(db + i * 2 * N + v, src + (size_t)i * ch + H * P + v);
                else *reinterpret_cast<float4 *>(db + i * 2 * N + v) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            for (int e = tid; e < kTok * (rows / 4); e += kCompute) {
                const int i = e / (rows / 4), v = e % (rows / 4) * 4;
                if (i < cnt) cp_async16(dx + i * kRows + v, src + (size_t)i * ch + h * P + p0 + v);
                else *reinterpret_cast<float4 *>(dx + i * kRows + v) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            if (tid < kTok) {
                if (tid < cnt)
                    cp_async16(dd + 4 * tid, reinterpret_cast<const float *>(dec + (size_t)(r.begin + k * kTok + tid) * H + h));
                else
                    *reinterpret_cast<float4 *>(dd + 4 * tid) = make_float4(0.0f, 1.0f, 0.0f, 0.0f);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    // rows kRp g .. kRp g + kRp - 1 of the slice, columns 4 lane + 4 kLpr j + e,
    // as packed pairs
    const int lane = tid % kLpr, g = tid / kLpr;
    const bool in = kRp * g < rows;   // (a thread's rows are all in or all out)
    const int pr = in ? kRp * g : 0;  // (rows past P compute on row 0's inputs and are not stored)
    const float D = lane == 0 ? q.D[h] : 0.0f;   // (one of a row's threads adds D x)
    copy(0);
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
    for (int k = 0; k < nchunks; ++k) {
        copy(k + 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        const int b = k & 1, cnt = min(kTok, len - k * kTok);
        const float *bk = bc + b * kTok * 2 * N, *xk = xs + b * kTok * kRows;
        const float4 *dk = reinterpret_cast<const float4 *>(ds) + b * kTok;
        float rest = 0.0f;
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
                const float4 d4 = dk[i];   // dt, decay, rest
                const float2 a2 = make_float2(d4.y, d4.y);
                rest += d4.z;
#pragma unroll
                for (int e = 0; e < kRp; ++e) {
                    const float dx = d4.x * x[e];
                    const float2 dx2 = make_float2(dx, dx);
                    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s[e][j] = tc::fma2(a2, s[e][j], tc::mul2(dx2, B[j]));
                        sum = tc::fma2(s[e][j], C[j], sum);
                    }
                    acc[t * kRp + e] = fmaf(D, x[e], sum.x + sum.y);
                }
            }
            transpose_sum<V, kLpr>(acc, lane);
#pragma unroll
            for (int e = 0; e < kOwn; ++e) {
                const int i = t0 + (base + e) / kRp, p = pr + (base + e) % kRp;
                if (in && i < cnt) Elem<T>::store(y + (size_t)(k * kTok + i) * H * P + p, acc[e]);
            }
        }
        const float2 rest2 = make_float2(rest, rest);
#pragma unroll
        for (int i = 0; i < kRp; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = tc::fma2(s[i][j], rest2, s[i][j]);
        __syncthreads();   // buffer b read: the copy of chunk k + 2 may overwrite it
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (in) {
#pragma unroll
        for (int i = 0; i < kRp; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                *reinterpret_cast<float4 *>(state + (size_t)(pr + i) * N + 4 * lane + 4 * kLpr * j) =
                    make_float4(s[i][2 * j].x, s[i][2 * j].y, s[i][2 * j + 1].x, s[i][2 * j + 1].y);
    }
    // the new tail (the old one was read by the kernel before): this CTA's x
    // channels, and from the first CTA the B and C channels
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
    for (int p = tid; p < rows; p += kCompute) commit(h * P + p0 + p);
    if (blockIdx.x == 0)
        for (int c = H * P + tid; c < ch; c += kCompute) commit(c);
}

template <typename T, int kLpr>
static cudaError_t launch_one(const PromptProblem &q, const float *act, const float4 *dec, cudaStream_t stream)
{
    constexpr int N = 8 * kLpr, kRows = kSlice<kLpr>;
    const int P = q.dims.headdim;
    constexpr size_t smem = sizeof(float) * 2 * kTok * (size_t)(2 * N + kRows + 4);
    cudaError_t e = cudaFuncSetAttribute(prompt_seq_kernel<T, kLpr>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    prompt_seq_kernel<T, kLpr><<<dim3(q.dims.heads * ((P + kRows - 1) / kRows), q.dims.batch), kCompute, smem, stream>>>(
        q, act, dec);
    return cudaGetLastError();
}

// workspace: dec (16 bytes per row and head), act (fp32 per row and channel)
size_t prompt_seq_ws_bytes(const bimamba_dims &d)
{
    return (size_t)d.len * (16 * (size_t)d.heads + 4 * ((size_t)d.heads * d.headdim + 2 * d.d_state));
}

template <typename T>
cudaError_t launch_prompt_seq(const PromptProblem &q, cudaStream_t stream)
{
    float4 *dec = static_cast<float4 *>(q.workspace);
    float *act = reinterpret_cast<float *>(dec + (size_t)q.dims.len * q.dims.heads);
    const int ch = q.dims.heads * q.dims.headdim + 2 * q.dims.d_state;
    cudaError_t e = cudaSuccess;
    if (q.dims.len > 0) {
        prompt_act_kernel<T><<<dim3((q.dims.len + kActRows - 1) / kActRows, (ch + kActThreads - 1) / kActThreads),
                               kActThreads, 0, stream>>>(q, act, dec);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        count_launch();
    }
    switch (q.dims.d_state) {
    case 8: e = launch_one<T, 1>(q, act, dec, stream); break;
    case 16: e = launch_one<T, 2>(q, act, dec, stream); break;
    case 32: e = launch_one<T, 4>(q, act, dec, stream); break;
    case 64: e = launch_one<T, 8>(q, act, dec, stream); break;
    case 128: e = launch_one<T, 16>(q, act, dec, stream); break;
    case 256: e = launch_one<T, 32>(q, act, dec, stream); break;
    default: return cudaErrorInvalidValue;
    }
    if (e == cudaSuccess) count_launch();
    return e;
}

template cudaError_t launch_prompt_seq<float>(const PromptProblem &, cudaStream_t);
template cudaError_t launch_prompt_seq<__nv_bfloat16>(const PromptProblem &, cudaStream_t);

}  // namespace bimamba
