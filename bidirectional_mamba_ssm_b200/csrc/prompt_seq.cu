// prompt_seq.cu -- the causal mixer core over packed ragged prompts on the
// CUDA cores, in fp32: fp32 activations (bf16 operands could not hold their
// 1e-4 bound) and the head shapes without a tensor-core kernel.
//
// Operation (Mamba-2 recurrence, d_conv = 4; the cache entry of "Fixed state,
// long reach: constant-size caches in large-scale block diffusion"), for each
// prompt from its pool entry's state and tail (or zeros), per head:
//     u_t = SiLU(bias + sum_j w_j raw_{t-3+j})        (x, B and C channels)
//     h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t^T,   y_t = h_t C_t + D x_t
//
// Bound by FP32 issue: 5 P N flops per token and head against 2 P + ... words
// of traffic.  One CTA owns (prompt, head) and walks its tokens.  A compute
// thread holds kRp state rows x 8 columns in registers; the dot products with
// C over the kLpr threads of a row are summed for several tokens at a time by a
// transposing reduction (each shuffle halves the number of values instead of
// repeating a full one per value: 15 shuffles for 16 sums, not 64).  Four
// staging warps convolve the next 32 tokens and store the outputs of the
// last 32 meanwhile.
#include "common.cuh"
#include "dispatch.h"

namespace bimamba {

namespace {

constexpr int kTok = 32;          // tokens per staged chunk
constexpr int kStagers = 128;     // staging threads

// Shapes of a compute thread's share, by threads per state row (N / 8):
// state rows, and tokens whose sums are reduced together.  At N = 256, 8 rows
// keep the CTA within 640 threads, and 2 tokens its registers within 96.
template <int kLpr> constexpr int kRowsOf = kLpr == 32 ? 8 : 4;
template <int kLpr> constexpr int kBatchOf = kLpr == 32 ? 2 : 4;

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

}  // namespace

template <typename T, int kLpr>
__global__ void __launch_bounds__(640)
prompt_seq_kernel(const PromptProblem q)
{
    constexpr int N = 8 * kLpr;
    constexpr int kRp = kRowsOf<kLpr>, kBatch = kBatchOf<kLpr>;
    constexpr int V = kBatch * kRp, kOwn = V > kLpr ? V / kLpr : 1;
    extern __shared__ __align__(16) float smem[];
    __shared__ int last_reader;
    const int h = blockIdx.x, seq = blockIdx.y, tid = threadIdx.x;
    const int P = q.dims.headdim, H = q.dims.heads, ch = H * P + 2 * N;
    const int nstage = P + 2 * N;
    // two buffers of [x | B | C | dt, decay, the chunk's decay correction] and of y
    const int buf_floats = kTok * (nstage + 2) + 4;
    float *ybuf = smem + 2 * buf_floats;   // [2][kTok][P]

    const int slot = q.slots[seq];
    const int begin = q.cu_seqlens[seq], end = q.cu_seqlens[seq + 1];
    // a prompt whose slot is not one of the pool's, or is another's too, or
    // whose range is not one, is skipped (negative slot: without an error)
    bool twice = false;
    if (slot >= 0)
        for (int r = tid; r < q.dims.batch; r += blockDim.x) twice |= r != seq && q.slots[r] == slot;
    twice = __syncthreads_or(twice);
    if (slot < 0 || slot >= q.pool || twice || begin < 0 || end < begin || end > q.dims.len) {
        if (slot >= 0 && h == 0 && tid == 0) record_error(q.status, kStatusBadSlot);
        return;
    }
    const int len = end - begin;
    const bool resume = q.resume && q.resume[seq] != 0;
    const int nchunks = (len + kTok - 1) / kTok;
    const int nthreads = blockDim.x - kStagers;   // compute threads (whole warps)
    float *state = q.state + ((size_t)slot * H + h) * P * N;
    T *tail = static_cast<T *>(q.tail) + (size_t)slot * 4 * ch;
    const T *raw = static_cast<const T *>(q.xbc) + (size_t)begin * ch;

    if (tid >= nthreads) {
        // ---- staging warps
        const int st = tid - nthreads;
        const T *dtp = static_cast<const T *>(q.dt) + (size_t)begin * H + h;
        T *y = static_cast<T *>(q.y) + ((size_t)begin * H + h) * P;
        const float A = q.A[h];
        for (int k = 0; k <= nchunks + 1; ++k) {
            if (k < nchunks) {
                const int s0 = k * kTok, cnt = min(kTok, len - s0);
                float *xs = smem + (k & 1) * buf_floats, *bs = xs + kTok * P, *cs = bs + kTok * N;
                float *dts = cs + kTok * N, *as = dts + kTok;
                for (int ci = st; ci < nstage; ci += kStagers) {
                    int c, stride;
                    float *dst;
                    if (ci < P) { c = h * P + ci; dst = xs + ci; stride = P; }
                    else if (ci < P + N) { c = H * P + (ci - P); dst = bs + (ci - P); stride = N; }
                    else { c = H * P + (ci - P); dst = cs + (ci - P - N); stride = N; }
                    auto at = [&](int t) -> float {
                        if (t >= 0) return Elem<T>::load(raw + (size_t)t * ch + c);
                        return resume ? Elem<T>::load(tail + (size_t)(4 + t) * ch + c) : 0.0f;
                    };
                    const float4 w = *reinterpret_cast<const float4 *>(q.conv_w + (size_t)c * 4);
                    const float bias = q.conv_b ? q.conv_b[c] : 0.0f;
                    float r0 = at(s0 - 3), r1 = at(s0 - 2), r2 = at(s0 - 1);
                    for (int i0 = 0; i0 < cnt; i0 += 8) {
                        float rv[8];   // requested together
#pragma unroll
                        for (int i = 0; i < 8; ++i) rv[i] = i0 + i < cnt ? at(s0 + i0 + i) : 0.0f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float a = bias;
                            a = fmaf(w.x, r0, a);
                            a = fmaf(w.y, r1, a);
                            a = fmaf(w.z, r2, a);
                            a = fmaf(w.w, rv[i], a);
                            // tokens past the end: zeros, read by a batch that ends past it
                            dst[(i0 + i) * stride] = i0 + i < cnt ? silu_f(a) : 0.0f;
                            r0 = r1; r1 = r2; r2 = rv[i];
                        }
                    }
                }
                if (st < kTok) {
                    // past the end: dt = 0 and decay = 1 leave the state as it is
                    const float d = st < cnt ? Elem<T>::load(dtp + (size_t)(s0 + st) * H) : 0.0f;
                    const float a = st < cnt ? expf(d * A) : 1.0f;
                    dts[st] = d;
                    as[st] = a;
                    // Slow decays: what rounding took from a is up to half a
                    // step of 2^-24 each token, alike for alike dt, which
                    // thousands of tokens would add up; the relative rest
                    // (from expm1, whose error is relative to 1 - a) is
                    // summed over the chunk and given back to the state once.
                    float rest = a >= 0.5f ? (expm1f(d * A) - (a - 1.0f)) / a : 0.0f;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
                    if (st == 0) as[kTok] = rest;
                }
            }
            if (k >= 2) {
                const int s0 = (k - 2) * kTok, cnt = min(kTok, len - s0);
                const float *ys = ybuf + (k & 1) * kTok * P;
                for (int e = st; e < cnt * P; e += kStagers) {
                    const int i = e / P, p = e - i * P;
                    Elem<T>::store(y + (size_t)(s0 + i) * H * P + p, ys[e]);
                }
            }
            __syncthreads();
            if (k == 0 && st == 0) {
                // this CTA has read the prompt's B and C tails (chunk 0's halo)
                __threadfence();
                last_reader = atomicAdd(q.tickets + seq, 1) == H - 1;
            }
        }
    } else {
        // ---- compute warps: rows kRp g .. kRp g + kRp - 1, columns
        // 4 lane + 4 kLpr j + e (two 16-byte pieces per staged row)
        const int lane = tid % kLpr, g = tid / kLpr;
        const int p0 = kRp * g;
        const bool in = p0 < P;   // (P is a multiple of 8: rows of a group are all in or all out)
        const float D = q.D[h];
        float s[kRp][8];
#pragma unroll
        for (int r = 0; r < kRp; ++r)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (in && resume)
                    v = *reinterpret_cast<const float4 *>(state + (size_t)(p0 + r) * N + 4 * lane + 4 * kLpr * j);
                s[r][4 * j] = v.x; s[r][4 * j + 1] = v.y; s[r][4 * j + 2] = v.z; s[r][4 * j + 3] = v.w;
            }
        const int base = transpose_base<V, kLpr>(lane);
        const int pr = in ? p0 : 0;   // (rows past P compute on row 0's inputs and are not stored)
        for (int k = 0; k <= nchunks + 1; ++k) {
            if (k >= 1 && k <= nchunks) {
                const int cnt = min(kTok, len - (k - 1) * kTok);
                const float *xs = smem + ((k - 1) & 1) * buf_floats, *bs = xs + kTok * P, *cs = bs + kTok * N;
                const float *dts = cs + kTok * N, *as = dts + kTok;
                float *ys = ybuf + ((k - 1) & 1) * kTok * P;
                for (int t0 = 0; t0 < cnt; t0 += kBatch) {
                    float acc[V];
#pragma unroll
                    for (int t = 0; t < kBatch; ++t) {
                        const int i = t0 + t;
                        float b[8], c[8], x[kRp];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float4 b4 = *reinterpret_cast<const float4 *>(bs + i * N + 4 * lane + 4 * kLpr * j);
                            const float4 c4 = *reinterpret_cast<const float4 *>(cs + i * N + 4 * lane + 4 * kLpr * j);
                            b[4 * j] = b4.x; b[4 * j + 1] = b4.y; b[4 * j + 2] = b4.z; b[4 * j + 3] = b4.w;
                            c[4 * j] = c4.x; c[4 * j + 1] = c4.y; c[4 * j + 2] = c4.z; c[4 * j + 3] = c4.w;
                        }
#pragma unroll
                        for (int r = 0; r < kRp; r += 4) {
                            const float4 x4 = *reinterpret_cast<const float4 *>(xs + i * P + pr + r);
                            x[r] = x4.x; x[r + 1] = x4.y; x[r + 2] = x4.z; x[r + 3] = x4.w;
                        }
                        const float dt = dts[i], a = as[i];
#pragma unroll
                        for (int r = 0; r < kRp; ++r) {
                            const float dx = dt * x[r];
                            float sum = 0.0f;
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                s[r][e] = fmaf(a, s[r][e], dx * b[e]);
                                sum = fmaf(s[r][e], c[e], sum);
                            }
                            acc[t * kRp + r] = lane == 0 ? fmaf(D, x[r], sum) : sum;
                        }
                    }
                    transpose_sum<V, kLpr>(acc, lane);
#pragma unroll
                    for (int e = 0; e < kOwn; ++e) {
                        const int i = t0 + (base + e) / kRp, r = (base + e) % kRp;
                        if (in) ys[i * P + p0 + r] = acc[e];
                    }
                }
                const float rest = as[kTok];
#pragma unroll
                for (int r = 0; r < kRp; ++r)
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[r][e] = fmaf(s[r][e], rest, s[r][e]);
            }
            __syncthreads();
        }
        if (in) {
#pragma unroll
            for (int r = 0; r < kRp; ++r)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    *reinterpret_cast<float4 *>(state + (size_t)(p0 + r) * N + 4 * lane + 4 * kLpr * j) =
                        make_float4(s[r][4 * j], s[r][4 * j + 1], s[r][4 * j + 2], s[r][4 * j + 3]);
        }
    }
    __syncthreads();
    // the new tail: this head's x channels, and from the last CTA to have
    // read them the row's B and C channels
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
    for (int c = tid; c < P; c += blockDim.x) commit(h * P + c);
    if (!last_reader) return;
    __threadfence();
    for (int c = H * P + tid; c < ch; c += blockDim.x) commit(c);
    if (tid == 0) q.tickets[seq] = 0;   // for the next call
}

template <typename T, int kLpr>
static cudaError_t launch_one(const PromptProblem &q, cudaStream_t stream)
{
    constexpr int N = 8 * kLpr, kRp = kRowsOf<kLpr>;
    const int P = q.dims.headdim;
    const int compute = ((P + kRp - 1) / kRp * kLpr + 31) / 32 * 32;
    const size_t smem = sizeof(float) * 2 * (kTok * (size_t)(P + 2 * N + 2 + P) + 4);
    cudaError_t e = cudaFuncSetAttribute(prompt_seq_kernel<T, kLpr>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    prompt_seq_kernel<T, kLpr><<<dim3(q.dims.heads, q.dims.batch), compute + kStagers, smem, stream>>>(q);
    e = cudaGetLastError();
    if (e == cudaSuccess) count_launch();
    return e;
}

template <typename T>
cudaError_t launch_prompt_seq(const PromptProblem &q, cudaStream_t stream)
{
    switch (q.dims.d_state) {
    case 8: return launch_one<T, 1>(q, stream);
    case 16: return launch_one<T, 2>(q, stream);
    case 32: return launch_one<T, 4>(q, stream);
    case 64: return launch_one<T, 8>(q, stream);
    case 128: return launch_one<T, 16>(q, stream);
    case 256: return launch_one<T, 32>(q, stream);
    default: return cudaErrorInvalidValue;
    }
}

template cudaError_t launch_prompt_seq<float>(const PromptProblem &, cudaStream_t);
template cudaError_t launch_prompt_seq<__nv_bfloat16>(const PromptProblem &, cudaStream_t);

}  // namespace bimamba
