// token_step.cu -- one new token of each of a batch of cached streams: the
// causal conv + SiLU, the state update and the output, in place in the pool.
//
// Operation (Mamba-2 recurrence, d_conv = 4; the cache entry of "Fixed state,
// long reach: constant-size caches in large-scale block diffusion": the
// forward SSM state and the last raw tokens), per row and head:
//     u = SiLU(bias + sum_j w_j raw_{t-3+j})          (x, B and C channels)
//     h <- exp(dt A) h + dt x B^T,   y = h C + D x
//     tail <- its last 3 tokens and the new one
//
// Bound by HBM: the fp32 state (4 P N bytes a head) is read and written once
// and is nearly all of the traffic (per 64 x 128 head 64 KB, against ~6 KB of
// conv inputs that its CTA reads mostly from L2).  One CTA per (row, head),
// so that a single row already spreads over many SMs; every thread requests
// the first kStepLoads of its vectors of the state before anything else (at
// 64 x 128 half of them: the others follow the first half's update), and the
// conv of the head's x and the row's B and C (recomputed by every head: they
// are small, and a launch of their own would cost more than the reads) runs
// under those loads.
// 64 heads of 64 x 128, calls one after another on the same buffers: 256 rows
// fp32 194 us (bytes 170), 32 rows bf16 29 (21; 2048 CTAs, 740 at a time: what
// is left is the overlap of a CTA's stores with its successor's loads), one row
// 12, the host's call.
#include "common.cuh"
#include "dispatch.h"

namespace bimamba {

namespace {

constexpr int kStepThreads = 256;
// 16-byte state loads a thread keeps in flight, and CTAs per SM.  256 rows of
// 64 heads x 64 x 128: 8 loads and 3 CTAs 210 us, 8 and 4 195 us, 4 and 5
// 182 us.
constexpr int kStepLoads = 4, kStepCtas = 5;

}  // namespace

// The B and C channels' tails are read by every head's CTA of a row and
// rewritten by the last of them to have read (a ticket per row in the
// workspace, returned to zero by that CTA); nobody waits for it.
template <typename T, int N>
__global__ void __launch_bounds__(kStepThreads, N == 256 ? 4 : kStepCtas)
token_step_kernel(const StepProblem q)
{
    constexpr int kRowVecs = N / 4;                       // float4s of one state row
    constexpr int kLanes = kRowVecs < 32 ? kRowVecs : 32; // threads that share a state row
    constexpr int kPer = kRowVecs / kLanes;               // float4s of a row per thread (N = 256: 2)
    constexpr int kRowsPass = kStepThreads / kLanes;      // state rows per pass
    constexpr int kPasses = kStepLoads / kPer;            // passes whose loads are in flight together
    __shared__ __align__(16) float act[128 + 2 * N];      // x (this head) | B | C; B and C read as float4
    __shared__ int last_reader;

    const int h = blockIdx.x, row = blockIdx.y, tid = threadIdx.x;
    const int P = q.P, ch = q.H * P + 2 * N;
    const int slot = q.slots[row];
    const int col = tid % kLanes, prow = tid / kLanes;
    const bool in_pool = slot >= 0 && slot < q.pool;
    float4 *state = reinterpret_cast<float4 *>(q.state + ((size_t)(in_pool ? slot : 0) * q.H + h) * P * N);
    T *tail = static_cast<T *>(q.tail) + (size_t)(in_pool ? slot : 0) * 4 * ch;
    const T *raw = static_cast<const T *>(q.xbc) + (size_t)row * ch;
    float4 s[kPasses][kPer];
    auto fetch = [&](int p0) {
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int p = p0 + i * kRowsPass + prow;
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                if (p < P) s[i][k] = state[(size_t)p * kRowVecs + col + kLanes * k];
        }
    };
    // this thread's conv channels, requested right behind the state
    constexpr int kConv = (128 + 2 * N + kStepThreads - 1) / kStepThreads;
    T t[kConv][4];
    float4 w[kConv];
    float bias[kConv];
    auto channel = [&](int i) { return i < P ? h * P + i : q.H * P + (i - P); };
    if (in_pool) {
        fetch(0);
#pragma unroll
        for (int j = 0; j < kConv; ++j) {
            const int i = tid + j * kStepThreads;
            if (i < P + 2 * N) {
                const int c = channel(i);
                t[j][0] = tail[ch + c];
                t[j][1] = tail[2 * ch + c];
                t[j][2] = tail[3 * ch + c];
                t[j][3] = raw[c];
                w[j] = *reinterpret_cast<const float4 *>(q.conv_w + (size_t)c * 4);
                bias[j] = q.conv_b ? q.conv_b[c] : 0.0f;
            }
        }
    }
    // a row whose slot is not one of the pool's, or is another row's too, is
    // skipped (a negative one without an error: a padding row)
    bool twice = false;
    if (slot >= 0)
        for (int r = tid; r < q.rows; r += kStepThreads) twice |= r != row && q.slots[r] == slot;
    twice = __syncthreads_or(twice);
    if (!in_pool || twice) {
        if (slot >= 0 && h == 0 && tid == 0) record_error(q.status, kStatusBadSlot);
        return;
    }

#pragma unroll
    for (int j = 0; j < kConv; ++j) {
        const int i = tid + j * kStepThreads;
        if (i >= P + 2 * N) break;
        float a = bias[j];
        a = fmaf(w[j].x, static_cast<float>(t[j][0]), a);
        a = fmaf(w[j].y, static_cast<float>(t[j][1]), a);
        a = fmaf(w[j].z, static_cast<float>(t[j][2]), a);
        a = fmaf(w[j].w, static_cast<float>(t[j][3]), a);
        act[i] = silu_f(a);
        if (i < P) {   // this head's own channels
            const int c = channel(i);
            tail[c] = t[j][0];
            tail[ch + c] = t[j][1];
            tail[2 * ch + c] = t[j][2];
            tail[3 * ch + c] = t[j][3];
        }
    }
    const float dt = Elem<T>::load(static_cast<const T *>(q.dt) + (size_t)row * q.H + h);
    // exp(dt A) h as h f + (h or 0).  f = exp - 1 for a slow decay: exp itself,
    // rounded, is off by up to 2^-25, alike for alike dt, and thousands of
    // tokens would add that up in the state
    const float v = dt * q.A[h];
    const bool slow = v > -0.5f;
    const float decay = slow ? expm1f(v) : expf(v), D = q.D[h];
    __syncthreads();
    // (the barrier: this CTA has read the row's B and C tails)
    if (tid == 0) {
        __threadfence();
        last_reader = atomicAdd(q.tickets + row, 1) == q.H - 1;
    }

    float4 B[kPer], C[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        B[k] = *reinterpret_cast<const float4 *>(act + P + 4 * (col + kLanes * k));
        C[k] = *reinterpret_cast<const float4 *>(act + P + N + 4 * (col + kLanes * k));
    }
    T *y = static_cast<T *>(q.y) + ((size_t)row * q.H + h) * P;
    for (int p0 = 0; p0 < P; p0 += kPasses * kRowsPass) {
        if (p0 > 0) fetch(p0);
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int p = p0 + i * kRowsPass + prow;
            const float x = p < P ? act[p] : 0.0f;
            const float dx = dt * x;
            float acc = 0.0f;
            if (p < P) {
#pragma unroll
                for (int k = 0; k < kPer; ++k) {
                    float4 v = s[i][k];
                    v.x = fmaf(dx, B[k].x, fmaf(decay, v.x, slow ? v.x : 0.0f));
                    v.y = fmaf(dx, B[k].y, fmaf(decay, v.y, slow ? v.y : 0.0f));
                    v.z = fmaf(dx, B[k].z, fmaf(decay, v.z, slow ? v.z : 0.0f));
                    v.w = fmaf(dx, B[k].w, fmaf(decay, v.w, slow ? v.w : 0.0f));
                    state[(size_t)p * kRowVecs + col + kLanes * k] = v;
                    acc = fmaf(v.x, C[k].x, acc);
                    acc = fmaf(v.y, C[k].y, acc);
                    acc = fmaf(v.z, C[k].z, acc);
                    acc = fmaf(v.w, C[k].w, acc);
                }
            }
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
            if (col == 0 && p < P) Elem<T>::store(y + p, fmaf(D, x, acc));
        }
    }
    __syncthreads();
    if (!last_reader) return;
    // every head's CTA has read the row's B and C tails
    __threadfence();
    for (int c = q.H * P + tid; c < ch; c += kStepThreads) {
        const T t1 = tail[ch + c], t2 = tail[2 * ch + c], t3 = tail[3 * ch + c];
        tail[c] = t1;
        tail[ch + c] = t2;
        tail[2 * ch + c] = t3;
        tail[3 * ch + c] = raw[c];
    }
    if (tid == 0) q.tickets[row] = 0;   // for the next call
}

template <typename T>
cudaError_t launch_token_step(const StepProblem &q, cudaStream_t stream)
{
    const dim3 grid(q.H, q.rows);
    switch (q.N) {
    case 8: token_step_kernel<T, 8><<<grid, kStepThreads, 0, stream>>>(q); break;
    case 16: token_step_kernel<T, 16><<<grid, kStepThreads, 0, stream>>>(q); break;
    case 32: token_step_kernel<T, 32><<<grid, kStepThreads, 0, stream>>>(q); break;
    case 64: token_step_kernel<T, 64><<<grid, kStepThreads, 0, stream>>>(q); break;
    case 128: token_step_kernel<T, 128><<<grid, kStepThreads, 0, stream>>>(q); break;
    case 256: token_step_kernel<T, 256><<<grid, kStepThreads, 0, stream>>>(q); break;
    default: return cudaErrorInvalidValue;
    }
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launch();
    return e;
}

template cudaError_t launch_token_step<float>(const StepProblem &, cudaStream_t);
template cudaError_t launch_token_step<__nv_bfloat16>(const StepProblem &, cudaStream_t);

}  // namespace bimamba
