// norm.cu -- the (residual add and) layer norm in front of a mixer's input
// projection, and its backward pass.
//
// Operation ("DiffuMamba" blog post, network-architecture listing: mixer
// blocks with a LayerNorm; eps inside the root, biased variance), per row:
//     h = x + r            (r optional; h kept in fp32, stored rounded once)
//     m = mean(h),  s = 1 / sqrt(mean((h - m)^2) + eps)
//     y = (h - m) s g + b
// and, with z = (h - m) s and a = dy g,
//     dx = s (a - mean(a) - z mean(a z)) + dsum
//     dg = sum over rows of dy z,   db = sum over rows of dy.
//
// Bound by HBM: every activation is read or written once, everything else
// stays in registers.  A row belongs to `kWarps` warps, each thread holding up
// to kFwdVec (backward: kBwdVec) vectors of 8 of its elements.  32768 x 2048
// bf16: the forward with a residual and the backward with dsum 89 and 99 us,
// where the bytes take 82 at the card's copy rate.
#include "common.cuh"
#include "dispatch.h"
#include "tc_ptx.cuh"

namespace bimamba {

namespace {

// 8 consecutive elements as loaded (bf16: 16 bytes, fp32: 32 bytes).
template <typename T> struct Raw8 {
    uint4 r[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
    }
    // as 4 packed pairs
    __device__ __forceinline__ void get(float2 (&v)[4]) const
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v[2 * i] = make_float2(__uint_as_float(r[i].x), __uint_as_float(r[i].y));
                v[2 * i + 1] = make_float2(__uint_as_float(r[i].z), __uint_as_float(r[i].w));
            }
        } else {
            const uint32_t w[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v[4 * i] = __uint_as_float(r[i].x);
                v[4 * i + 1] = __uint_as_float(r[i].y);
                v[4 * i + 2] = __uint_as_float(r[i].z);
                v[4 * i + 3] = __uint_as_float(r[i].w);
            }
        } else {
            const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&r[0]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = __bfloat1622float2(h[i]);
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Barrier over the warps of one row (rows of a CTA advance independently).
template <int kWarps> __device__ __forceinline__ void row_sync(int slot)
{
    if constexpr (kWarps > 1)
        asm volatile("bar.sync %0, %1;" ::"r"(slot + 1), "r"(32 * kWarps) : "memory");
}

constexpr int kNormThreads = 256;
constexpr int norm_threads(int warps) { return warps * 32 > kNormThreads ? warps * 32 : kNormThreads; }

constexpr int kFwdVec = 4;   // vectors a thread holds in the forward pass
constexpr int kBwdVec = 2;   // in the backward pass (which also keeps column sums)
// Rows in flight per thread (24 KB of ring each for 256 threads and bf16; two
// CTAs an SM, one of 512 threads).  32768 x 2048 bf16: 4 rows 105 us, 3 or 2
// 102 us (98 with 3 since the sums are packed pairs).
template <typename T> constexpr int bwd_depth = sizeof(T) == 2 ? 3 : 2;
template <typename T> constexpr size_t ring_bytes(int threads)
{
    return (size_t)bwd_depth<T> * 3 * kBwdVec * 8 * sizeof(T) * threads;
}

}  // namespace

// Forward: one row per `kWarps` warps.  Mean and squared deviations are
// formed per warp in two passes over its registers and merged across the
// row's warps (counts n_w, means m_w, deviations d_w):
//     m = sum n_w m_w / n,   var n = sum d_w + n_w (m_w - m)^2
// so one exchange through shared memory suffices and nothing cancels.
template <typename T, int kWarps>
__global__ void __launch_bounds__(norm_threads(kWarps))
layer_norm_kernel(const T *__restrict__ x, const T *__restrict__ residual, const float *__restrict__ gamma,
                  const float *__restrict__ beta, T *__restrict__ y, T *__restrict__ sum_out,
                  float *__restrict__ mean_out, float *__restrict__ rstd_out, long long rows, int cols, float eps)
{
    constexpr int kRows = norm_threads(kWarps) / (32 * kWarps);
    __shared__ float2 part[kRows][kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slot = warp / kWarps, rw = warp % kWarps;
    const long long row = (long long)blockIdx.x * kRows + slot;
    if (row >= rows) return;   // (a whole row's warps leave together)
    const int vecs = cols >> 3;
    const int v0 = rw * 32 + lane;   // this thread's vectors: v0 + 32 kWarps i
    const T *xr = x + row * cols;
    const T *rr = residual ? residual + row * cols : nullptr;

    float v[kFwdVec][8];
    {
        Raw8<T> a[kFwdVec], b[kFwdVec];
#pragma unroll
        for (int i = 0; i < kFwdVec; ++i) {
            const int e = v0 + 32 * kWarps * i;
            if (e < vecs) a[i].load(xr + 8 * e);
        }
        if (rr) {
#pragma unroll
            for (int i = 0; i < kFwdVec; ++i) {
                const int e = v0 + 32 * kWarps * i;
                if (e < vecs) b[i].load(rr + 8 * e);
            }
        }
#pragma unroll
        for (int i = 0; i < kFwdVec; ++i) {
            const int e = v0 + 32 * kWarps * i;
            if (e >= vecs) {
#pragma unroll
                for (int q = 0; q < 8; ++q) v[i][q] = 0.0f;
                continue;
            }
            a[i].get(v[i]);
            if (rr) {
                float w[8];
                b[i].get(w);
#pragma unroll
                for (int q = 0; q < 8; ++q) v[i][q] += w[q];
                Vec8<T>::store(sum_out + row * cols + 8 * e, v[i]);
            }
        }
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kFwdVec; ++i)
#pragma unroll
        for (int q = 0; q < 8; ++q) s += v[i][q];
    s = warp_sum(s);
    // elements of warp w: its full strides, and what is left of the last one
    auto count = [&](int w) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < kFwdVec; ++i) n += min(max(vecs - 32 * (w + kWarps * i), 0), 32);
        return 8.0f * n;
    };
    const float nw = count(rw);
    float mean = nw > 0.0f ? s / nw : 0.0f;
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < kFwdVec; ++i) {
        if (v0 + 32 * kWarps * i < vecs) {
#pragma unroll
            for (int q = 0; q < 8; ++q) d = fmaf(v[i][q] - mean, v[i][q] - mean, d);
        }
    }
    d = warp_sum(d);
    if constexpr (kWarps > 1) {
        if (lane == 0) part[slot][rw] = make_float2(mean, d);
        row_sync<kWarps>(slot);
        float m = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaf(count(w), part[slot][w].x, m);
        m /= (float)cols;
        d = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float2 q = part[slot][w];
            d += fmaf(count(w) * (q.x - m), q.x - m, q.y);
        }
        mean = m;
    }
    const float rstd = rsqrtf(d / (float)cols + eps);
    if (rw == 0 && lane == 0) {
        mean_out[row] = mean;
        rstd_out[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < kFwdVec; ++i) {
        const int e = v0 + 32 * kWarps * i;
        if (e >= vecs) continue;
        float g[8], o[8];
        Vec8<float>::load(gamma + 8 * e, g);
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] = (v[i][q] - mean) * rstd * g[q];
        if (beta) {
            Vec8<float>::load(beta + 8 * e, g);
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] += g[q];
        }
        Vec8<T>::store(y + row * cols + 8 * e, o);
    }
}

// Backward: a fixed set of rows per group of `kWarps` warps, so that each
// thread keeps its own columns of dg and db in registers over all of them;
// the CTA's groups join in shared memory and write one partial row
// part[cta][dg | db][cols].  The order of every sum is fixed by the launch.
// A thread reads only what it copied itself, kDepth rows ahead, by
// asynchronous 16-byte copies into its own places of a ring in shared memory:
// no barrier, and no registers for what is in flight (held in registers, one
// row ahead took 173 of them, one CTA per SM and 142 us for 32768 x 2048 bf16
// with dsum; the bytes take 82 us).
template <typename T, int kWarps>
__global__ void __launch_bounds__(norm_threads(kWarps), kWarps > 8 ? 1 : 2)
layer_norm_bwd_kernel(const T *__restrict__ dy, const T *__restrict__ h, const float *__restrict__ gamma,
                      const float *__restrict__ mean, const float *__restrict__ rstd, const T *__restrict__ dsum,
                      T *__restrict__ dx, float *__restrict__ part, long long rows, int cols)
{
    // the join kernel behind this one may take its place as CTAs end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kThreads = norm_threads(kWarps), kRows = kThreads / (32 * kWarps);
    constexpr int kPieces = sizeof(T) / 2;   // 16-byte pieces of a vector
    constexpr int kDepth = bwd_depth<T>;
    __shared__ float2 red[2][kRows][kWarps];
    extern __shared__ __align__(16) uint4 ring[];   // [kDepth][h, dy, dsum][kBwdVec][kPieces][thread]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int slot = warp / kWarps, rw = warp % kWarps;
    const int vecs = cols >> 3;
    const int v0 = rw * 32 + lane;
    const float inv_cols = 1.0f / (float)cols;

    float2 g[kBwdVec][4], dg[kBwdVec][4], db[kBwdVec][4];   // (packed pairs: 102 us without)
    const float2 zero = make_float2(0.0f, 0.0f), one = make_float2(1.0f, 1.0f);
#pragma unroll
    for (int i = 0; i < kBwdVec; ++i) {
        const int e = v0 + 32 * kWarps * i;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            dg[i][q] = db[i][q] = zero;
            g[i][q] = e < vecs ? *reinterpret_cast<const float2 *>(gamma + 8 * e + 2 * q) : zero;
        }
    }
    auto place = [&](int d, int t, int i) { return ring + (((d * 3 + t) * kBwdVec + i) * kPieces) * kThreads + tid; };
    auto copy = [&](int d, int t, int i, const T *src) {
#pragma unroll
        for (int j = 0; j < kPieces; ++j)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                         ::"r"((uint32_t)__cvta_generic_to_shared(place(d, t, i) + j * kThreads)),
                         "l"(reinterpret_cast<const uint4 *>(src) + j) : "memory");
    };
    auto fetch = [&](long long row, int d) {
        if (row < rows) {
#pragma unroll
            for (int i = 0; i < kBwdVec; ++i) {
                const int e = v0 + 32 * kWarps * i;
                if (e < vecs) {
                    copy(d, 0, i, h + row * cols + 8 * e);
                    copy(d, 1, i, dy + row * cols + 8 * e);
                    if (dsum) copy(d, 2, i, dsum + row * cols + 8 * e);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto take = [&](int d, int t, int i, float2 (&v)[4]) {
        Raw8<T> r;
#pragma unroll
        for (int j = 0; j < kPieces; ++j) r.r[j] = place(d, t, i)[j * kThreads];
        r.get(v);
    };
    const long long stride = (long long)gridDim.x * kRows;
    long long row = (long long)blockIdx.x * kRows + slot;
#pragma unroll
    for (int d = 0; d < kDepth; ++d) fetch(row + d * stride, d);
    float m = 0.0f, s = 0.0f;
    if (row < rows) {
        m = mean[row];
        s = rstd[row];
    }
    int d = 0;
    for (int it = 0; row < rows; row += stride, it ^= 1) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
        float2 z[kBwdVec][4], a[kBwdVec][4], sv[kBwdVec][4];
        const float rs_row = s;
        // (h - m) s: the difference first, which is exact where it matters
        const float2 s2 = make_float2(s, s), m2 = make_float2(-m, -m);
        float2 sa2 = zero, saz2 = zero;
#pragma unroll
        for (int i = 0; i < kBwdVec; ++i) {
#pragma unroll
            for (int q = 0; q < 4; ++q) z[i][q] = a[i][q] = sv[i][q] = zero;
            if (v0 + 32 * kWarps * i >= vecs) continue;
            take(d, 0, i, z[i]);
            take(d, 1, i, a[i]);
            if (dsum) take(d, 2, i, sv[i]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                z[i][q] = tc::mul2(tc::fma2(z[i][q], one, m2), s2);
                dg[i][q] = tc::fma2(a[i][q], z[i][q], dg[i][q]);
                db[i][q] = tc::fma2(a[i][q], one, db[i][q]);
                a[i][q] = tc::mul2(a[i][q], g[i][q]);
                sa2 = tc::fma2(a[i][q], one, sa2);
                saz2 = tc::fma2(a[i][q], z[i][q], saz2);
            }
        }
        float sa = sa2.x + sa2.y, saz = saz2.x + saz2.y;
        fetch(row + kDepth * stride, d);   // (this row's values have been read)
        d = d + 1 == kDepth ? 0 : d + 1;
        if (row + stride < rows) {
            m = mean[row + stride];
            s = rstd[row + stride];
        }
        sa = warp_sum(sa);
        saz = warp_sum(saz);
        if constexpr (kWarps > 1) {
            // (two buffers: a warp may be one row ahead of the slowest reader)
            if (lane == 0) red[it][slot][rw] = make_float2(sa, saz);
            row_sync<kWarps>(slot);
            sa = saz = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 q = red[it][slot][w];
                sa += q.x;
                saz += q.y;
            }
        }
        sa *= inv_cols;
        saz *= inv_cols;
#pragma unroll
        for (int i = 0; i < kBwdVec; ++i) {
            const int e = v0 + 32 * kWarps * i;
            if (e >= vecs) continue;
            float o[8];
            const float2 sa_2 = make_float2(-sa, -sa), saz_2 = make_float2(-saz, -saz), rs_2 = make_float2(rs_row, rs_row);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 v = tc::fma2(tc::fma2(z[i][q], saz_2, tc::fma2(a[i][q], one, sa_2)), rs_2, sv[i][q]);
                o[2 * q] = v.x;
                o[2 * q + 1] = v.y;
            }
            Vec8<T>::store(dx + row * cols + 8 * e, o);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    float *joined = reinterpret_cast<float *>(ring);   // [kRows - 1][2][cols]
    __syncthreads();
    if constexpr (kRows > 1) {
        if (slot > 0) {
            float *j = joined + (size_t)(slot - 1) * 2 * cols;
#pragma unroll
            for (int i = 0; i < kBwdVec; ++i) {
                const int e = v0 + 32 * kWarps * i;
                if (e < vecs) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        *reinterpret_cast<float2 *>(j + 8 * e + 2 * q) = dg[i][q];
                        *reinterpret_cast<float2 *>(j + cols + 8 * e + 2 * q) = db[i][q];
                    }
                }
            }
        }
        __syncthreads();
        if (slot > 0) return;
        for (int k = 0; k < kRows - 1; ++k) {
            const float *j = joined + (size_t)k * 2 * cols;
#pragma unroll
            for (int i = 0; i < kBwdVec; ++i) {
                const int e = v0 + 32 * kWarps * i;
                if (e >= vecs) continue;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    dg[i][q] = tc::fma2(*reinterpret_cast<const float2 *>(j + 8 * e + 2 * q), one, dg[i][q]);
                    db[i][q] = tc::fma2(*reinterpret_cast<const float2 *>(j + cols + 8 * e + 2 * q), one, db[i][q]);
                }
            }
        }
    }
    float *out = part + (size_t)blockIdx.x * 2 * cols;
#pragma unroll
    for (int i = 0; i < kBwdVec; ++i) {
        const int e = v0 + 32 * kWarps * i;
        if (e < vecs) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                *reinterpret_cast<float2 *>(out + 8 * e + 2 * q) = dg[i][q];
                *reinterpret_cast<float2 *>(out + cols + 8 * e + 2 * q) = db[i][q];
            }
        }
    }
}

// dg / db = sum over the partial rows.  A CTA owns 32 columns; its 32 warps
// take every 32nd partial row, then join in order.
constexpr int kJoinWarps = 32;

__global__ void __launch_bounds__(32 * kJoinWarps)
layer_norm_join_kernel(const float *__restrict__ part, float *__restrict__ dgamma, float *__restrict__ dbeta,
                       int nparts, int cols)
{
    // (a programmatic launch: the partial rows are complete after this)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float sums[kJoinWarps][33];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * 32 + lane;
    const int which = blockIdx.y;   // 0: dgamma, 1: dbeta
    float acc = 0.0f;
    if (c < cols) {
        const float *p = part + (size_t)which * cols + c;
#pragma unroll 8
        for (int r = warp; r < nparts; r += kJoinWarps) acc += p[(size_t)r * 2 * cols];
    }
    sums[warp][lane] = acc;
    __syncthreads();
    if (warp == 0 && c < cols) {
        acc = 0.0f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) acc += sums[w][lane];
        (which ? dbeta : dgamma)[c] = acc;
    }
}

namespace {

// Warps per row: the fewest (a power of two) that hold the row at `vec`
// vectors a thread.
int warps_per_row(int cols, int vec)
{
    int w = 1;
    while (w * 32 * vec * 8 < cols) w *= 2;
    return w;
}

// CTAs of the backward pass: what the SMs hold (two of 256 threads, one of
// 512), fewer where there are fewer rows.
int bwd_ctas(long long rows, int cols)
{
    const int w = warps_per_row(cols, kBwdVec);
    const int per = norm_threads(w) / (32 * w), most = 148 * (w > 8 ? 1 : 2);
    const long long need = (rows + per - 1) / per;
    return (int)(need < most ? need : most);
}

template <typename T, int kWarps>
cudaError_t launch_fwd(const NormProblem &q, cudaStream_t stream)
{
    constexpr int kRows = norm_threads(kWarps) / (32 * kWarps);
    const long long ctas = (q.rows + kRows - 1) / kRows;
    layer_norm_kernel<T, kWarps><<<(unsigned)ctas, norm_threads(kWarps), 0, stream>>>(
        static_cast<const T *>(q.x), static_cast<const T *>(q.residual), q.gamma, q.beta, static_cast<T *>(q.y),
        static_cast<T *>(q.sum_out), q.mean, q.rstd, q.rows, q.cols, q.eps);
    return cudaGetLastError();
}

template <typename T, int kWarps>
cudaError_t launch_bwd(const NormBackwardProblem &q, cudaStream_t stream)
{
    constexpr int kRows = norm_threads(kWarps) / (32 * kWarps);
    const int ctas = bwd_ctas(q.rows, q.cols);
    // (the rows that join need at most 28 KB of it)
    constexpr size_t smem = ring_bytes<T>(norm_threads(kWarps));
    static_assert((size_t)(kRows - 1) * 2 * 256 * kWarps * kBwdVec * sizeof(float) <= smem, "join");
    float *part = static_cast<float *>(q.workspace);
    cudaError_t e = cudaFuncSetAttribute(layer_norm_bwd_kernel<T, kWarps>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (ctas > 0) {   // (no rows: the sums are empty)
        layer_norm_bwd_kernel<T, kWarps><<<ctas, norm_threads(kWarps), smem, stream>>>(
            static_cast<const T *>(q.dy), static_cast<const T *>(q.h), q.gamma, q.mean, q.rstd,
            static_cast<const T *>(q.dsum), static_cast<T *>(q.dx), part, q.rows, q.cols);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        count_launch();
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((q.cols + 31) / 32, q.dbeta ? 2 : 1);
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 0 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, layer_norm_join_kernel, static_cast<const float *>(part), q.dgamma, q.dbeta, ctas,
                              q.cols);
}

}  // namespace

bool layer_norm_supported(long long rows, int cols)
{
    return cols % 8 == 0 && cols <= 8192 && rows <= (1ll << 31) - 1;
}

size_t layer_norm_backward_ws_bytes(long long rows, int cols)
{
    return (size_t)bwd_ctas(rows, cols) * 2 * cols * sizeof(float);
}

template <typename T>
cudaError_t launch_layer_norm(const NormProblem &q, cudaStream_t stream)
{
    cudaError_t e;
    switch (warps_per_row(q.cols, kFwdVec)) {
    case 1: e = launch_fwd<T, 1>(q, stream); break;
    case 2: e = launch_fwd<T, 2>(q, stream); break;
    case 4: e = launch_fwd<T, 4>(q, stream); break;
    default: e = launch_fwd<T, 8>(q, stream); break;
    }
    if (e == cudaSuccess) count_launch();
    return e;
}

template <typename T>
cudaError_t launch_layer_norm_backward(const NormBackwardProblem &q, cudaStream_t stream)
{
    cudaError_t e;
    switch (warps_per_row(q.cols, kBwdVec)) {
    case 1: e = launch_bwd<T, 1>(q, stream); break;
    case 2: e = launch_bwd<T, 2>(q, stream); break;
    case 4: e = launch_bwd<T, 4>(q, stream); break;
    case 8: e = launch_bwd<T, 8>(q, stream); break;
    default: e = launch_bwd<T, 16>(q, stream); break;
    }
    if (e == cudaSuccess) count_launch();
    return e;
}

template cudaError_t launch_layer_norm<float>(const NormProblem &, cudaStream_t);
template cudaError_t launch_layer_norm<__nv_bfloat16>(const NormProblem &, cudaStream_t);
template cudaError_t launch_layer_norm_backward<float>(const NormBackwardProblem &, cudaStream_t);
template cudaError_t launch_layer_norm_backward<__nv_bfloat16>(const NormBackwardProblem &, cudaStream_t);

}  // namespace bimamba
