// Short causal convolution of a selective state-space layer: token-major rows
// [B, N, D], one filter of w taps per channel, optional bias and SiLU, and a
// cache of the last w-1 inputs.
//
// Per sequence and channel, with xh = [cache (w-1 rows); x]:
//     y_t[c] = act(bias[c] + sum_{i=0}^{w-1} W[c][i] * xh[t + i][c])
// and the new cache is the last w-1 rows of xh.  act is the identity or
// silu(y) = y / (1 + e^-y).
//
// Memory-bound: one read of x and one write of y.  A thread owns V channels
// (8 as 16-byte accesses, or 1 where a row does not start on 16 bytes or D is
// no multiple of 8) of a run of consecutive tokens, which it takes in batches
// of kBatch rows: the window of the last w-1 rows stays in registers from
// batch to batch, and a batch's rows are requested before the previous batch
// is computed.  Threads are numbered channel groups first, so a warp reads 512
// consecutive bytes of a row.  Arithmetic is fp32 FMA in tap order from the
// bias up, rounded to the storage type once.
#include "la_internal.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;   // tokens whose rows are in flight at once; at least w-1, so only run 0 reads the cache

struct Lens {
    int use;
    int n[kMaxSeqLens];
};

template <typename T, int V> struct Row;
template <> struct Row<__nv_bfloat16, 8> { uint4 a; };
template <> struct Row<float, 8> { float4 a, b; };
template <> struct Row<__nv_bfloat16, 1> { __nv_bfloat16 a; };
template <> struct Row<float, 1> { float a; };

template <typename T, int V>
__device__ __forceinline__ Row<T, V> row_load(const T* p) { return *reinterpret_cast<const Row<T, V>*>(p); }
template <typename T, int V>
__device__ __forceinline__ Row<T, V> row_zero()
{
    Row<T, V> r;
    memset(&r, 0, sizeof(r));
    return r;
}
template <typename T, int V>
__device__ __forceinline__ void row_f32(const Row<T, V>& r, float (&f)[V])
{
    const T* e = reinterpret_cast<const T*>(&r);
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = to_f32<T>(e[j]);
}
template <typename T, int V>
__device__ __forceinline__ void row_store(T* p, const float (&f)[V])
{
    Row<T, V> r;
    T* e = reinterpret_cast<T*>(&r);
#pragma unroll
    for (int j = 0; j < V; ++j) e[j] = from_f32<T>(f[j]);
    *reinterpret_cast<Row<T, V>*>(p) = r;
}

// fp32 outputs take the accurate exponential; bf16 rounding hides the fast one's error
template <typename T> __device__ __forceinline__ float silu(float y);
template <> __device__ __forceinline__ float silu<float>(float y) { return y / (1.f + expf(-y)); }
template <> __device__ __forceinline__ float silu<__nv_bfloat16>(float y) { return __fdividef(y, 1.f + __expf(-y)); }

// One thread: V channels of `batches` * kBatch consecutive tokens of one sequence.
template <typename T, int W, int V>
__global__ void __launch_bounds__(kThreads)
ssm_conv_kernel(const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias,
                const T* cache, T* __restrict__ y, T* cache_out, const __grid_constant__ Lens lens, int N, int D,
                int groups, int runs, int batches, long long total, long long xb, long long xt, int act)
{
    constexpr int HIST = W - 1;
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (id >= total) return;
    const int cg = (int)(id % groups);
    const long long r = id / groups;
    const int run = (int)(r % runs), b = (int)(r / runs);
    const int len = lens.use ? lens.n[b] : N;
    const int c0 = cg * V;
    const int t0 = run * batches * kBatch, t1 = min(len, t0 + batches * kBatch);
    const T* xc = x + b * xb + c0;
    const T* cc = cache ? cache + (size_t)b * HIST * D + c0 : nullptr;
    T* yc = y + (size_t)b * N * D + c0;

    // row k of [cache; x]; rows past the sequence are not read
    auto fetch = [&](int k) {
        if (k >= HIST) return k - HIST < len ? row_load<T, V>(xc + (k - HIST) * xt) : row_zero<T, V>();
        return cc ? row_load<T, V>(cc + (size_t)k * D) : row_zero<T, V>();
    };

    Row<T, V> tail[HIST > 0 ? HIST : 1];
    const bool keeper = cache_out && run == 0;
    if (HIST > 0 && keeper) {
#pragma unroll
        for (int i = 0; i < HIST; ++i) tail[i] = fetch(len + i);
    }
    if (t0 < t1) {
        float wt[W][V], b0[V], win[W][V];
#pragma unroll
        for (int j = 0; j < V; ++j) b0[j] = bias ? bias[c0 + j] : 0.f;
        if (V == 8) {
            float4 raw[2 * W];
            const float4* wp = reinterpret_cast<const float4*>(weight + (size_t)c0 * W);
#pragma unroll
            for (int i = 0; i < 2 * W; ++i) raw[i] = wp[i];
            const float* wf = reinterpret_cast<const float*>(raw);
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int i = 0; i < W; ++i) wt[i][j] = wf[j * W + i];
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) wt[i][0] = weight[(size_t)c0 * W + i];
        }
        Row<T, V> next[kBatch];
#pragma unroll
        for (int i = 0; i < HIST; ++i) row_f32<T, V>(fetch(t0 + i), win[i]);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) next[u] = fetch(t0 + HIST + u);
        for (int t = t0; t < t1; t += kBatch) {
            Row<T, V> rows[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) rows[u] = next[u];
            if (t + kBatch < t1) {
#pragma unroll
                for (int u = 0; u < kBatch; ++u) next[u] = fetch(t + kBatch + HIST + u);
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                row_f32<T, V>(rows[u], win[HIST]);
                float acc[V];
#pragma unroll
                for (int j = 0; j < V; ++j) acc[j] = b0[j];
#pragma unroll
                for (int i = 0; i < W; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) acc[j] = fmaf(wt[i][j], win[i][j], acc[j]);
                if (act) {
#pragma unroll
                    for (int j = 0; j < V; ++j) acc[j] = silu<T>(acc[j]);
                }
                if (t + u < t1) row_store<T, V>(yc + (size_t)(t + u) * D, acc);
#pragma unroll
                for (int i = 0; i < HIST; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) win[i][j] = win[i + 1][j];
            }
        }
    }
    // every cache row this sequence's channels need has been read by this thread:
    // cache_out may be the cache itself
    if (HIST > 0 && keeper) {
#pragma unroll
        for (int i = 0; i < HIST; ++i)
            *reinterpret_cast<Row<T, V>*>(cache_out + ((size_t)b * HIST + i) * D + c0) = tail[i];
    }
}

template <typename T, int W, int V>
cudaError_t launch_v(const SsmConvArgs& a)
{
    const int groups = a.D / V;
    Lens lens{};
    lens.use = a.seq_lens != nullptr;
    if (a.seq_lens)
        for (int b = 0; b < a.B; ++b) lens.n[b] = a.seq_lens[b];
    // tokens a thread takes: longer runs re-read fewer rows of the window, but
    // about 148 * 2048 threads have to be left to fill the GPU
    int batches = 4;
    while (batches > 1 && (long long)a.B * groups * ((a.N + batches * kBatch - 1) / (batches * kBatch)) < 148ll * 2048)
        batches /= 2;
    const int run = batches * kBatch;
    const int runs = a.N > 0 ? (a.N + run - 1) / run : 1;
    const long long total = (long long)a.B * groups * runs;
    const long long grid = (total + kThreads - 1) / kThreads;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    ssm_conv_kernel<T, W, V><<<(unsigned)grid, kThreads, 0, a.stream>>>(
        (const T*)a.x, a.weight, a.bias, (const T*)a.cache, (T*)a.out, (T*)a.cache_out, lens, a.N, a.D, groups, runs,
        batches, total, a.x_batch, a.x_row, a.silu);
    return cudaGetLastError();
}

template <typename T, int W>
cudaError_t launch_w(const SsmConvArgs& a)
{
    auto on16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    const long long e = sizeof(T);
    const bool wide = a.D % 8 == 0 && on16(a.x) && on16(a.weight) && on16(a.cache) && on16(a.out) &&
                      on16(a.cache_out) && a.x_batch * e % 16 == 0 && a.x_row * e % 16 == 0;
    return wide ? launch_v<T, W, 8>(a) : launch_v<T, W, 1>(a);
}

template <typename T>
cudaError_t launch_t(const SsmConvArgs& a)
{
    switch (a.w) {
        case 1: return launch_w<T, 1>(a);
        case 2: return launch_w<T, 2>(a);
        case 3: return launch_w<T, 3>(a);
        case 4: return launch_w<T, 4>(a);
        case 5: return launch_w<T, 5>(a);
        case 6: return launch_w<T, 6>(a);
        case 7: return launch_w<T, 7>(a);
        case 8: return launch_w<T, 8>(a);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_ssm_conv(const SsmConvArgs& a)
{
    return a.dtype == LA_BF16 ? launch_t<__nv_bfloat16>(a) : launch_t<float>(a);
}

}  // namespace la
