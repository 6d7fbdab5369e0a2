// Short causal convolution of a selective state-space layer: token-major rows
// [B, N, D], one filter of w taps per channel, optional bias and SiLU, and a
// cache of the last w-1 inputs.
//
// Per sequence and channel, with xh = [cache (w-1 rows); x]:
//     y_t[c] = act(bias[c] + sum_{i=0}^{w-1} W[c][i] * xh[t + i][c])
// and the new cache is the last w-1 rows of xh.  act is the identity or
// silu(y) = y / (1 + e^-y).
//
// Memory-bound: one read of x and one write of y.  A thread owns V channels (4,
// accesses of 8 bytes in bf16 and 16 in fp32; 1 where rows do not start on that
// or D is no multiple of it).  Threads are numbered channel groups first, so a
// warp reads 256 or 512 consecutive bytes of a row.  Arithmetic is fp32 FMA in tap
// order from the bias up, rounded to the storage type once.
//
// Prompts: a thread walks a run of tokens and keeps w-1 unfinished outputs
// instead of a window of inputs: each row is converted once and added to the w
// outputs it belongs to, in the order of their taps.  Copies into the thread's own
// slots of shared memory keep 12 to 16 rows of it in flight without registers.  One
// token a sequence: a thread takes several sequences, so that the filter, larger
// than a token's rows, is loaded once for them.
//
// At 32768 tokens x 4096 channels, bf16, 4 taps, bias and SiLU the prompt kernel
// takes 94 us (5.7 TB/s; 82 us at the copy rate): issue slots are 60 % busy and the
// rest is waiting between dependent steps.  With the rows in flight held in
// registers it was 120; runs of 64 and 32 tokens: 97 and 108; rings of 8, 12 and 32
// rows: 105, 100 and 105; two CTAs an SM instead of three: 112, four: 114 (but from
// five taps on, where three spill, two are faster: eight taps 76 against 144 us at
// half the tokens); 8 channels a thread and two CTAs: 104.  One token of 256 sequences
// takes 4.3 us on the GPU.  fp32, 16384 x 4096: 92 us (5.9 TB/s).  Rows that allow one
// channel a thread only: 32768 x 4095 bf16 188 us, 16384 x 4095 fp32 124 us.
#include "f32x2.cuh"
#include "la_internal.cuh"
#include "sm100.cuh"

namespace la {
namespace {

using namespace sm100;

constexpr int kThreads = 256;
constexpr int kHalf = 4;    // rows of a half-batch, or of a group of copies
constexpr int kGroups = 4;  // groups of a thread's ring
constexpr int kSeqs = 4;    // sequences a thread takes where each has one token

struct Lens {
    int use;
    int n[kMaxSeqLens];
};

template <typename T, int V> struct Row;
template <> struct Row<__nv_bfloat16, 4> { uint2 a; };
template <> struct Row<float, 4> { float4 a; };
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

// bf16 rounding hides the shorter form's error
template <typename T> __device__ __forceinline__ float silu(float y);
template <> __device__ __forceinline__ float silu<float>(float y) { return silu_f32(y); }
template <> __device__ __forceinline__ float silu<__nv_bfloat16>(float y) { return silu_approx(y); }

// V channels' filters [V][W] and biases
template <int W, int V>
__device__ __forceinline__ void load_filter(const float* __restrict__ weight, const float* __restrict__ bias, int c0,
                                            float (&wt)[W][V], float (&b0)[V])
{
#pragma unroll
    for (int j = 0; j < V; ++j) b0[j] = bias ? bias[c0 + j] : 0.f;
    if (V > 1) {
        float4 raw[V > 1 ? V * W / 4 : 1];
        const float4* wp = reinterpret_cast<const float4*>(weight + (size_t)c0 * W);
#pragma unroll
        for (int i = 0; i < V * W / 4; ++i) raw[i] = wp[i];
        const float* wf = reinterpret_cast<const float*>(raw);
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < W; ++i) wt[i][j] = wf[j * W + i];
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) wt[i][0] = weight[(size_t)c0 * W + i];
    }
}

// BYTES (4, 8 or 16) from global to shared memory in the background, or zeros
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool on)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES),
                 "r"(on ? BYTES : 0)
                 : "memory");
}

// One thread: V channels of `run` consecutive tokens of one sequence (run a
// multiple of 2 kHalf, so that runs but the first start past the cache's reach).
template <typename T, int W, int V>
__global__ void __launch_bounds__(kThreads, W > 4 ? 2 : 3)
ssm_conv_kernel(const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias,
                const T* cache, T* __restrict__ y, T* cache_out, const __grid_constant__ Lens lens, int N, int D,
                int groups, int runs, int run, long long total, long long xb, long long xt, int act)
{
    constexpr int HIST = W - 1;
    static_assert(2 * kHalf >= HIST, "only the first run reads the cache");
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (id >= total) return;
    const int cg = (int)(id % groups);
    const long long r = id / groups;
    const int b = (int)(r / runs);
    const int len = lens.use ? lens.n[b] : N;
    const int c0 = cg * V;
    const int t0 = (int)(r % runs) * run, t1 = min(len, t0 + run);
    const T* xc = x + b * xb + c0;
    const T* cc = cache ? cache + (size_t)b * HIST * D + c0 : nullptr;

    // row k of [cache; x]; rows past the sequence are not read
    auto fetch = [&](int k) {
        if (k >= HIST) return k - HIST < len ? row_load<T, V>(xc + (k - HIST) * xt) : row_zero<T, V>();
        return cc ? row_load<T, V>(cc + (size_t)k * D) : row_zero<T, V>();
    };
    Row<T, V> tail[HIST > 0 ? HIST : 1];
    const bool keeper = HIST > 0 && cache_out && t0 == 0;
    if (t0 < t1) {
        Row<T, V> past[HIST > 0 ? HIST : 1];
#pragma unroll
        for (int i = 0; i < HIST; ++i) past[i] = fetch(t0 + i);
        // a wide row goes through the thread's own slots of a ring in shared memory, kGroups groups of
        // rows ahead; no other thread reads them, so a thread waits for its own copies only.  A narrow one
        // (2 bytes are no size of a copy) stays in registers, two half-batches.
        constexpr bool RING = V > 1;
        extern __shared__ __align__(16) char ring_bytes[];
        Row<T, V>* const ring = reinterpret_cast<Row<T, V>*>(ring_bytes) + threadIdx.x;
        Row<T, V> rows[2][kHalf];
        const T* xp = xc + t0 * xt;
        int tn = t0;
        auto bring = [&](int g) {
            if (tn < t1) {
#pragma unroll
                for (int u = 0; u < kHalf; ++u) {
                    copy_async<(int)sizeof(Row<T, V>)>(ring + (g * kHalf + u) * kThreads, tn + u < t1 ? xp : xc,
                                                       tn + u < t1);
                    xp += xt;
                }
                tn += kHalf;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        if constexpr (RING) {
#pragma unroll 1
            for (int g = 0; g < kGroups; ++g) bring(g);
        } else {
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int u = 0; u < kHalf; ++u) rows[a][u] = fetch(t0 + HIST + a * kHalf + u);
        }
        float wt[W][V], b0[V];
        load_filter<W, V>(weight, bias, c0, wt, b0);
        // pairs of channels go through packed FMAs: half the issue slots
        constexpr int VP = (V + 1) / 2;
        f2 w2[W][VP], b2[VP], acc[W][VP];      // acc[k]: the output k tokens ahead of the next row
#pragma unroll
        for (int j = 0; j < VP; ++j) {
            b2[j] = pack2(b0[2 * j], V > 1 ? b0[2 * j + (V > 1)] : 0.f);
#pragma unroll
            for (int k = 0; k < W; ++k) {
                w2[k][j] = pack2(wt[k][2 * j], V > 1 ? wt[k][2 * j + (V > 1)] : 0.f);
                acc[k][j] = b2[j];
            }
        }
        auto add = [&](const Row<T, V>& row) {
            float f[V];
            row_f32<T, V>(row, f);
#pragma unroll
            for (int j = 0; j < VP; ++j) {
                const f2 x2 = pack2(f[2 * j], V > 1 ? f[2 * j + (V > 1)] : 0.f);
#pragma unroll
                for (int k = 0; k < W; ++k) acc[k][j] = fma2(w2[W - 1 - k][j], x2, acc[k][j]);
            }
        };
        auto shift = [&]() {
#pragma unroll
            for (int j = 0; j < VP; ++j) {
#pragma unroll
                for (int k = 0; k + 1 < W; ++k) acc[k][j] = acc[k + 1][j];
                acc[W - 1][j] = b2[j];
            }
        };
        // the history: row t0 + i is tap i of the first output (acc[0] after HIST shifts)
#pragma unroll
        for (int i = 0; i < HIST; ++i) {
            add(past[i]);
            shift();
        }
        T* yp = y + ((size_t)b * N + t0) * D + c0;
        auto emit = [&](const Row<T, V>& row, bool on) {
            add(row);
            float out[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float2 q = unpack2(acc[0][j / 2]);
                const float y1 = j % 2 ? q.y : q.x;
                out[j] = act ? silu<T>(y1) : y1;
            }
            if (on) row_store<T, V>(yp, out);
            yp += D;
            shift();
        };
        if constexpr (RING) {
            int g = 0;
#pragma unroll 1
            for (int t = t0; t < t1; t += kHalf) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kGroups - 1) : "memory");
#pragma unroll
                for (int u = 0; u < kHalf; ++u) emit(ring[(g * kHalf + u) * kThreads], t + u < t1);
                bring(g);
                if (++g == kGroups) g = 0;
            }
        } else {
            for (int t = t0; t < t1; t += 2 * kHalf) {
#pragma unroll
                for (int a = 0; a < 2; ++a) {
#pragma unroll
                    for (int u = 0; u < kHalf; ++u) emit(rows[a][u], t + a * kHalf + u < t1);
                    if (t + 2 * kHalf < t1) {
#pragma unroll
                        for (int u = 0; u < kHalf; ++u) rows[a][u] = fetch(t + 2 * kHalf + HIST + a * kHalf + u);
                    }
                }
            }
        }
    }
    // every cache row this sequence's channels need is read by this thread alone,
    // before it writes: cache_out may be the cache itself
    if (keeper) {
#pragma unroll
        for (int i = 0; i < HIST; ++i) tail[i] = fetch(len + i);
#pragma unroll
        for (int i = 0; i < HIST; ++i)
            *reinterpret_cast<Row<T, V>*>(cache_out + ((size_t)b * HIST + i) * D + c0) = tail[i];
    }
}

// N = 1.  One thread: V channels of kSeqs sequences.  Two CTAs an SM: three spill the
// rows of longer filters (fp32, four taps, 256 sequences: 8.0 against 5.9 us).
template <typename T, int W, int V>
__global__ void __launch_bounds__(kThreads, 2)
ssm_conv_token_kernel(const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias,
                      const T* cache, T* __restrict__ y, T* cache_out, const __grid_constant__ Lens lens, int B, int D,
                      int groups, int seqs, long long total, long long xb, int act)
{
    constexpr int HIST = W - 1;
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (id >= total) return;
    const int c0 = (int)(id % groups) * V;
    const int b0 = (int)(id / groups) * seqs, nb = min(seqs, B - b0);
    Row<T, V> row[kSeqs][W];
#pragma unroll
    for (int s = 0; s < kSeqs; ++s) {
#pragma unroll
        for (int i = 0; i < HIST; ++i)
            row[s][i] = s < nb && cache ? row_load<T, V>(cache + ((size_t)(b0 + s) * HIST + i) * D + c0) : row_zero<T, V>();
        const bool on = s < nb && !(lens.use && lens.n[b0 + s] == 0);
        row[s][HIST] = on ? row_load<T, V>(x + (b0 + s) * xb + c0) : row_zero<T, V>();
    }
    float wt[W][V], bs[V];
    load_filter<W, V>(weight, bias, c0, wt, bs);
#pragma unroll
    for (int s = 0; s < kSeqs; ++s) {
        if (s >= nb) break;
        const bool on = !(lens.use && lens.n[b0 + s] == 0);
        if (on) {
            float acc[V];
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] = bs[j];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                float f[V];
                row_f32<T, V>(row[s][i], f);
#pragma unroll
                for (int j = 0; j < V; ++j) acc[j] = fmaf(wt[i][j], f[j], acc[j]);
            }
            if (act) {
#pragma unroll
                for (int j = 0; j < V; ++j) acc[j] = silu<T>(acc[j]);
            }
            row_store<T, V>(y + (size_t)(b0 + s) * D + c0, acc);
        }
        if (cache_out) {
#pragma unroll
            for (int i = 0; i < HIST; ++i)
                *reinterpret_cast<Row<T, V>*>(cache_out + ((size_t)(b0 + s) * HIST + i) * D + c0) = on ? row[s][i + 1] : row[s][i];
        }
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
    if (a.N == 1) {
        // several sequences a thread once there are threads for every SM without that
        const int seqs = (long long)a.B * groups >= 148ll * 512 ? kSeqs : 1;
        const long long total = (long long)((a.B + seqs - 1) / seqs) * groups;
        const long long grid = (total + kThreads - 1) / kThreads;
        if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
        ssm_conv_token_kernel<T, W, V><<<(unsigned)grid, kThreads, 0, a.stream>>>(
            (const T*)a.x, a.weight, a.bias, (const T*)a.cache, (T*)a.out, (T*)a.cache_out, lens, a.B, a.D, groups, seqs,
            total, a.x_batch, a.silu);
        return cudaGetLastError();
    }
    // tokens a thread takes: longer runs re-read fewer rows of the history, but
    // threads for two waves of every SM have to be left
    int run = 128;
    while (run > 2 * kHalf && (long long)a.B * groups * ((a.N + run - 1) / run) < 2 * 148ll * 512) run /= 2;
    const int runs = a.N > 0 ? (a.N + run - 1) / run : 1;
    const long long total = (long long)a.B * groups * runs;
    const long long grid = (total + kThreads - 1) / kThreads;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    auto kern = ssm_conv_kernel<T, W, V>;
    constexpr int SMEM = V > 1 ? kGroups * kHalf * kThreads * (int)sizeof(Row<T, V>) : 0;
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (err != cudaSuccess) return err;
    kern<<<(unsigned)grid, kThreads, SMEM, a.stream>>>(
        (const T*)a.x, a.weight, a.bias, (const T*)a.cache, (T*)a.out, (T*)a.cache_out, lens, a.N, a.D, groups, runs, run,
        total, a.x_batch, a.x_row, a.silu);
    return cudaGetLastError();
}

template <typename T, int W>
cudaError_t launch_w(const SsmConvArgs& a)
{
    constexpr int V = 4;   // channels of a wide thread
    constexpr int BYTES = V * (int)sizeof(T);
    auto on = [](const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
    const bool wide = a.D % V == 0 && on(a.x, BYTES) && on(a.weight, 16) && on(a.cache, BYTES) && on(a.out, BYTES) &&
                      on(a.cache_out, BYTES) && a.x_batch % V == 0 && a.x_row % V == 0;
    return wide ? launch_v<T, W, V>(a) : launch_v<T, W, 1>(a);
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
