// Sliding-window attention with sinks, prompts, fp32 arithmetic on the CUDA
// cores (fp32 inputs; a tensor-core operand would round them), and the kernel
// that moves a prompt's last tokens into the rolling cache.
//
//     o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i.k_j - m_i)
// over the visible keys, in one pass over the key tiles with a running maximum
// m_i and sum.  A CTA takes 64 queries of one head; a thread holds 4 x 4 scores
// and 4 rows of dv / 16 output columns in registers, so each 16-byte read of
// shared memory feeds 8 (scores) to 16 (outputs) FMAs.
// A 16384-token prompt (32 heads of 128, window 4096) takes 39.5 ms: 24 TFLOP/s, a
// third of the FMA pipe's 73.  Its 119 KB of shared memory leave one CTA, two
// warps a scheduler, which do not cover the waits for key tiles (no loads ahead),
// shared-memory reads and barriers: issue slots are 45 % busy, the FMA pipe 35 %.
#include <algorithm>

#include "la_window.cuh"

namespace la {
namespace {

constexpr int kT = 64;          // queries and keys of a tile
constexpr int kThreads = 256;   // 16 x 16
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int DV>
struct Plan {
    static constexpr int QP = D + 4, VP = DV + 4, PP = kT + 4;   // row pitches (fp32): neighbouring rows on other banks
    static constexpr int OFF_K = kT * QP, OFF_V = OFF_K + kT * QP, OFF_P = OFF_V + kT * VP;
    static constexpr int BYTES = (OFF_P + kT * PP) * 4;
};

// grid: (query tiles, heads, sequences)
template <int D, int DV>
__global__ void __launch_bounds__(kThreads)
window_prefill_simt(const __grid_constant__ WindowArgs a, const __grid_constant__ WindowLens lens)
{
    using P = Plan<D, DV>;
    extern __shared__ __align__(16) float smf[];
    float *Qs = smf, *Ks = smf + P::OFF_K, *Vs = smf + P::OFF_V, *Ps = smf + P::OFF_P;
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    const int b = blockIdx.z, h = blockIdx.y, kvh = h / (a.Hq / a.Hkv);
    const int len = lens.use ? lens.n[b] : a.N;
    const int start = a.pos ? a.pos[b] : 0;
    // the longest walks first: later queries see at least as many keys
    const int q0 = ((int)gridDim.x - 1 - (int)blockIdx.x) * kT;
    if (start < 0 || q0 >= len) return;
    const int q1 = min(len, q0 + kT);
    KeyWalk<kT> w;
    w.init(a.k_cache != nullptr, start, a.window, a.sinks, len, q0, q1);

    const float* qp = (const float*)a.q + b * a.st.q_batch + h * a.st.q_head;
    for (int e = tid; e < kT * (D / 4); e += kThreads) {
        const int r = e / (D / 4), c = e % (D / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (q0 + r < q1) x = *reinterpret_cast<const float4*>(qp + (q0 + r) * a.st.q_row + c);
        *reinterpret_cast<float4*>(Qs + r * P::QP + c) = x;
    }
    const size_t cap = (size_t)a.window + a.sinks;
    const size_t kv = (size_t)b * a.Hkv + kvh;
    const float sl = a.scale * kLog2e;
    float m[4], l[4], o[4][DV / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < DV / 16; ++c) o[i][c] = 0.f;
    }
    const int tiles = w.count();
    for (int it = 0; it < tiles; ++it) {
        const bool old = w.is_cache(it);
        const int base = w.base(it);
        const float* kp = old ? (const float*)a.k_cache + (kv * cap) * D : (const float*)a.k + b * a.st.k_batch + kvh * a.st.k_head;
        const float* vp = old ? (const float*)a.v_cache + (kv * cap) * DV : (const float*)a.v + b * a.st.v_batch + kvh * a.st.v_head;
        const long long ks = old ? D : a.st.k_row, vs = old ? DV : a.st.v_row;
        __syncthreads();
        // keys that hold nothing are zeros here: their bits never reach a product
        for (int e = tid; e < kT * (D / 4); e += kThreads) {
            const int r = e / (D / 4), c = e % (D / 4) * 4;
            const bool on = old ? w.slot_held(base + r) : base + r < len;
            *reinterpret_cast<float4*>(Ks + r * P::QP + c) =
                on ? *reinterpret_cast<const float4*>(kp + (base + r) * ks + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int e = tid; e < kT * (DV / 4); e += kThreads) {
            const int r = e / (DV / 4), c = e % (DV / 4) * 4;
            const bool on = old ? w.slot_held(base + r) : base + r < len;
            *reinterpret_cast<float4*>(Vs + r * P::VP + c) =
                on ? *reinterpret_cast<const float4*>(vp + (base + r) * vs + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        __syncthreads();
        float s[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
            float4 x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(Qs + (ty + 16 * i) * P::QP + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * j) * P::QP + c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[i][j] = fmaf(x[i].w, y[j].w, fmaf(x[i].z, y[j].z, fmaf(x[i].y, y[j].y, fmaf(x[i].x, y[j].x, s[i][j]))));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int qi = q0 + ty + 16 * i;
            float top = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = base + tx + 16 * j;
                const bool see = old ? w.sees_slot(qi, key) : w.sees_new(qi, key);
                s[i][j] = see ? s[i][j] * sl : -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
#pragma unroll
            for (int x = 8; x > 0; x /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
            // a row that has seen nothing yet keeps its zeros
            const float ref = top == -INFINITY ? 0.f : top;
            const float fade = exp2f(m[i] - ref);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(s[i][j] - ref);
                sum += p;
                Ps[(ty + 16 * i) * P::PP + tx + 16 * j] = p;
            }
            l[i] = fmaf(l[i], fade, sum);     // of this thread's keys; added over the row at the end
            m[i] = top;
#pragma unroll
            for (int c = 0; c < DV / 16; ++c) o[i][c] *= fade;
        }
        __syncthreads();
#pragma unroll 2
        for (int kk = 0; kk < kT; kk += 4) {
            float4 p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(Ps + (ty + 16 * i) * P::PP + kk);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
#pragma unroll
                for (int c = 0; c < DV / 64; ++c) {
                    const float4 y = *reinterpret_cast<const float4*>(Vs + (kk + x) * P::VP + c * 64 + tx * 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float pv = x == 0 ? p[i].x : x == 1 ? p[i].y : x == 2 ? p[i].z : p[i].w;
                        o[i][c * 4 + 0] = fmaf(pv, y.x, o[i][c * 4 + 0]);
                        o[i][c * 4 + 1] = fmaf(pv, y.y, o[i][c * 4 + 1]);
                        o[i][c * 4 + 2] = fmaf(pv, y.z, o[i][c * 4 + 2]);
                        o[i][c * 4 + 3] = fmaf(pv, y.w, o[i][c * 4 + 3]);
                    }
                }
            }
        }
    }
    float* op = (float*)a.out + b * a.st.out_batch + h * a.st.out_head;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float sum = l[i];
#pragma unroll
        for (int x = 8; x > 0; x /= 2) sum += __shfl_xor_sync(~0u, sum, x);
        const float inv = 1.f / sum;          // every query sees itself: the sum is at least its own term
        const int qi = q0 + ty + 16 * i;
        if (qi < q1) {
#pragma unroll
            for (int c = 0; c < DV / 64; ++c)
                *reinterpret_cast<float4*>(op + qi * a.st.out_row + c * 64 + tx * 4) =
                    make_float4(o[i][c * 4] * inv, o[i][c * 4 + 1] * inv, o[i][c * 4 + 2] * inv, o[i][c * 4 + 3] * inv);
        }
    }
}

template <int D, int DV>
cudaError_t launch_simt(const WindowArgs& a)
{
    using P = Plan<D, DV>;
    auto kern = window_prefill_simt<D, DV>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, P::BYTES);
    if (e != cudaSuccess) return e;
    kern<<<dim3((a.N + kT - 1) / kT, a.Hq, a.B), kThreads, P::BYTES, a.stream>>>(a, window_lens(a));
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// A prompt's tokens into the rolling cache: the sinks among them and the last
// `window` others.  One warp a (token, kv head, sequence), 16-byte copies.
constexpr int kCopyWarps = 8;

__global__ void __launch_bounds__(kCopyWarps * 32)
window_cache_update(const __grid_constant__ WindowArgs a, const __grid_constant__ WindowLens lens, int esize, int blocks)
{
    const int lane = threadIdx.x & 31, b = blockIdx.z, h = blockIdx.y;
    const int len = lens.use ? lens.n[b] : a.N;
    const int start = a.pos ? a.pos[b] : 0;
    if (start < 0) return;
    const int ns = start < a.sinks ? min(a.sinks - start, len) : 0;   // new tokens that are sinks
    const int first = max(ns, len - a.window);                        // first of the others that stays
    const int rows = ns + len - first;
    const size_t cap = (size_t)a.window + a.sinks, kv = (size_t)b * a.Hkv + h;
    const int dk = a.d * esize / 16, dvv = a.dv * esize / 16;         // 16-byte pieces of a row
    for (int r = blockIdx.x * kCopyWarps + (threadIdx.x >> 5); r < rows; r += blocks * kCopyWarps) {
        const int i = r < ns ? r : first + r - ns;
        const unsigned p = (unsigned)start + (unsigned)i;
        const size_t slot = p < (unsigned)a.sinks ? p : a.sinks + (p - a.sinks) % (unsigned)a.window;
        const char* ks = (const char*)a.k + (b * a.st.k_batch + h * a.st.k_head + i * a.st.k_row) * esize;
        const char* vs = (const char*)a.v + (b * a.st.v_batch + h * a.st.v_head + i * a.st.v_row) * esize;
        uint4* kd = (uint4*)((char*)a.k_cache + (kv * cap + slot) * a.d * esize);
        uint4* vd = (uint4*)((char*)a.v_cache + (kv * cap + slot) * a.dv * esize);
        if (lane < dk) kd[lane] = ((const uint4*)ks)[lane];
        if (lane < dvv) vd[lane] = ((const uint4*)vs)[lane];
    }
}

}  // namespace

cudaError_t launch_window_prefill_simt(const WindowArgs& a)
{
    if (a.d == 64) return a.dv == 64 ? launch_simt<64, 64>(a) : launch_simt<64, 128>(a);
    return a.dv == 64 ? launch_simt<128, 64>(a) : launch_simt<128, 128>(a);
}

cudaError_t launch_window_cache_update(const WindowArgs& a)
{
    const int esize = a.dtype == LA_BF16 ? 2 : 4;
    const long long rows = std::min<long long>(a.N, (long long)a.window + a.sinks);
    const int blocks = (int)std::min<long long>((rows + kCopyWarps - 1) / kCopyWarps, 4096);
    window_cache_update<<<dim3(blocks, a.Hkv, a.B), kCopyWarps * 32, 0, a.stream>>>(a, window_lens(a), esize, blocks);
    return cudaGetLastError();
}

}  // namespace la
