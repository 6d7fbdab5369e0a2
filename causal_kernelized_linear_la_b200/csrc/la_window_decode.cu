// Sliding-window attention with sinks, one token a sequence against the
// rolling cache, which takes the token's key and value in the same call.
//
// The cache's slots in use are always a prefix of the slot array (sinks, then
// ring), and softmax does not care about their order, so a step is attention
// of one query per head over min(pos + 1, sinks + window) slots.  Memory-bound
// on one read of the keys and values.
//
// One CTA takes a run of slots of one kv head and up to kHeads of its query
// heads; the CTAs of a cluster share a (sequence, kv head) and join their
// partial maxima, sums and outputs through distributed shared memory, so a
// step is one launch without a workspace, also for few sequences.  The slot
// that takes the new token is read from the call's k and v instead.
#include <cooperative_groups.h>

#include "la_window.cuh"

namespace la {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kHeads = 4;      // query heads a CTA serves at once
constexpr int kMaxSplit = 8;   // CTAs of a cluster
constexpr float kLog2e = 1.4426950408889634f;

template <typename T, int E>
__device__ __forceinline__ void load_row(const T* p, float (&f)[E])
{
    // E consecutive elements, 8 or 16 bytes
    if (sizeof(T) * E == 16) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] = to_f32<T>(t[i]);
    } else {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] = to_f32<T>(t[i]);
    }
}

// grid: (splits, Hkv * head chunks, sequences), clusters along x.  A warp
// handles one slot at a time; each lane holds D / 32 elements of q and k and
// DV / 32 columns of v and o.
template <typename T, int D, int DV>
__global__ void __launch_bounds__(kThreads)
window_decode_simt(const __grid_constant__ WindowArgs a, int chunks)
{
    constexpr int EK = D / 32, EV = DV / 32;
    __shared__ float part_o[kHeads][DV];
    __shared__ float part_ml[kHeads][2];
    __shared__ float warp_o[kWarps][kHeads][DV];
    __shared__ float warp_ml[kWarps][kHeads][2];
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int split = blockIdx.x, splits = gridDim.x, b = blockIdx.z;
    const int kvh = blockIdx.y / chunks, chunk = blockIdx.y % chunks;
    const int group = a.Hq / a.Hkv;
    const int h0 = kvh * group + chunk * kHeads, nh = min(kHeads, group - chunk * kHeads);
    const int pos = a.pos[b];
    if (pos < 0) return;        // an idle sequence: the whole cluster leaves
    const int cap = a.window + a.sinks;
    const int used = pos < cap ? pos + 1 : cap;
    const int slot_new = pos < a.sinks ? pos : a.sinks + (pos - a.sinks) % a.window;
    const int per = (used + splits - 1) / splits;
    const int s0 = min(used, split * per), s1 = min(used, s0 + per);

    const size_t kv = (size_t)b * a.Hkv + kvh;
    T* kc = (T*)a.k_cache + kv * cap * D;
    T* vc = (T*)a.v_cache + kv * cap * DV;
    const T* kn = (const T*)a.k + b * a.st.k_batch + kvh * a.st.k_head;
    const T* vn = (const T*)a.v + b * a.st.v_batch + kvh * a.st.v_head;
    const float sl = a.scale * kLog2e;

    float q[kHeads][EK], o[kHeads][EV], m[kHeads], l[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
#pragma unroll
        for (int i = 0; i < EV; ++i) o[h][i] = 0.f;
#pragma unroll
        for (int i = 0; i < EK; ++i) q[h][i] = 0.f;
        if (h < nh) {
            load_row<T, EK>((const T*)a.q + b * a.st.q_batch + (h0 + h) * a.st.q_head + lane * EK, q[h]);
#pragma unroll
            for (int i = 0; i < EK; ++i) q[h][i] *= sl;
        }
    }
    if (s0 <= slot_new && slot_new < s1 && chunk == 0) {
        for (int i = tid; i < D; i += kThreads) kc[(size_t)slot_new * D + i] = kn[i];
        for (int i = tid; i < DV; i += kThreads) vc[(size_t)slot_new * DV + i] = vn[i];
    }
    for (int s = s0 + warp; s < s1; s += kWarps) {
        const bool fresh = s == slot_new;
        float k[EK], v[EV];
        load_row<T, EK>((fresh ? kn : kc + (size_t)s * D) + lane * EK, k);
        load_row<T, EV>((fresh ? vn : vc + (size_t)s * DV) + lane * EV, v);
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < EK; ++i) x = fmaf(q[h][i], k[i], x);
#pragma unroll
            for (int w = 16; w > 0; w /= 2) x += __shfl_xor_sync(~0u, x, w);
            const float top = fmaxf(m[h], x), ref = top == -INFINITY ? 0.f : top;
            const float fade = exp2f(m[h] - ref), p = exp2f(x - ref);
            m[h] = top;
            l[h] = fmaf(l[h], fade, p);
#pragma unroll
            for (int i = 0; i < EV; ++i) o[h][i] = fmaf(p, v[i], o[h][i] * fade);
        }
    }
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
#pragma unroll
        for (int i = 0; i < EV; ++i) warp_o[warp][h][lane * EV + i] = o[h][i];
        if (lane == 0) {
            warp_ml[warp][h][0] = m[h];
            warp_ml[warp][h][1] = l[h];
        }
    }
    __syncthreads();
    for (int e = tid; e < kHeads * DV; e += kThreads) {
        const int h = e / DV, c = e % DV;
        float top = -INFINITY, sum = 0.f, acc = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, warp_ml[w][h][0]);
        const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2f(warp_ml[w][h][0] - ref);
            sum = fmaf(warp_ml[w][h][1], f, sum);
            acc = fmaf(warp_o[w][h][c], f, acc);
        }
        part_o[h][c] = acc;
        if (c == 0) {
            part_ml[h][0] = top;
            part_ml[h][1] = sum;
        }
    }
    cluster.sync();
    for (int e = split * kThreads + tid; e < nh * DV; e += splits * kThreads) {
        const int h = e / DV, c = e % DV;
        float top = -INFINITY, sum = 0.f, acc = 0.f;
        for (int r = 0; r < splits; ++r) top = fmaxf(top, cluster.map_shared_rank(&part_ml[h][0], r)[0]);
        for (int r = 0; r < splits; ++r) {
            const float f = exp2f(cluster.map_shared_rank(&part_ml[h][0], r)[0] - top);
            sum = fmaf(cluster.map_shared_rank(&part_ml[h][1], r)[0], f, sum);
            acc = fmaf(cluster.map_shared_rank(&part_o[h][c], r)[0], f, acc);
        }
        ((T*)a.out)[b * a.st.out_batch + (h0 + h) * a.st.out_head + c] = from_f32<T>(acc / sum);
    }
    cluster.sync();   // the others' shared memory stays until everyone has read it
}

template <typename T, int D, int DV>
cudaError_t launch_simt(const WindowArgs& a)
{
    const int group = a.Hq / a.Hkv, chunks = (group + kHeads - 1) / kHeads;
    const long long units = (long long)a.B * a.Hkv * chunks;
    int splits = 1;
    while (splits < kMaxSplit && units * splits < 296 && (a.window + a.sinks) / (splits * 2) >= 64) splits *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(splits, a.Hkv * chunks, a.B);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = a.stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = splits;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, window_decode_simt<T, D, DV>, a, chunks);
}

template <typename T>
cudaError_t launch_t(const WindowArgs& a)
{
    if (a.d == 64) return a.dv == 64 ? launch_simt<T, 64, 64>(a) : launch_simt<T, 64, 128>(a);
    return a.dv == 64 ? launch_simt<T, 128, 64>(a) : launch_simt<T, 128, 128>(a);
}

}  // namespace

cudaError_t launch_window_decode(const WindowArgs& a)
{
    return a.dtype == LA_BF16 ? launch_t<__nv_bfloat16>(a) : launch_t<float>(a);
}

}  // namespace la
