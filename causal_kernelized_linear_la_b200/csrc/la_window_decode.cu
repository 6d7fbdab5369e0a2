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
//
// 64 sequences of 32 heads over 8, 4100 slots of 128 + 128
// columns, bf16: 163 to 179 us on different cards, 98 to 90 % of the measured copy rate.
// One sequence: 10.7 us, where the floor is 2.6: launch, one wave of loads and the
// cluster's join.  fp32: 494 us (65 %) and 53 us; a warp takes one slot a turn with
// no load ahead and five shuffles a head, and waits for its loads.
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

// ---------------------------------------------------------------------------
// bf16 on the tensor cores' warp instructions (mma m16n8k16): eight query
// heads of a kv head are the N of both products, so grouped heads cost no more
// than one,
//     S^T = K Q^T   (16 keys x 8 heads, K-axis d)
//     O^T += V^T P^T   (dv x 8 heads, K-axis 16 keys)
// and one register operand per product comes straight from global memory:
// the order of an MMA's K-axis and of its M rows is free as long as both
// operands, or the output, follow it.
//   K: lane (g, t) takes 16 bytes at d = 32 s + 8 t of the keys g and g + 8; its
//      four 32-bit words are the K-slots (2t, 2t+1), (2t+8, 2t+9) of the steps
//      2 s and 2 s + 1, and q is loaded with the same map.
//   V: lane (g, t) takes 16 bytes at column 64 c + 8 g of the keys 2t, 2t+1, 2t+8,
//      2t+9; byte permutes pair the keys, and row g (g + 8) of output tile
//      4 c + j is column 64 c + 8 g + 2 j (+ 1).
// No shared memory is staged: each warp keeps one block of 16 keys of K and V
// in flight, twelve warps an SM some 90 KB.  The weights meet V as two bf16 parts,
// two products that keep 2^-15 of each weight: beside the loads the second costs 1
// to 2 % (64 sequences of 4100 slots 168 -> 170 us on one card, 176 -> 179 on another),
// while weights rounded to one bf16 took the error from 0.0017 of the output to 0.0021.
constexpr int kMmaHeads = 8;
constexpr int kAhead = 2;      // blocks of a warp between an L2 prefetch and its use

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8 x 8 fragment of 16-bit values -> the fragment of its transpose
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint4 load_stream(const __nv_bfloat16* p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Two weights' upper bf16 halves (cut off, not rounded), and what that leaves of them.  The rest is
// at least 1e-30, far below anything that counts: a rest of zero would make an infinite value NaN.
__device__ __forceinline__ uint32_t upper_pair(float a, float b)
{
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ uint32_t lower_pair(float a, float b)
{
    auto rest = [](float x) { return fmaxf(x - __uint_as_float(__float_as_uint(x) & 0xffff0000u), 1e-30f); };
    return bf16_pair(rest(a), rest(b));
}

// grid: (splits, Hkv * head chunks, sequences), clusters along x
template <int D, int DV, int kMmaWarps>
__global__ void __launch_bounds__(kMmaWarps * 32, 12 / kMmaWarps)
window_decode_mma(const __grid_constant__ WindowArgs a, int chunks)
{
    constexpr int KS = D / 32, VC = DV / 64, OT = DV / 16;   // 16-byte pieces of a K row, of a V row per lane; output tiles
    constexpr int OP = DV + 4;                               // row pitch of the partial outputs
    __shared__ float part_o[kMmaWarps][kMmaHeads][OP];
    __shared__ float part_ml[kMmaWarps + 1][kMmaHeads][2];   // the last: of the whole CTA
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int split = blockIdx.x, splits = gridDim.x, b = blockIdx.z;
    const int kvh = blockIdx.y / chunks, chunk = blockIdx.y % chunks;
    const int group = a.Hq / a.Hkv;
    const int h0 = kvh * group + chunk * kMmaHeads, nh = min(kMmaHeads, group - chunk * kMmaHeads);
    const int pos = a.pos[b];
    if (pos < 0) return;        // an idle sequence: the whole cluster leaves
    const int cap = a.window + a.sinks;
    const int used = pos < cap ? pos + 1 : cap;
    const int slot_new = pos < a.sinks ? pos : a.sinks + (pos - a.sinks) % a.window;
    const int per = ((used + splits - 1) / splits + 15) / 16 * 16;
    const int s0 = min(used, split * per), s1 = min(used, s0 + per);

    const size_t kv = (size_t)b * a.Hkv + kvh;
    __nv_bfloat16* kc = (__nv_bfloat16*)a.k_cache + kv * cap * D;
    __nv_bfloat16* vc = (__nv_bfloat16*)a.v_cache + kv * cap * DV;
    const __nv_bfloat16* kn = (const __nv_bfloat16*)a.k + b * a.st.k_batch + kvh * a.st.k_head;
    const __nv_bfloat16* vn = (const __nv_bfloat16*)a.v + b * a.st.v_batch + kvh * a.st.v_head;
    const float sl = a.scale * kLog2e;

    uint4 kr[2][KS], vr[4][VC];
    // slots past the run repeat its last one; their scores are -inf, and their values zero by the time they
    // meet the weights: the last slot's may be infinite
    auto k_row = [&](int s) { const int x = min(s, s1 - 1); return (x == slot_new ? kn : kc + (size_t)x * D) + 8 * t; };
    auto v_row = [&](int s) { const int x = min(s, s1 - 1); return (x == slot_new ? vn : vc + (size_t)x * DV) + 8 * g; };
    auto load_k = [&](int s) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const __nv_bfloat16* p = k_row(s + g + 8 * i);
#pragma unroll
            for (int x = 0; x < KS; ++x) kr[i][x] = load_stream(p + 32 * x);
        }
    };
    auto load_v = [&](int s) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat16* p = v_row(s + 2 * t + (i & 1) + 8 * (i >> 1));
#pragma unroll
            for (int x = 0; x < VC; ++x) vr[i][x] = load_stream(p + 64 * x);
        }
    };

    // a block of this warp's keys some turns ahead into L2: one 128-byte line a lane and row half
    auto ahead = [&](int s) {
        const int row = min(s + (lane >> 1), s1 - 1), half = (lane & 1) * 64;
        if (s < s1 && half < D) asm volatile("prefetch.global.L2 [%0];" ::"l"(kc + (size_t)row * D + half));
        if (s < s1 && half < DV) asm volatile("prefetch.global.L2 [%0];" ::"l"(vc + (size_t)row * DV + half));
    };

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};   // of heads 2t, 2t+1 (l: this lane's keys)
    float o[OT][4];
#pragma unroll
    for (int j = 0; j < OT; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[j][x] = 0.f;
    int s = s0 + warp * 16;
    if (s < s1) {
        load_k(s);
        load_v(s);
#pragma unroll
        for (int i = 1; i < kAhead; ++i) ahead(s + i * kMmaWarps * 16);
    }
    uint4 qr[KS];
#pragma unroll
    for (int x = 0; x < KS; ++x) {
        qr[x] = make_uint4(0u, 0u, 0u, 0u);
        if (g < nh)
            qr[x] = *reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.q + b * a.st.q_batch + (h0 + g) * a.st.q_head + 32 * x + 8 * t);
    }
    for (; s < s1; s += kMmaWarps * 16) {
        const int next = s + kMmaWarps * 16;
        ahead(s + kAhead * kMmaWarps * 16);
        // two sums of every other step: half the chain of dependent products
        float c[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < KS; ++x) {
            mma_16816(c, kr[0][x].x, kr[1][x].x, kr[0][x].y, kr[1][x].y, qr[x].x, qr[x].y);
            mma_16816(c1, kr[0][x].z, kr[1][x].z, kr[0][x].w, kr[1][x].w, qr[x].z, qr[x].w);
        }
        if (next < s1) load_k(next);
        // c: keys g (0, 1) and g + 8 (2, 3) of heads 2t, 2t + 1
        const bool on0 = s + g < s1, on1 = s + g + 8 < s1;
        float top[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            c[j] = on0 ? (c[j] + c1[j]) * sl : -INFINITY;
            c[2 + j] = on1 ? (c[2 + j] + c1[2 + j]) * sl : -INFINITY;
            top[j] = fmaxf(c[j], c[2 + j]);
#pragma unroll
            for (int w = 4; w < 32; w *= 2) top[j] = fmaxf(top[j], __shfl_xor_sync(~0u, top[j], w));
        }
        if (__any_sync(~0u, top[0] > m[0] || top[1] > m[1])) {
            float f[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float nm = fmaxf(m[j], top[j]);
                f[j] = m[j] == -INFINITY ? 0.f : exp2f(m[j] - nm);
                m[j] = nm;
                l[j] *= f[j];
            }
#pragma unroll
            for (int j = 0; j < OT; ++j) {
                o[j][0] *= f[0];
                o[j][1] *= f[1];
                o[j][2] *= f[0];
                o[j][3] *= f[1];
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float ref = m[j] == -INFINITY ? 0.f : m[j];
            c[j] = exp2f(c[j] - ref);
            c[2 + j] = exp2f(c[2 + j] - ref);
            l[j] += c[j] + c[2 + j];
        }
        if (s + 16 > s1) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (s + 2 * t + (i & 1) + 8 * (i >> 1) >= s1)
#pragma unroll
                    for (int x = 0; x < VC; ++x) vr[i][x] = make_uint4(0u, 0u, 0u, 0u);
        }
        const uint32_t p0 = transpose8(upper_pair(c[0], c[1])), p1 = transpose8(upper_pair(c[2], c[3]));
        const uint32_t r0 = transpose8(lower_pair(c[0], c[1])), r1 = transpose8(lower_pair(c[2], c[3]));
#pragma unroll
        for (int x = 0; x < VC; ++x) {
            const uint32_t* v0 = reinterpret_cast<const uint32_t*>(&vr[0][x]);
            const uint32_t* v1 = reinterpret_cast<const uint32_t*>(&vr[1][x]);
            const uint32_t* v2 = reinterpret_cast<const uint32_t*>(&vr[2][x]);
            const uint32_t* v3 = reinterpret_cast<const uint32_t*>(&vr[3][x]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t a0 = __byte_perm(v0[j], v1[j], 0x5410), a1 = __byte_perm(v0[j], v1[j], 0x7632),
                               a2 = __byte_perm(v2[j], v3[j], 0x5410), a3 = __byte_perm(v2[j], v3[j], 0x7632);
                mma_16816(o[4 * x + j], a0, a1, a2, a3, p0, p1);
                mma_16816(o[4 * x + j], a0, a1, a2, a3, r0, r1);
            }
        }
        if (next < s1) load_v(next);
    }
    // the new token takes its slot; every reader of the slot reads kn, vn
    if (s0 <= slot_new && slot_new < s1 && chunk == 0) {
        if (tid < D / 8) reinterpret_cast<uint4*>(kc + (size_t)slot_new * D)[tid] = reinterpret_cast<const uint4*>(kn)[tid];
        if (tid < DV / 8) reinterpret_cast<uint4*>(vc + (size_t)slot_new * DV)[tid] = reinterpret_cast<const uint4*>(vn)[tid];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int w = 4; w < 32; w *= 2) l[j] += __shfl_xor_sync(~0u, l[j], w);
        if (g == 0) {
            part_ml[warp][2 * t + j][0] = m[j];
            part_ml[warp][2 * t + j][1] = l[j];
        }
    }
#pragma unroll
    for (int j = 0; j < OT; ++j) {
        const int col = 64 * (j / 4) + 8 * g + 2 * (j % 4);
        *reinterpret_cast<float2*>(&part_o[warp][2 * t][col]) = make_float2(o[j][0], o[j][2]);
        *reinterpret_cast<float2*>(&part_o[warp][2 * t + 1][col]) = make_float2(o[j][1], o[j][3]);
    }
    __syncthreads();
    // the warps' parts into warp 0's place
    for (int e = tid; e < nh * DV; e += kMmaWarps * 32) {
        const int h = e / DV, c = e % DV;
        float top = -INFINITY, sum = 0.f, acc = 0.f;
#pragma unroll
        for (int w = 0; w < kMmaWarps; ++w) top = fmaxf(top, part_ml[w][h][0]);
        const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int w = 0; w < kMmaWarps; ++w) {
            const float f = exp2f(part_ml[w][h][0] - ref);
            sum = fmaf(part_ml[w][h][1], f, sum);
            acc = fmaf(part_o[w][h][c], f, acc);
        }
        if (splits == 1) {
            ((__nv_bfloat16*)a.out)[b * a.st.out_batch + (h0 + h) * a.st.out_head + c] = __float2bfloat16_rn(acc / sum);
        } else {
            part_o[0][h][c] = acc;       // this thread alone reads and writes column c of head h
            if (c == 0) {
                part_ml[kMmaWarps][h][0] = top;
                part_ml[kMmaWarps][h][1] = sum;
            }
        }
    }
    if (splits == 1) return;
    cluster.sync();
    for (int e = split * kMmaWarps * 32 + tid; e < nh * DV; e += splits * kMmaWarps * 32) {
        const int h = e / DV, c = e % DV;
        float top = -INFINITY, sum = 0.f, acc = 0.f;
        for (int r = 0; r < splits; ++r) top = fmaxf(top, cluster.map_shared_rank(&part_ml[kMmaWarps][h][0], r)[0]);
        for (int r = 0; r < splits; ++r) {
            const float f = exp2f(cluster.map_shared_rank(&part_ml[kMmaWarps][h][0], r)[0] - top);
            sum = fmaf(cluster.map_shared_rank(&part_ml[kMmaWarps][h][1], r)[0], f, sum);
            acc = fmaf(cluster.map_shared_rank(&part_o[0][h][c], r)[0], f, acc);
        }
        ((__nv_bfloat16*)a.out)[b * a.st.out_batch + (h0 + h) * a.st.out_head + c] = __float2bfloat16_rn(acc / sum);
    }
    cluster.sync();   // the others' shared memory stays until everyone has read it
}

// One launch: clusters of `splits` CTAs share a (sequence, kv head, head chunk).
template <typename F>
cudaError_t launch_clusters(F kern, const WindowArgs& a, int heads, int threads, int splits)
{
    const int chunks = (a.Hq / a.Hkv + heads - 1) / heads;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(splits, a.Hkv * chunks, a.B);
    cfg.blockDim = dim3(threads);
    cfg.stream = a.stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = splits;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, chunks);
}

// CTAs a (sequence, kv head, head chunk): enough for `want` in all, each with at least `least` slots.
int splits_for(const WindowArgs& a, int heads, int want, int least, int most)
{
    const int chunks = (a.Hq / a.Hkv + heads - 1) / heads;
    const long long units = (long long)a.B * a.Hkv * chunks;
    int splits = 1;
    while (splits < most && units * splits < want && (a.window + a.sinks) / (splits * 2) >= least) splits *= 2;
    return splits;
}

template <int D, int DV>
cudaError_t launch_dd(const WindowArgs& a)
{
    if (a.dtype == LA_BF16) {
        // Few CTAs (one wave of one an SM, or two waves in small clusters, which pack): eight warps
        // each halve a warp's serial walk (128 units of 4100 slots 58 -> 52 us).  Else four warps, three
        // CTAs an SM: at least 64 slots a CTA up to four an SM, and eight an SM, which even out the last
        // wave, while a CTA keeps 512 slots (512 units of 4100 slots 184 -> 173 us; with 257 slots a CTA
        // its 4 us of set-up and joining cost more than that: 256 units of 1028 slots 33 -> 52 us).
        const int wide = splits_for(a, kMmaHeads, 148, 128, kMaxSplit);
        const int chunks = (a.Hq / a.Hkv + kMmaHeads - 1) / kMmaHeads;
        const long long ctas = (long long)a.B * a.Hkv * chunks * wide;
        if (ctas <= 148 || (wide <= 2 && ctas <= 296))
            return launch_clusters(window_decode_mma<D, DV, 8>, a, kMmaHeads, 256, wide);
        const int fill = splits_for(a, kMmaHeads, 148 * 4, 64, 8), even = splits_for(a, kMmaHeads, 148 * 8, 512, 8);
        return launch_clusters(window_decode_mma<D, DV, 4>, a, kMmaHeads, 128, fill > even ? fill : even);
    }
    return launch_clusters(window_decode_simt<float, D, DV>, a, kHeads, kThreads, splits_for(a, kHeads, 148 * 4, 64, 8));
}

}  // namespace

cudaError_t launch_window_decode(const WindowArgs& a)
{
    if (a.d == 64) return a.dv == 64 ? launch_dd<64, 64>(a) : launch_dd<64, 128>(a);
    return a.dv == 64 ? launch_dd<128, 64>(a) : launch_dd<128, 128>(a);
}

}  // namespace la
