// Selective state-space recurrence.  Per sequence, channel c and state s:
//     dt_t   = delta_t[c] + bias[c], through softplus if asked
//     h_t[s] = exp(dt_t A[c,s]) h_{t-1}[s] + dt_t x_t[c] B_t[s]
//     y_t[c] = (sum_s C_t[s] h_t[s] + D[c] x_t[c]) * silu(z_t[c])
// B and C are shared by the channels of a group.  States, step sizes, decays
// and sums are fp32; y is rounded to the storage type once.
//
// Prompt scan.  A CTA walks the tokens of 32 channels in tiles of kTile.  Four
// lanes share a channel, each with NS states in registers; the raw rows of
// the tile after this one arrive by cp.async while this one is computed.  Per
// tile the CTA first turns delta and x into (dt, dt x) and B, C into fp32, then
// runs the recurrence, then finishes y: the softplus, the gate and the type
// conversions are done once a value, not once a lane.
// The decay needs one exponential per (token, channel, state): the SFU's 16 a
// clock and SM bound the scan (at n = 16 its 2^x alone take three times as
// long as reading delta, x, z and writing y), not memory.
//
// Few channels leave SMs idle, so a long sequence is cut into segments: a
// first kernel runs every segment but the last from a zero state and keeps
// its end state and sum of dt; since the decay over a segment is
// exp(A sum dt), each segment of the second kernel folds the segments before
// it into its own start state and runs once more with outputs.
#include "la_internal.cuh"
#include "sm100.cuh"

namespace la {
namespace {

using namespace sm100;

constexpr int kCh = 32;        // channels of a CTA
constexpr int kLanes = 4;      // lanes sharing a channel
constexpr int kThreads = kCh * kLanes;
constexpr int kTile = 32;      // tokens of a tile
constexpr int kYPitch = 40;    // fp32 row pitch of the y tile: four tokens x eight channels hit 32 banks
constexpr float kLog2e = 1.4426950408889634f;

struct Lens {
    int use;
    int n[kMaxSeqLens];
};

// Two fp32 values in one register pair, for the packed arithmetic of sm_100.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack2(float a, float b)
{
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(f2 v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b)
{
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c)
{
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ float softplus(float v) { return v > 20.f ? v : log1pf(expf(v)); }
template <typename T> __device__ __forceinline__ float silu(float v);
template <> __device__ __forceinline__ float silu<float>(float v) { return v / (1.f + expf(-v)); }
template <> __device__ __forceinline__ float silu<__nv_bfloat16>(float v) { return __fdividef(v, 1.f + __expf(-v)); }

template <int BYTES>
__device__ __forceinline__ void cp_async_n(void* dst, const void* src, uint32_t src_bytes)
{
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(src_bytes)
                     : "memory");
    else
        cp_async4(dst, src, src_bytes);
}

// A tile of `rows` (of kTile) x `cols` (of PITCH) elements of a row-major
// tensor into shared memory, zeros elsewhere, in pieces of `piece` bytes (16,
// 4, or the element itself where rows do not start on 4 bytes).
template <typename T>
__device__ __forceinline__ void load_tile(T* dst, const T* src, long long row_stride, int rows, int cols, int pitch,
                                          int piece)
{
    const int per = piece / (int)sizeof(T);   // elements of a piece
    const int n = pitch / per;
    for (int e = threadIdx.x; e < kTile * n; e += kThreads) {
        const int t = e / n, c = (e % n) * per;
        const int left = t < rows ? min(per, max(0, cols - c)) : 0;
        const T* s = left > 0 ? src + t * row_stride + c : src;
        T* d = dst + t * pitch + c;
        if (piece == 16) cp_async_n<16>(d, s, left * sizeof(T));
        else if (piece == 4) cp_async_n<4>(d, s, left * sizeof(T));
        else *d = left > 0 ? *s : from_f32<T>(0.f);
    }
}

template <typename T, int NS>
struct Plan {
    static constexpr int NP = kLanes * NS;     // states, padded
    static constexpr int BCP = NP < 8 ? 8 : NP;   // elements of a B or C row in shared memory: whole 16-byte pieces
    static constexpr int ROW = kTile * kCh * (int)sizeof(T), BC = kTile * BCP * (int)sizeof(T);
    // a stage: x, delta, z tiles, B, C tiles
    static constexpr int STAGE = 3 * ROW + 2 * BC;
    static constexpr int OFF_DU = 2 * STAGE;                    // (dt, dt, dt x, dt x) fp32 [kTile][kCh]
    static constexpr int OFF_B = OFF_DU + kTile * kCh * 16;     // fp32 [kTile][NP]
    static constexpr int OFF_C = OFF_B + kTile * NP * 4;
    static constexpr int OFF_Y = OFF_C + kTile * NP * 4;        // fp32 [kTile][kYPitch]
    static constexpr int BYTES = OFF_Y + kTile * kYPitch * 4;
};

// A segment's summary: end state [kCh][NP] from zero, then sum of dt [kCh].
template <int NS> __host__ __device__ constexpr int slot_floats() { return kCh * (kLanes * NS + 1); }

// grid: (channel tiles, segments, sequences).  SUMMARY: the first kernel of a
// segmented scan; otherwise outputs and the final state.
template <typename T, int NS, bool SUMMARY>
__global__ void __launch_bounds__(kThreads)
ssm_scan_kernel(const __grid_constant__ SsmArgs a, const __grid_constant__ Lens lens, int tiles_per_group, int px,
                int pb)
{
    using P = Plan<T, NS>;
    constexpr int NP = P::NP;
    extern __shared__ __align__(16) unsigned char sm[];
    const int tid = threadIdx.x;
    const int ch = tid / kLanes, l = tid % kLanes;     // a warp holds 8 channels x 4 lanes
    const int b = blockIdx.z, seg = blockIdx.y, tile = blockIdx.x;
    const int grp = tile / tiles_per_group, per = a.D / a.G;
    const int cg0 = (tile % tiles_per_group) * kCh;    // first channel inside the group
    const int c0 = grp * per + cg0, nch = min(kCh, per - cg0);
    const int len = lens.use ? lens.n[b] : a.N;
    const int s0 = seg * a.seg_len, s1 = min(len, s0 + a.seg_len);
    const bool mine = ch < nch;
    const int c = c0 + (mine ? ch : 0);

    if (SUMMARY) grid_launch_dependents();
    if (s0 >= len && !(seg == 0 && !SUMMARY)) return;   // an empty sequence still reports its start state

    // this lane's states and decay rates (in log2 units); padded states stay zero
    f2 A2[(NS + 1) / 2], h[(NS + 1) / 2];
#pragma unroll
    for (int i = 0; i < NS; i += 2) {
        const int s = l * NS + i;
        const float* ap = a.A + (size_t)c * a.n;
        A2[i / 2] = pack2(mine && s < a.n ? ap[s] * kLog2e : 0.f, NS > 1 && mine && s + 1 < a.n ? ap[s + 1] * kLog2e : 0.f);
        const float* hp = a.h0 + ((size_t)b * a.D + c) * a.n;
        const bool from = a.h0 && mine && seg == 0;
        h[i / 2] = pack2(from && s < a.n ? hp[s] : 0.f, NS > 1 && from && s + 1 < a.n ? hp[s + 1] : 0.f);
    }
    const size_t unit0 = ((size_t)b * gridDim.x + tile) * a.segs;   // this chain's first summary slot
    if (!SUMMARY && a.segs > 1) {
        grid_dependency_wait();   // the summaries
        for (int g = 0; g < seg; ++g) {
            const float* slot = a.workspace + (unit0 + g) * slot_floats<NS>();
            const float dt = slot[kCh * NP + ch];
#pragma unroll
            for (int i = 0; i < NS; i += 2) {
                const float2 ar = unpack2(A2[i / 2]);
                const float* e = slot + ch * NP + l * NS + i;
                h[i / 2] = fma2(pack2(ex2_approx(dt * ar.x), ex2_approx(dt * ar.y)), h[i / 2],
                                pack2(e[0], NS > 1 ? e[1] : 0.f));
            }
        }
    }

    const T* xp = (const T*)a.x + b * a.st.x_batch + c0;
    const T* dp = (const T*)a.delta + b * a.st.delta_batch + c0;
    const T* zp = a.z ? (const T*)a.z + b * a.st.z_batch + c0 : nullptr;
    const T* bp = (const T*)a.Bm + b * a.st.B_batch + (size_t)grp * a.n;
    const T* cp = (const T*)a.Cm + b * a.st.C_batch + (size_t)grp * a.n;
    auto fetch = [&](int t, int stage) {
        unsigned char* st = sm + stage * P::STAGE;
        const int rows = s1 - t;
        load_tile<T>((T*)st, xp + t * a.st.x_row, a.st.x_row, rows, nch, kCh, px);
        load_tile<T>((T*)(st + P::ROW), dp + t * a.st.delta_row, a.st.delta_row, rows, nch, kCh, px);
        if (!SUMMARY && zp) load_tile<T>((T*)(st + 2 * P::ROW), zp + t * a.st.z_row, a.st.z_row, rows, nch, kCh, px);
        load_tile<T>((T*)(st + 3 * P::ROW), bp + t * a.st.B_row, a.st.B_row, rows, a.n, P::BCP, pb);
        if (!SUMMARY) load_tile<T>((T*)(st + 3 * P::ROW + P::BC), cp + t * a.st.C_row, a.st.C_row, rows, a.n, P::BCP, pb);
    };

    float4* du = reinterpret_cast<float4*>(sm + P::OFF_DU);
    float* Bf = reinterpret_cast<float*>(sm + P::OFF_B);
    float* Cf = reinterpret_cast<float*>(sm + P::OFF_C);
    float* yf = reinterpret_cast<float*>(sm + P::OFF_Y);
    const int cc = tid % kCh, tr = tid / kCh;            // element-wise passes: channel and first token
    const float bias = a.delta_bias && cc < nch ? a.delta_bias[c0 + cc] : 0.f;
    const float skip = !SUMMARY && a.skip && cc < nch ? a.skip[c0 + cc] : 0.f;
    float dt_sum = 0.f;                                   // of channel cc, over this thread's tokens

    if (s0 < s1) fetch(s0, 0);
    cp_async_commit();
    int stage = 0;
    for (int t0 = s0; t0 < s1; t0 += kTile, stage ^= 1) {
        const int rows = min(kTile, s1 - t0);
        cp_async_wait_all();
        __syncthreads();   // this tile's rows are in, and the previous tile is done with
        if (t0 + kTile < s1) fetch(t0 + kTile, stage ^ 1);
        cp_async_commit();
        const unsigned char* st = sm + stage * P::STAGE;
        const T* xs = (const T*)st;
        const T* ds = (const T*)(st + P::ROW);
        const T* zs = (const T*)(st + 2 * P::ROW);
        const T* bs = (const T*)(st + 3 * P::ROW);
        const T* cs = (const T*)(st + 3 * P::ROW + P::BC);
        for (int t = tr; t < kTile; t += kThreads / kCh) {
            float dt = to_f32<T>(ds[t * kCh + cc]) + bias;
            if (a.softplus) dt = softplus(dt);
            if (t >= rows) dt = 0.f;                      // decay 1, nothing added
            const float u = dt * to_f32<T>(xs[t * kCh + cc]);
            du[t * kCh + cc] = make_float4(dt, dt, u, u);
            if (SUMMARY) dt_sum += dt;
        }
        for (int e = tid; e < kTile * NP; e += kThreads) {
            const int at = (e / NP) * P::BCP + e % NP;
            Bf[e] = to_f32<T>(bs[at]);
            if (!SUMMARY) Cf[e] = to_f32<T>(cs[at]);
        }
        __syncthreads();
#pragma unroll 1
        for (int t = 0; t < kTile; t += 4) {
            float part[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const ulonglong2 d2 = reinterpret_cast<const ulonglong2*>(du)[(t + j) * kCh + ch];
                f2 acc = 0;
                if (NS == 1) {
                    const float a1 = ex2_approx(unpack2(d2.x).x * unpack2(A2[0]).x);
                    const float h1 = fmaf(a1, unpack2(h[0]).x, unpack2(d2.y).x * Bf[(t + j) * NP + l]);
                    h[0] = pack2(h1, 0.f);
                    if (!SUMMARY) acc = pack2(h1 * Cf[(t + j) * NP + l], 0.f);
                } else {
                    const f2* B2 = reinterpret_cast<const f2*>(Bf + (t + j) * NP + l * NS);
                    const f2* C2 = reinterpret_cast<const f2*>(Cf + (t + j) * NP + l * NS);
#pragma unroll
                    for (int i = 0; i < NS / 2; ++i) {
                        const float2 e = unpack2(mul2(d2.x, A2[i]));
                        h[i] = fma2(pack2(ex2_approx(e.x), ex2_approx(e.y)), h[i], mul2(d2.y, B2[i]));
                        if (!SUMMARY) acc = fma2(C2[i], h[i], acc);
                    }
                }
                const float2 s = unpack2(acc);
                part[j] = s.x + s.y;
            }
            if (!SUMMARY) {
                // sum over the channel's four lanes; lane l ends with token t + l
                const bool o2 = l & 2, o1 = l & 1;
                const float k0 = (o2 ? part[2] : part[0]) + __shfl_xor_sync(~0u, o2 ? part[0] : part[2], 2);
                const float k1 = (o2 ? part[3] : part[1]) + __shfl_xor_sync(~0u, o2 ? part[1] : part[3], 2);
                yf[(t + l) * kYPitch + ch] = (o1 ? k1 : k0) + __shfl_xor_sync(~0u, o1 ? k0 : k1, 1);
            }
        }
        if (!SUMMARY) {
            __syncthreads();
            T* yp = (T*)a.out + (size_t)b * a.N * a.D + c0 + cc;
            if (cc < nch) {
                for (int t = tr; t < rows; t += kThreads / kCh) {
                    float y = fmaf(skip, to_f32<T>(xs[t * kCh + cc]), yf[t * kYPitch + cc]);
                    if (zp) y *= silu<T>(to_f32<T>(zs[t * kCh + cc]));
                    yp[(size_t)(t0 + t) * a.D] = from_f32<T>(y);
                }
            }
        }
    }

    if (SUMMARY) {
        // sum of dt over the four threads of each channel
        __syncthreads();
        yf[tr * kYPitch + cc] = dt_sum;
        __syncthreads();
        float* slot = a.workspace + (unit0 + seg) * slot_floats<NS>();
        if (tid < kCh)
            slot[kCh * NP + tid] = yf[tid] + yf[kYPitch + tid] + yf[2 * kYPitch + tid] + yf[3 * kYPitch + tid];
#pragma unroll
        for (int i = 0; i < NS; i += 2) {
            const float2 v = unpack2(h[i / 2]);
            slot[ch * NP + l * NS + i] = v.x;
            if (NS > 1) slot[ch * NP + l * NS + i + 1] = v.y;
        }
    } else if (s1 == len && mine && a.h_out) {
        float* hp = a.h_out + ((size_t)b * a.D + c) * a.n;
#pragma unroll
        for (int i = 0; i < NS; i += 2) {
            const int s = l * NS + i;
            const float2 v = unpack2(h[i / 2]);
            if (s < a.n) hp[s] = v.x;
            if (NS > 1 && s + 1 < a.n) hp[s + 1] = v.y;
        }
    }
}

// Largest piece (16, 4 or the element's own bytes) that divides an address and its row strides.
int piece_of(const void* p, long long batch, long long row, int e)
{
    const unsigned long long m = reinterpret_cast<uintptr_t>(p) | (unsigned long long)(batch * e) | (unsigned long long)(row * e);
    return m % 16 == 0 ? 16 : m % 4 == 0 ? 4 : e;
}

template <typename T, int NS>
cudaError_t launch_scan_ns(const SsmArgs& a)
{
    using P = Plan<T, NS>;
    const int e = sizeof(T);
    const int per = a.D / a.G, tpg = (per + kCh - 1) / kCh;
    Lens lens{};
    lens.use = a.seq_lens != nullptr;
    if (a.seq_lens)
        for (int b = 0; b < a.B; ++b) lens.n[b] = a.seq_lens[b];
    // a group's channels start per * group elements into a row
    const long long goff = a.G > 1 ? per : 0, noff = a.G > 1 ? a.n : 0;
    int px = piece_of(a.x, a.st.x_batch, a.st.x_row, e);
    px = min(px, piece_of(a.delta, a.st.delta_batch, a.st.delta_row, e));
    if (a.z) px = min(px, piece_of(a.z, a.st.z_batch, a.st.z_row, e));
    px = min(px, piece_of(nullptr, goff, 0, e));
    int pb = piece_of(a.Bm, a.st.B_batch, a.st.B_row, e);
    pb = min(pb, piece_of(a.Cm, a.st.C_batch, a.st.C_row, e));
    pb = min(pb, piece_of(nullptr, noff, 0, e));
    auto main_k = ssm_scan_kernel<T, NS, false>;
    auto sum_k = ssm_scan_kernel<T, NS, true>;
    cudaError_t err = cudaFuncSetAttribute(main_k, cudaFuncAttributeMaxDynamicSharedMemorySize, P::BYTES);
    if (err == cudaSuccess) err = cudaFuncSetAttribute(sum_k, cudaFuncAttributeMaxDynamicSharedMemorySize, P::BYTES);
    if (err != cudaSuccess) return err;
    int stage = 0;
    if (a.segs > 1) {
        sum_k<<<dim3(tpg * a.G, a.segs - 1, a.B), kThreads, P::BYTES, a.stream>>>(a, lens, tpg, px, pb);
        if ((err = cudaGetLastError()) != cudaSuccess) return err;
        stage_mark(stage++, a.stream);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(tpg * a.G, a.segs, a.B);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = P::BYTES;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = a.segs > 1 ? 1 : 0;
    err = cudaLaunchKernelEx(&cfg, main_k, a, lens, tpg, px, pb);
    if (err == cudaSuccess) stage_mark(stage, a.stream);
    return err;
}

template <typename T>
cudaError_t launch_scan_t(const SsmArgs& a)
{
    if (a.n <= 4) return launch_scan_ns<T, 1>(a);
    if (a.n <= 8) return launch_scan_ns<T, 2>(a);
    if (a.n <= 16) return launch_scan_ns<T, 4>(a);
    if (a.n <= 32) return launch_scan_ns<T, 8>(a);
    return launch_scan_ns<T, 16>(a);
}

}  // namespace

void ssm_scan_segments(int B, int N, int D, int G, int n, int* segs, int* seg_len)
{
    (void)n;
    const int per = D / G;
    const long long units = (long long)B * G * ((per + kCh - 1) / kCh);
    // enough CTAs for every SM sub-partition to hold a warp or two; segments stay long enough to pay for their summary
    int g = 1;
    if (units < 96) {
        const int want = (int)((256 + units - 1) / units);
        const int most = N / 256;
        g = max(1, min(min(want, most), 64));
    }
    const int L = ((N + g - 1) / g + kTile - 1) / kTile * kTile;
    *seg_len = L > 0 ? L : kTile;
    *segs = N > 0 ? (N + *seg_len - 1) / *seg_len : 1;
}

size_t ssm_scan_workspace_bytes(int B, int N, int D, int G, int n)
{
    int segs, len;
    ssm_scan_segments(B, N, D, G, n, &segs, &len);
    if (segs <= 1) return 0;
    const int np = n <= 4 ? 4 : n <= 8 ? 8 : n <= 16 ? 16 : n <= 32 ? 32 : 64;
    const int per = D / G;
    return (size_t)B * G * ((per + kCh - 1) / kCh) * segs * kCh * (np + 1) * sizeof(float);
}

cudaError_t launch_ssm_scan(const SsmArgs& a)
{
    return a.dtype == LA_BF16 ? launch_scan_t<__nv_bfloat16>(a) : launch_scan_t<float>(a);
}

// ---------------------------------------------------------------------------
// Token step: one token of each sequence, the state [B, D, n] updated in
// place.  Memory-bound on the state's read and write.  A warp takes 32
// consecutive channels of one sequence: lane i prepares channel i's scalars
// (dt, dt x, D x, the gate), then the states pass as a flat run of 32 n values,
// V at a time per lane (16-byte accesses where n is a multiple of four), with
// the scalars fetched by shuffles.  P lanes share a channel and add their
// parts of y by shuffles.
namespace {

constexpr int kStepWarps = 4;

// V consecutive states a lane, P = lanes a channel (a power of two >= ceil(n / V))
template <typename T, int V, int P>
__global__ void __launch_bounds__(kStepWarps * 32)
ssm_step_kernel(const __grid_constant__ SsmArgs a, int tiles_per_group)
{
    const int lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * kStepWarps + (threadIdx.x >> 5);
    const int tiles = tiles_per_group * a.G;
    if (unit >= (long long)a.B * tiles) return;
    const int b = (int)(unit / tiles), tile = (int)(unit % tiles);
    const int grp = tile / tiles_per_group, per = a.D / a.G;
    const int cg0 = (tile % tiles_per_group) * 32;
    const int c0 = grp * per + cg0, nch = min(32, per - cg0);
    const int n = a.n;

    float dt = 0.f, u = 0.f, add = 0.f, gate = 1.f;
    if (lane < nch) {
        const int c = c0 + lane;
        const float xv = to_f32<T>(((const T*)a.x)[b * a.st.x_batch + c]);
        dt = to_f32<T>(((const T*)a.delta)[b * a.st.delta_batch + c]) + (a.delta_bias ? a.delta_bias[c] : 0.f);
        if (a.softplus) dt = softplus(dt);
        u = dt * xv;
        if (a.skip) add = a.skip[c] * xv;
        if (a.z) gate = silu<T>(to_f32<T>(((const T*)a.z)[b * a.st.z_batch + c]));
    }
    const int part = lane % P, sub = lane / P;     // this lane's states of channel (32 / P) * it + sub
    const int s0 = part * V;
    float Bv[V], Cv[V];
    {
        const T* bp = (const T*)a.Bm + b * a.st.B_batch + (size_t)grp * n;
        const T* cp = (const T*)a.Cm + b * a.st.C_batch + (size_t)grp * n;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            Bv[i] = s0 + i < n ? to_f32<T>(bp[s0 + i]) : 0.f;
            Cv[i] = s0 + i < n ? to_f32<T>(cp[s0 + i]) : 0.f;
        }
    }
    constexpr int STEP = 32 / P;                   // channels per pass
    constexpr int U = P < 4 ? P : 4;               // passes whose loads are in flight together
    float y = 0.f;
    for (int i0 = 0; i0 < P; i0 += U) {
        float hv[U][V], av[U][V];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int ch = (i0 + i) * STEP + sub;
            const size_t c = (size_t)(c0 + (ch < nch ? ch : 0));
            const float* hp = a.h_out + ((size_t)b * a.D + c) * n + s0;
            const float* ap = a.A + c * n + s0;
            const bool on = ch < nch && s0 < n;
            if (V == 4) {
                const float4 hq = on ? __ldcs(reinterpret_cast<const float4*>(hp)) : make_float4(0.f, 0.f, 0.f, 0.f);
                const float4 aq = on ? *reinterpret_cast<const float4*>(ap) : make_float4(0.f, 0.f, 0.f, 0.f);
                hv[i][0] = hq.x; hv[i][V > 1 ? 1 : 0] = hq.y; hv[i][V > 2 ? 2 : 0] = hq.z; hv[i][V > 3 ? 3 : 0] = hq.w;
                av[i][0] = aq.x; av[i][V > 1 ? 1 : 0] = aq.y; av[i][V > 2 ? 2 : 0] = aq.z; av[i][V > 3 ? 3 : 0] = aq.w;
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    hv[i][j] = on && s0 + j < n ? hp[j] : 0.f;
                    av[i][j] = on && s0 + j < n ? ap[j] : 0.f;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int ch = (i0 + i) * STEP + sub;
            const float d = __shfl_sync(~0u, dt, ch) * kLog2e, ux = __shfl_sync(~0u, u, ch);
            float acc = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                hv[i][j] = fmaf(ex2_approx(d * av[i][j]), hv[i][j], ux * Bv[j]);
                acc = fmaf(Cv[j], hv[i][j], acc);
            }
            if (ch < nch && s0 < n) {
                float* hp = a.h_out + ((size_t)b * a.D + c0 + ch) * n + s0;
                if (V == 4) {
                    __stcs(reinterpret_cast<float4*>(hp), make_float4(hv[i][0], hv[i][V > 1 ? 1 : 0], hv[i][V > 2 ? 2 : 0],
                                                                      hv[i][V > 3 ? 3 : 0]));
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (s0 + j < n) hp[j] = hv[i][j];
                }
            }
#pragma unroll
            for (int o = P / 2; o > 0; o /= 2) acc += __shfl_xor_sync(~0u, acc, o);
            // channel ch's sum is in the P lanes of its group; lane ch takes it
            const float got = __shfl_sync(~0u, acc, ((lane % STEP) * P) & 31);
            if (lane / STEP == i0 + i) y = got;
        }
    }
    if (lane < nch) ((T*)a.out)[(size_t)b * a.D + c0 + lane] = from_f32<T>((y + add) * gate);
}

template <typename T, int V, int P>
cudaError_t launch_step_vp(const SsmArgs& a)
{
    const int per = a.D / a.G, tpg = (per + 31) / 32;
    const long long units = (long long)a.B * tpg * a.G;
    const long long grid = (units + kStepWarps - 1) / kStepWarps;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    ssm_step_kernel<T, V, P><<<(unsigned)grid, kStepWarps * 32, 0, a.stream>>>(a, tpg);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) stage_mark(0, a.stream);
    return e;
}

template <typename T>
cudaError_t launch_step_t(const SsmArgs& a)
{
    // whole 16-byte pieces of the state where n allows them, else two states a lane (P <= 32 covers n <= 64)
    if (a.n % 4 == 0) {
        if (a.n <= 4) return launch_step_vp<T, 4, 1>(a);
        if (a.n <= 8) return launch_step_vp<T, 4, 2>(a);
        if (a.n <= 16) return launch_step_vp<T, 4, 4>(a);
        if (a.n <= 32) return launch_step_vp<T, 4, 8>(a);
        return launch_step_vp<T, 4, 16>(a);
    }
    if (a.n <= 2) return launch_step_vp<T, 2, 1>(a);
    if (a.n <= 8) return launch_step_vp<T, 2, 4>(a);
    if (a.n <= 16) return launch_step_vp<T, 2, 8>(a);
    if (a.n <= 32) return launch_step_vp<T, 2, 16>(a);
    return launch_step_vp<T, 2, 32>(a);
}

}  // namespace

cudaError_t launch_ssm_step(const SsmArgs& a)
{
    return a.dtype == LA_BF16 ? launch_step_t<__nv_bfloat16>(a) : launch_step_t<float>(a);
}

}  // namespace la
