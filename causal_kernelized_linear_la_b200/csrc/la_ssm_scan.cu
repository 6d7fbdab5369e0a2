// Selective state-space recurrence.  Per sequence, channel c and state s:
//     dt_t   = delta_t[c] + bias[c], through softplus if asked
//     h_t[s] = exp(dt_t A[c,s]) h_{t-1}[s] + dt_t x_t[c] B_t[s]
//     y_t[c] = (sum_s C_t[s] h_t[s] + D[c] x_t[c]) * silu(z_t[c])
// B and C are shared by the channels of a group.  States, step sizes, decays
// and sums are fp32; y is rounded to the storage type once.
//
// Prompt scan.  A CTA walks the tokens of a few channels in tiles of 16 or 32.
// LANES lanes share a channel, each with NS states in registers, and do nothing
// but the recurrence: per token and pair of states two products, two
// exponentials and two FMAs as packed fp32 pairs, and one partial sum of y.
// Other warps keep them fed and carry their results away: four bring the raw
// rows by cp.async some tiles ahead and put (dt, dt x) and fp32 B, C of the
// next tile into shared memory, four take y of the tile before out of it (the
// lanes' partial sums, skip, gate), so softplus, gate and conversions are done
// once a value, off the recurrence's path.
// The decay needs one exponential per (token, channel, state): the SFU's 16 a
// clock and SM bound the scan (at n = 16 its 2^x alone take three times as
// long as reading delta, x, z and writing y), not memory.  At 8192 tokens x 4096
// channels x 16 states (bf16, softplus, skip, gate) those two floors are 119 and
// 41 us; the kernel takes 264 (fp32 271; four prompts of 4096 tokens, 3.5 waves of
// CTAs, 529).  The recurrence warps issue in order and need about 48 clocks a
// token where the SFU alone needs 32: without exponentials 244 us, with idle
// helpers 199 to 217 (both measured on copies).
//
// Few channels leave SMs idle, so a long sequence is cut into segments: a
// first kernel runs every segment but the last, from a zero state (the first
// from the call's start state), and keeps its end state and sum of dt; since the
// decay over a segment is exp(A sum dt), each segment of the second kernel folds
// the segments before it into its own start state and runs once more with outputs.
#include "f32x2.cuh"
#include "la_internal.cuh"
#include "sm100.cuh"

namespace la {
namespace {

using namespace sm100;

constexpr int kCh = 32;        // channels of a CTA; LANES lanes share one
constexpr int kPrep = 128;     // threads that load and prepare
constexpr int kFin = 128;      // threads that finish y
constexpr int kBufs = 3;       // prepared tiles: one in the recurrence, one being finished, one being prepared
constexpr int kRaw = kBufs + 4;   // tiles of raw rows: those of the prepared tiles and one being prepared, the others in flight
constexpr float kLog2e = 1.4426950408889634f;
// The SFU's 2^x comes out low on average (measured, in units of 2^-24: 0.09 to
// 0.17 for x in [-0.003, 0], 0.30 to 0.44 for x in [-1, -0.003]), and a slow state's
// many decays add that up.  So each exponent is lifted by the middle of its
// range, in log2 units; which one goes by the step size against a limit per
// lane, where the exponent in the lane's middle passes 0.003.  2^lift itself is
// exactly 1: a step of zero changes nothing.
constexpr float kLiftSlow = 0.12f * 5.9604645e-8f * kLog2e, kLiftFast = 0.36f * 5.9604645e-8f * kLog2e;
constexpr float kSlow = 0.003f;
__device__ __forceinline__ float lift_limit(float a2_first, float a2_last) { return kSlow / (0.5f * fabsf(a2_first + a2_last)); }

// A decay rate in log2 units.  An infinite one (a state that keeps nothing) becomes the largest finite: the
// tokens behind a sequence in its last tile take no step, and 0 * inf is not the 0 that keeps the state.
__device__ __forceinline__ float log2_rate(float a)
{
    const float r = a * kLog2e;
    return r == -INFINITY ? -3.4028235e38f : r;
}

struct Lens {
    int use;
    int n[kMaxSeqLens];
};

// log(1 + e^v) = max(v, 0) + log1p(e), e = e^-|v| in (0, 1], and log1p(e) =
// 2 atanh(r) with r = e / (2 + e) <= 1/3: the odd series of atanh to r^13 is
// off by r^14 / 15 < 2e-8 relative.
__device__ __forceinline__ float softplus(float v)
{
    const float e = ex2_approx(-fabsf(v) * kLog2e);
    const float r = e * rcp_approx(2.f + e), q = r * r;
    float p = fmaf(q, 1.f / 13.f, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    p = fmaf(p, q, 1.f);
    return fmaf(2.f * r, p, fmaxf(v, 0.f));
}
template <typename T> __device__ __forceinline__ float silu(float v);
template <> __device__ __forceinline__ float silu<float>(float v) { return silu_f32(v); }
template <> __device__ __forceinline__ float silu<__nv_bfloat16>(float v) { return silu_approx(v); }

__device__ __forceinline__ void cp_async16(void* dst, const void* src, uint32_t src_bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(src_bytes)
                 : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t id, uint32_t count)
{
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// A tile of `rows` (of ROWS) x `cols` (of PITCH) elements of a row-major
// tensor into shared memory, zeros elsewhere, by the preparing threads, where
// rows do not start on 16 bytes.  A thread keeps its column: copies of 4 bytes, or ...
template <typename T, int ROWS, int PITCH>
__device__ __forceinline__ void copy_words(T* dst, const T* src, long long row_stride, int rows, int cols, int tid)
{
    constexpr int PER = 4 / (int)sizeof(T), N = PITCH / PER, STEP = kPrep / N;   // pieces of a row, rows of a pass
    static_assert(kPrep % N == 0 && ROWS % STEP == 0, "a thread keeps its columns");
    const int c = tid % N * PER, t0 = tid / N;
    const int left = min(PER, max(0, cols - c));
    const T* s = src + (left > 0 ? t0 * row_stride + c : 0);
    const long long step = left > 0 ? STEP * row_stride : 0;
    T* d = dst + t0 * PITCH + c;
    if (rows >= ROWS) {
#pragma unroll
        for (int i = 0; i < ROWS / STEP; ++i, s += step) cp_async4(d + i * STEP * PITCH, s, left * sizeof(T));
    } else {
#pragma unroll
        for (int i = 0; i < ROWS / STEP; ++i, s += step) {
            const bool on = t0 + i * STEP < rows;
            cp_async4(d + i * STEP * PITCH, on ? s : src, on ? left * sizeof(T) : 0);
        }
    }
}
// ... single elements (2 bytes are no size of a copy) through registers: loaded
// for one tile while the tile before it is put down.
template <typename T, int ROWS, int PITCH>
struct Elements {
    static constexpr int STEP = kPrep / PITCH, COUNT = ROWS / STEP;
    static_assert(kPrep % PITCH == 0 && ROWS % STEP == 0, "a thread keeps its column");
    T v[COUNT];
    __device__ __forceinline__ void load(const T* src, long long row_stride, int rows, int cols, int tid)
    {
        const int c = tid % PITCH, t0 = tid / PITCH;
        const T* s = src + t0 * row_stride + c;
#pragma unroll
        for (int i = 0; i < COUNT; ++i, s += STEP * row_stride)
            v[i] = c < cols && t0 + i * STEP < rows ? *s : from_f32<T>(0.f);
    }
    __device__ __forceinline__ void store(T* dst, int tid) const
    {
        T* d = dst + tid / PITCH * PITCH + tid % PITCH;
#pragma unroll
        for (int i = 0; i < COUNT; ++i) d[i * STEP * PITCH] = v[i];
    }
};

// Two neighbouring values (the first at an even place).
template <typename T> __device__ __forceinline__ float2 load2(const T* p);
template <> __device__ __forceinline__ float2 load2<float>(const float* p) { return *reinterpret_cast<const float2*>(p); }
template <> __device__ __forceinline__ float2 load2<__nv_bfloat16>(const __nv_bfloat16* p)
{
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
}
__device__ __forceinline__ void store2(float* p, float a, float b) { *reinterpret_cast<float2*>(p) = make_float2(a, b); }
__device__ __forceinline__ void store2(__nv_bfloat16* p, float a, float b)
{
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}

// Bytes of shared memory with tiles of tt tokens: the raw tiles, kBufs prepared buffers.
constexpr int plan_bytes(int esize, int ns, int lanes, int tt)
{
    const int ch = kCh, np = lanes * ns, bcp = np < 8 ? 8 : np;
    return kRaw * tt * (3 * ch + 2 * bcp) * esize + kBufs * tt * (ch * 8 + np * 8 + lanes * (ch + 8) * 4);
}

// LANES lanes share a channel, NS states each; tiles of TT tokens: 32 halve the
// barriers a token costs, 16 where shared memory does not hold 32.
template <typename T, int NS, int LANES>
struct Plan {
    static constexpr int TT = plan_bytes(sizeof(T), NS, LANES, 32) <= 232448 ? 32 : 16;
    static constexpr int CH = kCh;
    static constexpr int REC = kCh * LANES, THREADS = REC + kPrep + kFin;   // threads of the recurrence, of the CTA
    static constexpr int NP = LANES * NS;          // states, padded
    static constexpr int BCP = NP < 8 ? 8 : NP;    // elements of a raw B or C row: whole 16-byte pieces
    static constexpr int ROW = TT * CH * (int)sizeof(T), BC = TT * BCP * (int)sizeof(T);
    static constexpr int STAGE = 3 * ROW + 2 * BC; // raw x, delta, z, B, C
    // partial sums of y: [TT][LANES][CH], 8 floats of padding a row put a warp's LANES rows on different banks
    static constexpr int YP = CH + 8, YROW = LANES * YP;
    // a buffer of prepared values: (dt, dt x) [TT][CH], (B.., C..) [TT][LANES][2 NS], y parts
    static constexpr int DU = TT * CH * 8, BCF = TT * NP * 2 * 4, Y = TT * YROW * 4;
    static constexpr int BUF = DU + BCF + Y;
    static constexpr int OFF_BUF = kRaw * STAGE;
    static constexpr int BYTES = OFF_BUF + kBufs * BUF;
    // 16-byte pieces of a raw row and of a tile
    static constexpr int XP = CH * (int)sizeof(T) / 16, BP = BCP * (int)sizeof(T) / 16;
    static constexpr int PIECES = TT * (3 * XP + 2 * BP), SLOTS = (PIECES + kPrep - 1) / kPrep;
};

// Floats of a segment's summary: end states from zero [CH][NP], then sums of dt [CH].
template <int NS, int LANES> __host__ __device__ constexpr int slot_floats() { return kCh * (LANES * NS + 1); }

// Named barriers over the whole CTA; + buffer (tile % kBufs).
//   kReady: the preparing threads (its values are in) and the finishing threads (its y parts are free) arrive,
//           the recurrence waits
//   kDone:  the recurrence arrives, the others wait
enum Bars : uint32_t { kReady = 1, kDone = kReady + kBufs, kPrepBar = kDone + kBufs };

// grid: (channel tiles, segments, sequences).  SUMMARY: the first kernel of a
// segmented scan; otherwise outputs and the final state.
// PIECE: how rows come into shared memory, by what their starts are aligned to:
// copies of 16 bytes, of 4, or single elements of 2 through registers (4096
// tokens and about 4096 channels x 16 states: bf16 134 us with pieces of 16, 177 of 2;
// fp32 137 of 16, 191 of 4).
template <typename T, int NS, int LANES, bool SUMMARY, int PIECE>
__global__ void __launch_bounds__(Plan<T, NS, LANES>::THREADS, 1)
ssm_scan_kernel(const __grid_constant__ SsmArgs a, const __grid_constant__ Lens lens, int tiles_per_group)
{
    using P = Plan<T, NS, LANES>;
    constexpr int NP = P::NP, CH = P::CH, TT = P::TT, kRec = P::REC, kThreads = P::THREADS;
    static_assert(P::BYTES <= 232448 && P::BYTES == plan_bytes(sizeof(T), NS, LANES, TT), "shared memory plan");
    extern __shared__ __align__(16) unsigned char sm[];
    const int b = blockIdx.z, seg = blockIdx.y, tile = blockIdx.x;
    const int grp = tile / tiles_per_group, per = a.D / a.G;
    const int cg0 = (tile % tiles_per_group) * CH;     // first channel inside the group
    const int c0 = grp * per + cg0, nch = min(CH, per - cg0);
    const int len = lens.use ? lens.n[b] : a.N;
    const int s0 = seg * a.seg_len, s1 = min(len, s0 + a.seg_len);
    const size_t unit0 = ((size_t)b * gridDim.x + tile) * a.segs;   // this chain's first summary slot

    if (SUMMARY) grid_launch_dependents();
    if (s0 >= len && !(seg == 0 && !SUMMARY)) return;   // an empty sequence still reports its start state
    const int nt = s0 < s1 ? (s1 - s0 + TT - 1) / TT : 0;

    if (threadIdx.x < kRec) {
        // ---------------- the recurrence ----------------
        // neighbouring lanes are channels: the lanes that read one (B, C) piece sit side by side,
        // which halves the shared-memory cycles of a 16-byte read (2 instead of 4, measured)
        constexpr int WCH = 32 / LANES;    // channels of a warp
        const int ch = threadIdx.x / 32 * WCH + threadIdx.x % WCH, l = threadIdx.x % 32 / WCH;
        const bool mine = ch < nch;
        const int c = c0 + (mine ? ch : 0);
        // this lane's decay rates (in log2 units) and states; padded states stay zero
        f2 A2[(NS + 1) / 2], h[(NS + 1) / 2];
#pragma unroll
        for (int i = 0; i < NS; i += 2) {
            const int s = l * NS + i;
            const float* ap = a.A + (size_t)c * a.n;
            A2[i / 2] = pack2(mine && s < a.n ? log2_rate(ap[s]) : 0.f,
                              NS > 1 && mine && s + 1 < a.n ? log2_rate(ap[s + 1]) : 0.f);
            const float* hp = a.h0 + ((size_t)b * a.D + c) * a.n;
            const bool from = a.h0 && mine && seg == 0;
            h[i / 2] = pack2(from && s < a.n ? hp[s] : 0.f, NS > 1 && from && s + 1 < a.n ? hp[s + 1] : 0.f);
        }
        if (!SUMMARY && a.segs > 1) {
            grid_dependency_wait();   // the summaries
            for (int g = 0; g < seg; ++g) {
                const float* slot = a.workspace + (unit0 + g) * slot_floats<NS, LANES>();
                const float dt = slot[CH * NP + ch];
#pragma unroll
                for (int i = 0; i < NS; i += 2) {
                    const float2 ar = unpack2(A2[i / 2]);
                    const float* e = slot + ch * NP + l * NS + i;
                    h[i / 2] = fma2(pack2(ex2_approx(dt * ar.x), ex2_approx(dt * ar.y)), h[i / 2],
                                    pack2(e[0], NS > 1 ? e[1] : 0.f));
                }
            }
        }
        // Tokens go NB at a time: decays, written terms and C of the next NB are
        // loaded and computed ahead of this NB's chain of FMAs, so that the
        // exponentials (8 clocks each) and the chain overlap in one warp; the
        // loads also come before the stores of y, above which none is moved.
        constexpr int NB = NS <= 2 ? 4 : NS == 4 ? 4 : 2, NH = (NS + 1) / 2;
        const float slow_below = lift_limit(unpack2(A2[0]).x, NS > 1 ? unpack2(A2[NH - 1]).y : unpack2(A2[0]).x);
        float2 dv[2][NB];                               // (dt, dt x)
        f2 dec[2][NB][NH], bv[2][NB][NH], cv[2][NB][NH];
        auto load = [&](int k, int t0, int w) {
            const unsigned char* buf = sm + P::OFF_BUF + (k % kBufs) * P::BUF;
            const float2* du = reinterpret_cast<const float2*>(buf) + ch;
            const float* bc = reinterpret_cast<const float*>(buf + P::DU) + l * 2 * NS;
#pragma unroll
            for (int t = 0; t < NB; ++t) {
                dv[w][t] = du[(t0 + t) * CH];
                const float* q = bc + (t0 + t) * NP * 2;
                if (NS == 1) {
                    const float2 v = *reinterpret_cast<const float2*>(q);
                    bv[w][t][0] = pack2(v.x, 0.f);
                    cv[w][t][0] = pack2(v.y, 0.f);
                } else if (NS == 2) {
                    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(q);
                    bv[w][t][0] = v.x;
                    cv[w][t][0] = v.y;
                } else {
#pragma unroll
                    for (int i = 0; i < NH; i += 2) {
                        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(q + 2 * i);
                        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(q + NS + 2 * i);
                        bv[w][t][i] = v.x;
                        bv[w][t][i + (NH > 1)] = v.y;
                        cv[w][t][i] = x.x;
                        cv[w][t][i + (NH > 1)] = x.y;
                    }
                }
            }
        };
        auto decays = [&](int t, int w) {
            const f2 dt = pack2(dv[w][t].x, dv[w][t].x);
            // the first of each two tokens decides: 4 us of 260 more than one lift for all
            // exponents (every token deciding: 11 us), but that left some states' errors at two to
            // four times those of exact decays
            const float up = dv[w][t & ~1].x < slow_below ? kLiftSlow : kLiftFast;
            const f2 lift = pack2(up, up);
#pragma unroll
            for (int i = 0; i < NH; ++i) {
                const float2 e = unpack2(fma2(dt, A2[i], lift));
                dec[w][t][i] = pack2(ex2_approx(e.x), NS > 1 ? ex2_approx(e.y) : 0.f);
            }
        };
        for (int k = 0; k < nt; ++k) {
            float* yp = reinterpret_cast<float*>(sm + P::OFF_BUF + (k % kBufs) * P::BUF + P::DU + P::BCF) + l * P::YP + ch;
            named_bar(kReady + k % kBufs, kThreads);
            load(k, 0, 0);
#pragma unroll
            for (int t = 0; t < NB; ++t) decays(t, 0);
#pragma unroll
            for (int t0 = 0; t0 < TT; t0 += NB) {
                const int w = t0 / NB & 1;
                const bool more = t0 + NB < TT;
                if (more) load(k, t0 + NB, w ^ 1);
#pragma unroll
                for (int t = 0; t < NB; ++t) {
                    const f2 u = pack2(dv[w][t].y, dv[w][t].y);
                    f2 acc = 0;
#pragma unroll
                    for (int i = 0; i < NH; ++i) {
                        h[i] = fma2(dec[w][t][i], h[i], mul2(u, bv[w][t][i]));
                        acc = i == 0 ? mul2(cv[w][t][i], h[i]) : fma2(cv[w][t][i], h[i], acc);
                    }
                    if (more) decays(t, w ^ 1);
                    if (!SUMMARY) {
                        const float2 q = unpack2(acc);
                        yp[(t0 + t) * P::YROW] = q.x + q.y;
                    }
                }
            }
            bar_arrive(kDone + k % kBufs, kThreads);
        }
        if (SUMMARY) {
            float* slot = a.workspace + (unit0 + seg) * slot_floats<NS, LANES>();
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
    } else if (threadIdx.x < kRec + kPrep) {
        // ---------------- load and prepare ----------------
        const int tid = threadIdx.x - kRec;
        const int cc = tid % (CH / 2) * 2, tr = tid / (CH / 2);   // this thread's channels cc, cc + 1 and first row
        constexpr int TR = kPrep / (CH / 2);                      // rows a pass covers
        const T* xp = (const T*)a.x + b * a.st.x_batch + s0 * a.st.x_row + c0;
        const T* dp = (const T*)a.delta + b * a.st.delta_batch + s0 * a.st.delta_row + c0;
        const T* zp = a.z ? (const T*)a.z + b * a.st.z_batch + s0 * a.st.z_row + c0 : nullptr;
        const T* bp = (const T*)a.Bm + b * a.st.B_batch + s0 * a.st.B_row + (size_t)grp * a.n;
        const T* cp = (const T*)a.Cm + b * a.st.C_batch + s0 * a.st.C_row + (size_t)grp * a.n;
        float bias[2], dt_sum[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 2; ++j) bias[j] = a.delta_bias && cc + j < nch ? a.delta_bias[c0 + cc + j] : 0.f;

        // this thread's 16-byte pieces of every tile, where all rows start on 16 bytes
        const char* src[P::SLOTS];
        long long step[P::SLOTS];
        int dst[P::SLOTS], rowof[P::SLOTS];      // rowof: the piece's token of the tile, past TT where there is nothing to read
        uint32_t bytes[P::SLOTS];
        if constexpr (PIECE == 16) {
#pragma unroll
            for (int i = 0; i < P::SLOTS; ++i) {
                const int e = tid + i * kPrep;
                const bool is_x = e < TT * 3 * P::XP;
                const int r = is_x ? e % (TT * P::XP) : (e - TT * 3 * P::XP) % (TT * P::BP);
                const int which = is_x ? e / (TT * P::XP) : 3 + (e - TT * 3 * P::XP) / (TT * P::BP);
                const int n16 = is_x ? P::XP : P::BP, t = r / n16, col = r % n16 * (16 / (int)sizeof(T));
                const T* base = which == 0 ? xp : which == 1 ? dp : which == 2 ? zp : which == 3 ? bp : cp;
                const long long row = which == 0 ? a.st.x_row : which == 1 ? a.st.delta_row : which == 2 ? a.st.z_row :
                                      which == 3 ? a.st.B_row : a.st.C_row;
                const int left = (is_x ? nch : a.n) - col;
                const bool on = e < P::PIECES && left > 0 && base && !(SUMMARY && (which == 2 || which == 4));
                src[i] = (const char*)(base ? base + t * row + col : xp);
                step[i] = row * TT * (long long)sizeof(T);
                dst[i] = (which < 3 ? which * P::ROW : 3 * P::ROW + (which - 3) * P::BC) + r * 16;
                bytes[i] = on ? min(left * (int)sizeof(T), 16) : 0;
                rowof[i] = on ? t : 0x3fffffff;
                if (e >= P::PIECES) dst[i] = -1;
            }
        }
        Elements<T, TT, CH> ex, ed, ez;
        Elements<T, TT, P::BCP> eb, ec;
        static_assert(kRaw - kBufs - 1 >= 2, "single elements reach shared memory one tile later than copies");
        auto raw = [&](int k) { return sm + (k % kRaw) * P::STAGE; };
        auto fetch = [&](int k) {
            const int rows = s1 - s0 - k * TT;
            [[maybe_unused]] const long long t = (long long)k * TT;
            if constexpr (PIECE == 16) {
                if (k < nt) {
                    unsigned char* st = raw(k);
#pragma unroll
                    for (int i = 0; i < P::SLOTS; ++i) {
                        if (dst[i] >= 0) {
                            const bool on = rowof[i] < rows;
                            cp_async16(st + dst[i], on ? src[i] : (const char*)xp, on ? bytes[i] : 0);
                        }
                        src[i] += step[i];
                    }
                }
            } else if constexpr (PIECE == 4) {
                if (k < nt) {
                    unsigned char* st = raw(k);
                    copy_words<T, TT, CH>((T*)st, xp + t * a.st.x_row, a.st.x_row, rows, nch, tid);
                    copy_words<T, TT, CH>((T*)(st + P::ROW), dp + t * a.st.delta_row, a.st.delta_row, rows, nch, tid);
                    if (!SUMMARY && zp)
                        copy_words<T, TT, CH>((T*)(st + 2 * P::ROW), zp + t * a.st.z_row, a.st.z_row, rows, nch, tid);
                    copy_words<T, TT, P::BCP>((T*)(st + 3 * P::ROW), bp + t * a.st.B_row, a.st.B_row, rows, a.n, tid);
                    if (!SUMMARY)
                        copy_words<T, TT, P::BCP>((T*)(st + 3 * P::ROW + P::BC), cp + t * a.st.C_row, a.st.C_row, rows,
                                                  a.n, tid);
                }
            } else {
                if (k > 0 && k <= nt) {
                    unsigned char* st = raw(k - 1);
                    ex.store((T*)st, tid);
                    ed.store((T*)(st + P::ROW), tid);
                    if (!SUMMARY && zp) ez.store((T*)(st + 2 * P::ROW), tid);
                    eb.store((T*)(st + 3 * P::ROW), tid);
                    if (!SUMMARY) ec.store((T*)(st + 3 * P::ROW + P::BC), tid);
                }
                if (k < nt) {
                    ex.load(xp + t * a.st.x_row, a.st.x_row, rows, nch, tid);
                    ed.load(dp + t * a.st.delta_row, a.st.delta_row, rows, nch, tid);
                    if (!SUMMARY && zp) ez.load(zp + t * a.st.z_row, a.st.z_row, rows, nch, tid);
                    eb.load(bp + t * a.st.B_row, a.st.B_row, rows, a.n, tid);
                    if (!SUMMARY) ec.load(cp + t * a.st.C_row, a.st.C_row, rows, a.n, tid);
                }
            }
            cp_async_commit();
        };
        // (B.., C..) of one lane and token side by side
        auto spread = [&](float* bc, const T* bs, const T* cs) {
            if (NS == 1) {
#pragma unroll
                for (int e = tid; e < TT * NP; e += kPrep) {
                    const int t = e / NP, s = e % NP;
                    bc[e * 2] = to_f32<T>(bs[t * P::BCP + s]);
                    if (!SUMMARY) bc[e * 2 + 1] = to_f32<T>(cs[t * P::BCP + s]);
                }
            } else {
#pragma unroll
                for (int e = tid; e < TT * NP / 2; e += kPrep) {
                    const int t = e / (NP / 2), s = e % (NP / 2) * 2;
                    float* to = bc + t * NP * 2 + s / NS * 2 * NS + s % NS;
                    *reinterpret_cast<float2*>(to) = load2<T>(bs + t * P::BCP + s);
                    if (!SUMMARY) *reinterpret_cast<float2*>(to + NS) = load2<T>(cs + t * P::BCP + s);
                }
            }
        };
#pragma unroll
        for (int k = 0; k < kRaw - kBufs - 1; ++k) fetch(k);
        for (int k = 0; k < nt; ++k) {
            // tile k - kBufs is through the recurrence (its buffer is free) and the one before it is finished (its raw
            // rows are free)
            if (k >= kBufs) named_bar(kDone + k % kBufs, kThreads);
            cp_async_wait<kRaw - kBufs - 2>();
            named_bar(kPrepBar, kPrep);               // tile k is in shared memory for every preparing thread
            const unsigned char* st = raw(k);
            unsigned char* buf = sm + P::OFF_BUF + (k % kBufs) * P::BUF;
            const T* xs = (const T*)st;
            const T* ds = (const T*)(st + P::ROW);
            float2* du = reinterpret_cast<float2*>(buf);
            const int rows = s1 - s0 - k * TT;
            spread(reinterpret_cast<float*>(buf + P::DU), (const T*)(st + 3 * P::ROW), (const T*)(st + 3 * P::ROW + P::BC));
#pragma unroll
            for (int i = 0; i < (TT + TR - 1) / TR; ++i) {
                const int t = tr + i * TR;
                if (TR > TT && t >= TT) break;
                const float2 d2 = load2<T>(ds + t * CH + cc), x2 = load2<T>(xs + t * CH + cc);
                float dt[2] = {d2.x + bias[0], d2.y + bias[1]};
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (a.softplus) dt[j] = softplus(dt[j]);
                    if (t >= rows) dt[j] = 0.f;           // decay 1, nothing added
                    if (SUMMARY) dt_sum[j] += dt[j];
                }
                *reinterpret_cast<float4*>(du + t * CH + cc) = make_float4(dt[0], dt[0] * x2.x, dt[1], dt[1] * x2.y);
            }
            bar_arrive(kReady + k % kBufs, kThreads);
            fetch(k + kRaw - kBufs - 1);                  // into the rows of tile k - kBufs - 1
        }
        // the barriers that the other threads still pass
        for (int k = max(nt, kBufs); k < nt + kBufs; ++k) named_bar(kDone + k % kBufs, kThreads);
        if (SUMMARY) {
            // sum of dt over the threads of each channel
            named_bar(kPrepBar, kPrep);
            float* part = reinterpret_cast<float*>(sm);
            part[tr * CH + cc] = dt_sum[0];
            part[tr * CH + cc + 1] = dt_sum[1];
            named_bar(kPrepBar, kPrep);
            if (tid < CH) {
                float sum = 0.f;
                for (int i = 0; i < TR; ++i) sum += part[i * CH + tid];
                a.workspace[(unit0 + seg) * slot_floats<NS, LANES>() + CH * NP + tid] = sum;
            }
        }
    } else {
        // ---------------- finish y ----------------
        const int tid = threadIdx.x - kRec - kPrep;
        const int cc = tid % (CH / 2) * 2, tr = tid / (CH / 2);
        constexpr int TR = kFin / (CH / 2);
        float skip[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) skip[j] = !SUMMARY && a.skip && cc + j < nch ? a.skip[c0 + cc + j] : 0.f;
        // rows of out that take two values in one store
        const bool pairs = a.D % 2 == 0 && c0 % 2 == 0 && nch % 2 == 0 && reinterpret_cast<uintptr_t>(a.out) % (2 * sizeof(T)) == 0;
        T* op = (T*)a.out + ((size_t)b * a.N + s0) * a.D + c0 + cc;
        for (int k = 0; k < min(nt, kBufs); ++k) bar_arrive(kReady + k, kThreads);     // the y parts are free
        for (int k = 0; k < nt; ++k) {
            named_bar(kDone + k % kBufs, kThreads);
            if (!SUMMARY) {
                const unsigned char* st = sm + (k % kRaw) * P::STAGE;
                const float* yp = reinterpret_cast<const float*>(sm + P::OFF_BUF + (k % kBufs) * P::BUF + P::DU + P::BCF) + cc;
                const T* xs = (const T*)st;
                const T* zs = (const T*)(st + 2 * P::ROW);
                const int rows = s1 - s0 - k * TT;
#pragma unroll 4
                for (int i = 0; i < (TT + TR - 1) / TR; ++i) {
                    const int t = tr + i * TR;
                    if (TR > TT && t >= TT) break;
                    const float2 x2 = load2<T>(xs + t * CH + cc);
                    float y[2] = {0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < LANES; ++j) {
                        const float2 p = *reinterpret_cast<const float2*>(yp + t * P::YROW + j * P::YP);
                        y[0] += p.x;
                        y[1] += p.y;
                    }
                    y[0] = fmaf(skip[0], x2.x, y[0]);
                    y[1] = fmaf(skip[1], x2.y, y[1]);
                    if (a.z) {
                        const float2 z2 = load2<T>(zs + t * CH + cc);
                        y[0] *= silu<T>(z2.x);
                        y[1] *= silu<T>(z2.y);
                    }
                    T* o = op + (size_t)(k * TT + t) * a.D;
                    if (t < rows && pairs && cc < nch) store2(o, y[0], y[1]);
                    else if (t < rows) {
                        if (cc < nch) o[0] = from_f32<T>(y[0]);
                        if (cc + 1 < nch) o[1] = from_f32<T>(y[1]);
                    }
                }
            }
            if (k + kBufs < nt) bar_arrive(kReady + k % kBufs, kThreads);
        }
    }
}

// Largest piece (16, 4 or the element's own bytes) that divides an address and its row strides.
int piece_of(const void* p, long long batch, long long row, int e)
{
    const unsigned long long m = reinterpret_cast<uintptr_t>(p) | (unsigned long long)(batch * e) | (unsigned long long)(row * e);
    return m % 16 == 0 ? 16 : m % 4 == 0 ? 4 : e;
}

template <typename T, int NS, int LANES, int PIECE>
cudaError_t launch_scan_piece(const SsmArgs& a)
{
    using P = Plan<T, NS, LANES>;
    const int per = a.D / a.G, tpg = (per + P::CH - 1) / P::CH;
    Lens lens{};
    lens.use = a.seq_lens != nullptr;
    if (a.seq_lens)
        for (int b = 0; b < a.B; ++b) lens.n[b] = a.seq_lens[b];
    auto main_k = ssm_scan_kernel<T, NS, LANES, false, PIECE>;
    auto sum_k = ssm_scan_kernel<T, NS, LANES, true, PIECE>;
    cudaError_t err = cudaFuncSetAttribute(main_k, cudaFuncAttributeMaxDynamicSharedMemorySize, P::BYTES);
    if (err == cudaSuccess) err = cudaFuncSetAttribute(sum_k, cudaFuncAttributeMaxDynamicSharedMemorySize, P::BYTES);
    if (err != cudaSuccess) return err;
    int stage = 0;
    if (a.segs > 1) {
        sum_k<<<dim3(tpg * a.G, a.segs - 1, a.B), P::THREADS, P::BYTES, a.stream>>>(a, lens, tpg);
        if ((err = cudaGetLastError()) != cudaSuccess) return err;
        stage_mark(stage++, a.stream);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(tpg * a.G, a.segs, a.B);
    cfg.blockDim = dim3(P::THREADS);
    cfg.dynamicSmemBytes = P::BYTES;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = a.segs > 1 ? 1 : 0;
    err = cudaLaunchKernelEx(&cfg, main_k, a, lens, tpg);
    if (err == cudaSuccess) stage_mark(stage, a.stream);
    return err;
}

template <typename T, int NS, int LANES>
cudaError_t launch_scan_ns(const SsmArgs& a)
{
    const int e = sizeof(T), per = a.D / a.G;
    // a group's channels start per * group elements into a row
    const long long goff = a.G > 1 ? per : 0, noff = a.G > 1 ? a.n : 0;
    int px = piece_of(a.x, a.st.x_batch, a.st.x_row, e);
    px = min(px, piece_of(a.delta, a.st.delta_batch, a.st.delta_row, e));
    if (a.z) px = min(px, piece_of(a.z, a.st.z_batch, a.st.z_row, e));
    px = min(px, piece_of(nullptr, goff, 0, e));
    int pb = piece_of(a.Bm, a.st.B_batch, a.st.B_row, e);
    pb = min(pb, piece_of(a.Cm, a.st.C_batch, a.st.C_row, e));
    pb = min(pb, piece_of(nullptr, noff, 0, e));
    const int piece = min(px, pb);
    if (piece == 16) return launch_scan_piece<T, NS, LANES, 16>(a);
    if (piece == 4) return launch_scan_piece<T, NS, LANES, 4>(a);
    if constexpr (sizeof(T) == 2) return launch_scan_piece<T, NS, LANES, 2>(a);
    return cudaErrorInvalidValue;   // an fp32 element is 4 bytes
}

template <typename T>
cudaError_t launch_scan_t(const SsmArgs& a)
{
    if (a.n <= 4) return launch_scan_ns<T, 1, 4>(a);
    if (a.n <= 8) return launch_scan_ns<T, 2, 4>(a);
    if (a.n <= 16) return launch_scan_ns<T, 4, 4>(a);
    if (a.n <= 32) return launch_scan_ns<T, 8, 4>(a);
    return launch_scan_ns<T, 8, 8>(a);
}

}  // namespace

void ssm_scan_segments(int B, int N, int D, int G, int n, int* segs, int* seg_len)
{
    const long long units = (long long)B * G * ((D / G + kCh - 1) / kCh);
    int g = 1;
    // a segment more than one costs a second pass over the exponentials
    if (units < 60) g = (int)max(1ll, min(min(148 / units, (long long)N / 128), 64ll));
    const int L = ((N + g - 1) / g + 31) / 32 * 32;   // whole tiles
    *seg_len = L > 0 ? L : 32;
    *segs = N > 0 ? (N + *seg_len - 1) / *seg_len : 1;
}

size_t ssm_scan_workspace_bytes(int B, int N, int D, int G, int n)
{
    int segs, len;
    ssm_scan_segments(B, N, D, G, n, &segs, &len);
    if (segs <= 1) return 0;
    const int np = n <= 4 ? 4 : n <= 8 ? 8 : n <= 16 ? 16 : n <= 32 ? 32 : 64;
    return (size_t)B * G * ((D / G + kCh - 1) / kCh) * segs * kCh * (np + 1) * sizeof(float);
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
// parts of y by shuffles.  256 sequences x 4096 channels x 16 states, bf16: 24.4 us
// (5.9 TB/s, 90 % of the measured copy rate).
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

    constexpr int STEP = 32 / P;                   // channels per pass
    constexpr int U = P < 4 ? P : 4;               // passes whose loads are in flight together
    const int part = lane % P, sub = lane / P;     // this lane's states of channel STEP * pass + sub
    const int s0 = part * V;
    float hv[U][V], av[U][V];
    // this lane's place in the tile's states and decay rates; a pass is STEP channels on
    const int mine = sub * n + s0;
    float* const hb = a.h_out + ((size_t)b * a.D + c0) * n + mine;
    const float* const ab = a.A + (size_t)c0 * n + mine;
    const int last = s0 < n ? nch - sub : 0;       // passes below last / STEP hold a channel
    auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const float* hp = hb + (i0 + i) * STEP * n;
            const float* ap = ab + (i0 + i) * STEP * n;
            const bool on = (i0 + i) * STEP < last;
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
    };
    load(0);     // the states are on their way while the scalars are prepared

    float dt = 0.f, u = 0.f, add = 0.f, gate = 1.f;
    float Bv[V], Cv[V];
    {
        const T* bp = (const T*)a.Bm + b * a.st.B_batch + (size_t)grp * n + s0;
        const T* cp = (const T*)a.Cm + b * a.st.C_batch + (size_t)grp * n + s0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            Bv[i] = s0 + i < n ? to_f32<T>(bp[i]) : 0.f;
            Cv[i] = s0 + i < n ? to_f32<T>(cp[i]) : 0.f;
        }
    }
    if (lane < nch) {
        const int c = c0 + lane;
        const float xv = to_f32<T>(((const T*)a.x)[b * a.st.x_batch + c]);
        dt = to_f32<T>(((const T*)a.delta)[b * a.st.delta_batch + c]) + (a.delta_bias ? a.delta_bias[c] : 0.f);
        if (a.softplus) dt = softplus(dt);
        u = dt * xv;
        if (a.skip) add = a.skip[c] * xv;
        if (a.z) gate = silu<T>(to_f32<T>(((const T*)a.z)[b * a.st.z_batch + c]));
    }
    float y = 0.f;
    for (int i0 = 0; i0 < P; i0 += U) {
        if (i0 > 0) load(i0);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int ch = (i0 + i) * STEP + sub;
            const float d = __shfl_sync(~0u, dt, ch) * kLog2e, ux = __shfl_sync(~0u, u, ch);
            // the lift of the prompt scan's decays
            const float up = fabsf(d * (av[i][0] + av[i][V - 1])) < 2.f * kSlow ? kLiftSlow : kLiftFast;
            float acc = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                hv[i][j] = fmaf(ex2_approx(fmaf(d, av[i][j], up)), hv[i][j], ux * Bv[j]);
                acc = fmaf(Cv[j], hv[i][j], acc);
            }
            if ((i0 + i) * STEP < last) {
                float* hp = hb + (i0 + i) * STEP * n;
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
