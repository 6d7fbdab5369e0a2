// C ABI entry points: argument validation and dispatch to the kernels.
// Nothing here computes; every step of the path runs in the kernels.
#include <stdint.h>

#include "la_internal.cuh"
#include "la_overlap.cuh"
#include "la_prefill_tc.cuh"
#include "la_window.cuh"

namespace la {
namespace {

bool aligned16(const void* p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool head_ok(int x) { return x == 64 || x == 128; }

// Byte ranges [a, a + na) and [b, b + nb) share at least one byte.
bool overlap(const void* a, size_t na, const void* b, size_t nb)
{
    if (!a || !b || na == 0 || nb == 0) return false;
    const char* pa = static_cast<const char*>(a);
    const char* pb = static_cast<const char*>(b);
    return pa < pb + nb && pb < pa + na;
}

// The final-state outputs of a prefill share no byte with its start state:
// blocks of one call read S0 / z0 while others write S_out / z_out.
bool state_outputs_alias(const float* S_out, const float* z_out, const float* S0, const float* z0, int B, int H, int d,
                         int dv)
{
    const size_t chains = (size_t)B * H;
    const size_t sb = chains * d * dv * sizeof(float), zb = chains * d * sizeof(float);
    const void* outs[2] = {S_out, z_out};
    const size_t on[2] = {sb, zb};
    const void* ins[2] = {S0, z0};
    const size_t in_n[2] = {sb, zb};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j)
            if (overlap(outs[i], on[i], ins[j], in_n[j])) return true;
    return false;
}

// Stage events of la_set_stage_events (process-wide; see la.h).
constexpr int kMaxStageEvents = 16;
cudaEvent_t g_stage_events[kMaxStageEvents];
int g_stage_count = 0;

la_status from_cuda(cudaError_t e) { return e == cudaSuccess ? LA_OK : LA_ERR_CUDA; }

}  // namespace

void stage_mark(int i, cudaStream_t stream)
{
    if (i < g_stage_count) cudaEventRecord(g_stage_events[i], stream);
}

// bf16 kernelized prefill runs on the tensor cores; fp32 inputs stay on the
// fp32 SIMT kernels (bf16 operands could not meet a 1e-4 error bound).
bool uses_tc_kernelized(la_dtype dt, la_mode m) { return dt == LA_BF16 && (m == LA_PLAIN || m == LA_DECAY); }

namespace {

// Final state for an empty sequence: the start state, or zero.
la_status write_start_state(const PrefillArgs& a)
{
    const size_t chains = (size_t)a.B * a.H;
    const size_t sbytes = chains * a.d * a.dv * sizeof(float);
    const size_t zbytes = chains * a.d * sizeof(float);
    cudaError_t e = cudaSuccess;
    if (a.S0) e = cudaMemcpyAsync(a.S_out, a.S0, sbytes, cudaMemcpyDeviceToDevice, a.stream);
    else e = cudaMemsetAsync(a.S_out, 0, sbytes, a.stream);
    if (e == cudaSuccess && a.z_out) {
        if (a.z0) e = cudaMemcpyAsync(a.z_out, a.z0, zbytes, cudaMemcpyDeviceToDevice, a.stream);
        else e = cudaMemsetAsync(a.z_out, 0, zbytes, a.stream);
    }
    return from_cuda(e);
}

// Argument checks of a prefill over a [B,H,N,.] batch (all but the workspace size).
la_status check_prefill(const void* q, const void* k, const void* v, const float* gamma_or_alpha, const float* g,
                        const void* out, const float* S_out, const float* z_out, int B, int H, int N, int d, int dv,
                        const la_config* cfg)
{
    if (!cfg) return LA_ERR_INVALID;
    if (B < 0 || H < 0 || N < 0) return LA_ERR_INVALID;
    if (cfg->dtype != LA_F32 && cfg->dtype != LA_BF16) return LA_ERR_INVALID;
    if (cfg->mode != LA_PLAIN && cfg->mode != LA_DECAY && cfg->mode != LA_GATED_DELTA && cfg->mode != LA_GLA)
        return LA_ERR_INVALID;
    if (!head_ok(d) || !head_ok(dv)) return LA_ERR_UNSUPPORTED;
    const bool delta = cfg->mode == LA_GATED_DELTA;
    const bool gla = cfg->mode == LA_GLA;
    const bool no_norm = delta || gla;   // modes without the z normaliser
    const bool work = (long long)B * H > 0;
    if (work) {
        if (!S_out) return LA_ERR_INVALID;
        if (!no_norm && !z_out) return LA_ERR_INVALID;
        if (no_norm && z_out) return LA_ERR_INVALID;
        if (N > 0 && (!q || !k || !v || !out)) return LA_ERR_INVALID;
        if (cfg->mode == LA_PLAIN && (gamma_or_alpha || g)) return LA_ERR_INVALID;
        if (cfg->mode == LA_DECAY && (!gamma_or_alpha || g)) return LA_ERR_INVALID;
        if (delta && N > 0 && (!gamma_or_alpha || !g)) return LA_ERR_INVALID;
        if (gla && (g || (N > 0 && !gamma_or_alpha))) return LA_ERR_INVALID;
    }
    if (!(cfg->eps >= 0.f)) return LA_ERR_INVALID;
    if (work && state_outputs_alias(S_out, z_out, cfg->S0, no_norm ? nullptr : cfg->z0, B, H, d, dv))
        return LA_ERR_INVALID;
    const void* ptrs[] = {q, k, v, gamma_or_alpha, g, out, S_out, z_out, cfg->S0, cfg->z0, cfg->workspace};
    for (const void* p : ptrs)
        if (!aligned16(p)) return LA_ERR_ALIGN;
    return LA_OK;
}

PrefillArgs prefill_args(const void* q, const void* k, const void* v, const float* gamma_or_alpha, const float* g,
                         void* out, float* S_out, float* z_out, int B, int H, int N, int d, int dv,
                         const la_config* cfg)
{
    const bool delta = cfg->mode == LA_GATED_DELTA;
    const bool no_norm = delta || cfg->mode == LA_GLA;
    PrefillArgs a{};
    a.q = q; a.k = k; a.v = v;
    a.gamma = cfg->mode == LA_DECAY ? gamma_or_alpha : nullptr;
    a.alpha = no_norm ? gamma_or_alpha : nullptr;
    a.g = delta ? g : nullptr;
    a.out = out; a.S_out = S_out; a.z_out = no_norm ? nullptr : z_out;
    a.S0 = cfg->S0; a.z0 = no_norm ? nullptr : cfg->z0;
    a.B = B; a.H = H; a.N = N; a.d = d; a.dv = dv;
    a.ld = N;
    a.eps = cfg->eps; a.dtype = cfg->dtype; a.mode = cfg->mode;
    a.stream = static_cast<cudaStream_t>(cfg->stream);
    a.workspace = cfg->workspace; a.workspace_bytes = cfg->workspace_bytes;
    return a;
}

// A right-padded batch runs as one launch set (instead of one per sequence)
// on the bf16 tensor-core path of the kernelized modes, up to kMaxVarlenSeqs
// sequences.
bool varlen_one_launch_set(const int* lens, int B, int H, int d, int dv, const la_config* cfg)
{
    if (!cfg || !lens || B <= 0 || B > kMaxVarlenSeqs || H <= 0 || !head_ok(d) || !head_ok(dv)) return false;
    for (int b = 0; b < B; ++b)
        if (lens[b] < 0) return false;
    return uses_tc_kernelized(cfg->dtype, cfg->mode);
}

// Workspace slice of one sequence of la_prefill_varlen: 256-byte aligned.
size_t varlen_slice(size_t bytes) { return (bytes + 255) / 256 * 256; }

// One checked prefill to the kernels of its dtype and mode.
la_status run_prefill(const PrefillArgs& a)
{
    if (a.N == 0) return write_start_state(a);
    if (a.mode == LA_GLA) {
        if (a.dtype == LA_BF16) return from_cuda(launch_prefill_tc_gla(a, tc_segments(a.B, a.H, a.N, a.d, a.dv)));
        return from_cuda(launch_prefill_simt_gla(a));
    }
    if (a.mode == LA_GATED_DELTA) {
        if (a.dtype == LA_BF16) return from_cuda(launch_prefill_tc_gated_delta(a));
        return from_cuda(launch_prefill_simt_gated_delta(a));
    }
    if (uses_tc_kernelized(a.dtype, a.mode)) return from_cuda(launch_prefill_tc_kernelized(a));
    return from_cuda(launch_prefill_simt_kernelized(a));
}

// ---- state-space layer ---------------------------------------------------------

bool aligned_to(const void* p, size_t e) { return (reinterpret_cast<uintptr_t>(p) % e) == 0; }

// Lengths of a right-padded batch lie inside it.
bool lens_ok(const int* lens, int B, int N)
{
    for (int b = 0; lens && b < B; ++b)
        if (lens[b] < 0 || lens[b] > N) return false;
    return true;
}

// Tokens of a state-space call's sequences: token numbers add up inside 32 bits.
constexpr int kMostRows = 1 << 30;

// Sequences of one launch: all of them, or kMaxSeqLens where lengths travel with the launch.
int launch_group(const int* lens) { return lens ? kMaxSeqLens : 32768; }

// Checks shared by la_ssm_scan and la_ssm_step; `tokens` counts the rows of x.
la_status check_ssm(const void* x, const void* delta, const float* A, const void* Bm, const void* Cm,
                    const float* D_skip, const void* z, const float* delta_bias, const void* out, const float* h,
                    long long tokens, int B, int D, int G, int n, const la_ssm_strides* st, const la_config* cfg)
{
    if (!cfg || B < 0 || D < 0 || G < 0 || n < 1) return LA_ERR_INVALID;
    if (cfg->dtype != LA_F32 && cfg->dtype != LA_BF16) return LA_ERR_INVALID;
    if (n > 64) return LA_ERR_UNSUPPORTED;
    if (D > 0 && (G == 0 || D % G != 0)) return LA_ERR_INVALID;
    if ((long long)B * D > 0 && tokens > 0 && (!x || !delta || !A || !Bm || !Cm || !out)) return LA_ERR_INVALID;
    if (st) {
        const long long v[] = {st->x_batch, st->x_row, st->delta_batch, st->delta_row, st->z_batch,
                               st->z_row,   st->B_batch, st->B_row,     st->C_batch,     st->C_row};
        for (long long k : v)
            if (k < 0) return LA_ERR_INVALID;
    }
    const size_t e = cfg->dtype == LA_BF16 ? 2 : 4;
    const void* rows[] = {x, delta, Bm, Cm, z, out};
    for (const void* p : rows)
        if (!aligned_to(p, e)) return LA_ERR_ALIGN;
    const void* whole[] = {A, D_skip, delta_bias, h, cfg->S0, cfg->workspace};
    for (const void* p : whole)
        if (!aligned16(p)) return LA_ERR_ALIGN;
    return LA_OK;
}

SsmArgs ssm_args(const void* x, const void* delta, const float* A, const void* Bm, const void* Cm, const float* D_skip,
                 const void* z, const float* delta_bias, void* out, float* h, int B, int N, int D, int G, int n,
                 int softplus, const la_ssm_strides* st, const la_config* cfg)
{
    SsmArgs a{};
    a.x = x; a.delta = delta; a.A = A; a.Bm = Bm; a.Cm = Cm; a.skip = D_skip; a.z = z; a.delta_bias = delta_bias;
    a.out = out; a.h_out = h;
    a.B = B; a.N = N; a.D = D; a.G = G; a.n = n;
    a.softplus = softplus;
    const long long bc = (long long)G * n;
    if (st) a.st = *st;
    else a.st = {(long long)N * D, D, (long long)N * D, D, (long long)N * D, D, N * bc, bc, N * bc, bc};
    a.dtype = cfg->dtype;
    a.stream = static_cast<cudaStream_t>(cfg->stream);
    return a;
}

// Blocks read the inputs while others write out, the states (h) and the summaries of the workspace: none of
// these shares a byte with another argument.  But out may be x, delta or z: a block reads the rows of its
// channels before it writes them, and no other block reads them.
bool ssm_shares(const SsmArgs& a, const float* h0, const void* workspace, size_t workspace_bytes)
{
    const size_t e = a.dtype == LA_BF16 ? 2 : 4, states = (size_t)a.B * a.D * a.n * sizeof(float);
    const size_t channels = (size_t)a.D * sizeof(float);
    auto rows = [&](const void* p, long long cols, long long batch, long long row) {
        return region(p, e, cols, {a.B, a.N, 1}, {batch, row, 0});
    };
    auto out_is = [&](const void* p, long long batch, long long row) {
        return p == a.out && (a.B == 1 || batch == (long long)a.N * a.D) && (a.N == 1 || row == a.D);
    };
    const long long bc = (long long)a.G * a.n;
    const la_ssm_strides& st = a.st;
    const Region in[] = {rows(a.x, a.D, st.x_batch, st.x_row), rows(a.delta, a.D, st.delta_batch, st.delta_row),
                         rows(a.z, a.D, st.z_batch, st.z_row), rows(a.Bm, bc, st.B_batch, st.B_row),
                         rows(a.Cm, bc, st.C_batch, st.C_row), dense(a.A, channels * a.n), dense(a.skip, channels),
                         dense(a.delta_bias, channels), dense(h0, states)};
    const bool in_place[] = {out_is(a.x, st.x_batch, st.x_row), out_is(a.delta, st.delta_batch, st.delta_row),
                             out_is(a.z, st.z_batch, st.z_row)};
    const Region out = rows(a.out, a.D, (long long)a.N * a.D, a.D), h = dense(a.h_out, states),
                 ws = dense(workspace, workspace_bytes);
    for (int i = 0; i < 9; ++i)
        if ((!(i < 3 && in_place[i]) && shared(out, in[i])) || shared(h, in[i]) || shared(ws, in[i])) return true;
    return shared(out, h) || shared(out, ws) || shared(h, ws);
}

// The sequences from b0 on of a batch's arguments.
SsmArgs ssm_from(SsmArgs a, int b0, int count)
{
    const size_t e = a.dtype == LA_BF16 ? 2 : 4;
    auto move = [&](const void* p, long long stride) {
        return p ? static_cast<const char*>(p) + (size_t)b0 * stride * e : nullptr;
    };
    a.x = move(a.x, a.st.x_batch);
    a.delta = move(a.delta, a.st.delta_batch);
    a.z = move(a.z, a.st.z_batch);
    a.Bm = move(a.Bm, a.st.B_batch);
    a.Cm = move(a.Cm, a.st.C_batch);
    a.out = const_cast<char*>(move(a.out, (long long)a.N * a.D));
    const size_t states = (size_t)b0 * a.D * a.n;
    if (a.h0) a.h0 += states;
    if (a.h_out) a.h_out += states;
    if (a.seq_lens) a.seq_lens += b0;
    a.B = count;
    return a;
}

// ---- sliding-window attention --------------------------------------------------

// Checks shared by la_window_prefill and la_window_decode_step (N = 1); fills the arguments.
la_status check_window(WindowArgs* w, const void* q, const void* k, const void* v, void* out, void* k_cache,
                       void* v_cache, const int* pos, int B, int Hq, int Hkv, int N, int d, int dv, int window,
                       int sinks, float scale, const la_window_strides* st, const la_config* cfg)
{
    if (!cfg || B < 0 || Hq < 0 || Hkv < 0 || N < 0 || window < 1 || sinks < 0) return LA_ERR_INVALID;
    if (cfg->dtype != LA_F32 && cfg->dtype != LA_BF16) return LA_ERR_INVALID;
    if (!head_ok(d) || !head_ok(dv)) return LA_ERR_UNSUPPORTED;
    constexpr int kTop = (1 << 30) - 1;   // row and slot numbers add up inside 32 bits
    constexpr int kMostTokens = 65535 * 256;   // query tiles of one launch
    if (N > kMostTokens || (k_cache && (long long)window + sinks > kTop)) return LA_ERR_UNSUPPORTED;
    if (window > kTop) window = kTop;     // without a cache: more than any prompt reaches back
    if (sinks > kTop) sinks = kTop;
    if (Hq > 0 && (Hkv == 0 || Hq % Hkv != 0)) return LA_ERR_INVALID;
    if (Hq > 65535) return LA_ERR_UNSUPPORTED;
    if (!(scale == scale) || scale - scale != 0.f) return LA_ERR_INVALID;   // NaN or infinite
    if ((k_cache == nullptr) != (v_cache == nullptr)) return LA_ERR_INVALID;
    const long long work = (long long)B * Hq * N;
    if (work > 0 && (!q || !k || !v || !out)) return LA_ERR_INVALID;
    la_window_strides s{(long long)Hq * N * d,  (long long)N * d,  d,  (long long)Hkv * N * d, (long long)N * d,  d,
                        (long long)Hkv * N * dv, (long long)N * dv, dv, (long long)Hq * N * dv, (long long)N * dv, dv};
    if (st) s = *st;
    const size_t e = cfg->dtype == LA_BF16 ? 2 : 4;
    const long long strides[] = {s.q_batch, s.q_head, s.q_row, s.k_batch, s.k_head, s.k_row,
                                 s.v_batch, s.v_head, s.v_row, s.out_batch, s.out_head, s.out_row};
    for (long long x : strides) {
        if (x < 0) return LA_ERR_INVALID;
        if (x * (long long)e % 16 != 0) return LA_ERR_ALIGN;
    }
    const void* ptrs[] = {q, k, v, out, k_cache, v_cache};
    for (const void* p : ptrs)
        if (!aligned16(p)) return LA_ERR_ALIGN;
    if (!aligned_to(pos, sizeof(int))) return LA_ERR_ALIGN;
    // rows of one head do not share memory
    if (N > 1 && (s.q_row < d || s.k_row < d || s.v_row < dv || s.out_row < dv)) return LA_ERR_INVALID;
    // nor do two heads or sequences of out
    if (work > 0 && ((Hq > 1 && s.out_head == 0) || (B > 1 && s.out_batch == 0))) return LA_ERR_INVALID;
    if (work > 0) {
        const Region rq = region(q, e, d, {B, Hq, N}, {s.q_batch, s.q_head, s.q_row});
        const Region rk = region(k, e, d, {B, Hkv, N}, {s.k_batch, s.k_head, s.k_row});
        const Region rv = region(v, e, dv, {B, Hkv, N}, {s.v_batch, s.v_head, s.v_row});
        const Region ro = region(out, e, dv, {B, Hq, N}, {s.out_batch, s.out_head, s.out_row});
        const size_t slots = (size_t)B * Hkv * ((size_t)window + sinks);
        const Region rkc = dense(k_cache, slots * d * e), rvc = dense(v_cache, slots * dv * e);
        const Region rp = dense(pos, (size_t)B * sizeof(int));
        if (overlaps_itself(ro)) return LA_ERR_INVALID;
        // blocks read k and v, positions and caches while others write; q's rows are read by the block
        // that writes the same rows of out alone, so out may take q's place, but not a shifted one
        auto alike = [](int count, long long x, long long y) { return count == 1 || x == y; };
        const bool in_place = out == q && dv == d && alike(B, s.q_batch, s.out_batch) && alike(Hq, s.q_head, s.out_head) &&
                              alike(N, s.q_row, s.out_row);
        if (!in_place && shared(ro, rq)) return LA_ERR_INVALID;
        const Region* written[] = {&ro, &rkc, &rvc};
        for (int i = 0; i < 3; ++i) {
            for (const Region* r : {&rk, &rv, &rp})
                if (shared(*written[i], *r)) return LA_ERR_INVALID;
            if (i > 0 && (shared(*written[i], rq) || shared(*written[i], ro))) return LA_ERR_INVALID;
        }
        if (shared(rkc, rvc)) return LA_ERR_INVALID;
    }
    *w = WindowArgs{};
    w->q = q; w->k = k; w->v = v; w->out = out; w->k_cache = k_cache; w->v_cache = v_cache; w->pos = pos;
    w->B = B; w->Hq = Hq; w->Hkv = Hkv; w->N = N; w->d = d; w->dv = dv;
    w->window = window; w->sinks = sinks; w->scale = scale;
    w->st = s;
    w->dtype = cfg->dtype;
    w->stream = static_cast<cudaStream_t>(cfg->stream);
    return LA_OK;
}

// The sequences from b0 on.
WindowArgs window_from(WindowArgs a, int b0, int count)
{
    const size_t e = a.dtype == LA_BF16 ? 2 : 4;
    auto move = [&](const void* p, long long stride) {
        return p ? const_cast<char*>(static_cast<const char*>(p)) + (size_t)b0 * stride * e : nullptr;
    };
    const long long cap = (long long)a.window + a.sinks;
    a.q = move(a.q, a.st.q_batch);
    a.k = move(a.k, a.st.k_batch);
    a.v = move(a.v, a.st.v_batch);
    a.out = move(a.out, a.st.out_batch);
    a.k_cache = move(a.k_cache, a.Hkv * cap * a.d);
    a.v_cache = move(a.v_cache, a.Hkv * cap * a.dv);
    if (a.pos) a.pos += b0;
    if (a.seq_lens) a.seq_lens += b0;
    a.B = count;
    return a;
}

}  // namespace
}  // namespace la

using la::PrefillArgs;
using la::DecodeArgs;

extern "C" {

const char* la_version(void) { return "0.1.0"; }

const char* la_status_string(la_status s)
{
    switch (s) {
        case LA_OK: return "LA_OK";
        case LA_ERR_INVALID: return "LA_ERR_INVALID: invalid argument";
        case LA_ERR_UNSUPPORTED: return "LA_ERR_UNSUPPORTED: head size or dtype/mode not supported";
        case LA_ERR_ALIGN: return "LA_ERR_ALIGN: pointer not 16-byte aligned";
        case LA_ERR_CUDA: return "LA_ERR_CUDA: CUDA call or kernel launch failed";
        case LA_ERR_TIMEOUT: return "LA_ERR_TIMEOUT: a bounded device-side wait gave up";
        case LA_ERR_WORKSPACE: return "LA_ERR_WORKSPACE: workspace missing or too small";
    }
    return "unknown la_status";
}

size_t la_prefill_workspace_bytes(int B, int H, int N, int d, int dv, const la_config* cfg)
{
    if (!cfg || B <= 0 || H <= 0 || N <= 0 || !la::head_ok(d) || !la::head_ok(dv)) return 0;
    if (la::uses_tc_kernelized(cfg->dtype, cfg->mode)) return la::tc_workspace_bytes(B, H, N, d, dv);
    if (cfg->dtype == LA_BF16 && cfg->mode == LA_GLA) return la::tc_workspace_bytes(B, H, N, d, dv);
    if (cfg->dtype == LA_BF16 && cfg->mode == LA_GATED_DELTA) return la::gd_workspace_bytes(B, H, N, d, dv);
    return 0;
}

int la_prefill_kernel_count(int B, int H, int N, int d, int dv, const la_config* cfg)
{
    if (!cfg || B <= 0 || H <= 0 || N <= 0 || !la::head_ok(d) || !la::head_ok(dv)) return 0;
    if (la::uses_tc_kernelized(cfg->dtype, cfg->mode)) return 3;
    if (cfg->dtype == LA_BF16 && cfg->mode == LA_GLA) return 3;
    if (cfg->dtype == LA_BF16 && cfg->mode == LA_GATED_DELTA) return 2 * la::gd_parts(B, H, N, d, dv).P;
    if (cfg->mode == LA_PLAIN || cfg->mode == LA_DECAY) return la::simt_kernelized_kernel_count(N, cfg->dtype);
    return 1;
}

la_status la_prefill(const void* q, const void* k, const void* v,
                     const float* gamma_or_alpha, const float* g,
                     void* out, float* S_out, float* z_out,
                     int B, int H, int N, int d, int dv, const la_config* cfg)
{
    const la_status st = la::check_prefill(q, k, v, gamma_or_alpha, g, out, S_out, z_out, B, H, N, d, dv, cfg);
    if (st != LA_OK) return st;
    if (cfg->workspace_bytes < la_prefill_workspace_bytes(B, H, N, d, dv, cfg)) return LA_ERR_WORKSPACE;
    if ((long long)B * H == 0) return LA_OK;
    return la::run_prefill(la::prefill_args(q, k, v, gamma_or_alpha, g, out, S_out, z_out, B, H, N, d, dv, cfg));
}

size_t la_prefill_varlen_workspace_bytes(const int* seq_lens, int B, int H, int d, int dv, const la_config* cfg)
{
    if (!seq_lens || B <= 0) return 0;
    if (la::varlen_one_launch_set(seq_lens, B, H, d, dv, cfg))
        return la::tc_varlen_workspace_bytes(seq_lens, B, H, d, dv);
    size_t total = 0;
    for (int b = 0; b < B; ++b) total += la::varlen_slice(la_prefill_workspace_bytes(1, H, seq_lens[b], d, dv, cfg));
    return total;
}

la_status la_prefill_varlen(const void* q, const void* k, const void* v,
                            const float* gamma_or_alpha, const float* g,
                            void* out, float* S_out, float* z_out, const int* seq_lens,
                            int B, int H, int N, int d, int dv, const la_config* cfg)
{
    const la_status st = la::check_prefill(q, k, v, gamma_or_alpha, g, out, S_out, z_out, B, H, N, d, dv, cfg);
    if (st != LA_OK) return st;
    if ((long long)B * H == 0) return LA_OK;
    if (!seq_lens) return LA_ERR_INVALID;
    for (int b = 0; b < B; ++b)
        if (seq_lens[b] < 0 || seq_lens[b] > N) return LA_ERR_INVALID;
    if (cfg->workspace_bytes < la_prefill_varlen_workspace_bytes(seq_lens, B, H, d, dv, cfg))
        return LA_ERR_WORKSPACE;

    // Sequence b is the B = 1 batch of its H chains over its own length; its
    // chains keep the batch's row stride N, so the padding rows are neither
    // read (the TMA maps and the SIMT loops end at the length) nor written.
    // Each sequence has a slice of the workspace of its own, so the first
    // kernel of sequence b > 0 may start while sequence b-1's kernels drain
    // (programmatic serialization); it finishes after them.
    const PrefillArgs base = la::prefill_args(q, k, v, gamma_or_alpha, g, out, S_out, z_out, B, H, N, d, dv, cfg);
    if (la::varlen_one_launch_set(seq_lens, B, H, d, dv, cfg)) {
        // one launch set over every sequence of the batch
        bool any = false;
        for (int b = 0; b < B; ++b) any = any || seq_lens[b] > 0;
        if (!any) return la::write_start_state(base);
        return la::from_cuda(la::launch_prefill_tc_kernelized_varlen(base, seq_lens));
    }
    const size_t esz = cfg->dtype == LA_BF16 ? 2 : 4;
    size_t ws_off = 0;
    for (int b = 0; b < B; ++b) {
        PrefillArgs a = base;
        const size_t ws_b = la_prefill_workspace_bytes(1, H, seq_lens[b], d, dv, cfg);
        a.workspace = ws_b ? static_cast<char*>(cfg->workspace) + ws_off : nullptr;
        a.workspace_bytes = ws_b;
        ws_off += la::varlen_slice(ws_b);
        a.pdl_first = b > 0 && seq_lens[b - 1] > 0;   // behind a kernel of sequence b-1
        const size_t row0 = (size_t)b * H * N;   // first row of sequence b
        const size_t st_s = (size_t)b * H * d * dv, st_z = (size_t)b * H * d;
        a.q = static_cast<const char*>(q) + row0 * d * esz;
        a.k = static_cast<const char*>(k) + row0 * d * esz;
        a.v = static_cast<const char*>(v) + row0 * dv * esz;
        a.out = static_cast<char*>(out) + row0 * dv * esz;
        if (a.alpha) a.alpha += cfg->mode == LA_GLA ? row0 * d : row0;
        if (a.g) a.g += row0;
        a.S_out += st_s;
        if (a.z_out) a.z_out += st_z;
        if (a.S0) a.S0 += st_s;
        if (a.z0) a.z0 += st_z;
        a.B = 1;
        a.N = seq_lens[b];
        a.ld = N;
        const la_status r = la::run_prefill(a);
        if (r != LA_OK) return r;
    }
    return LA_OK;
}

la_status la_prefill_noalloc(const void* q, const void* k, const void* v,
                             const float* gamma_or_alpha, const float* g,
                             void* out, float* S_out, float* z_out,
                             int B, int H, int N, int d, int dv, const la_config* cfg)
{
    if (!cfg) return LA_ERR_INVALID;
    la_config c = *cfg;   // cfg->workspace is ignored
    c.workspace = nullptr;
    c.workspace_bytes = 0;
    const la_status st = la::check_prefill(q, k, v, gamma_or_alpha, g, out, S_out, z_out, B, H, N, d, dv, &c);
    if (st != LA_OK) return st;
    if ((long long)B * H == 0) return LA_OK;
    PrefillArgs a = la::prefill_args(q, k, v, gamma_or_alpha, g, out, S_out, z_out, B, H, N, d, dv, &c);
    if (c.dtype == LA_BF16 && c.mode == LA_GLA) {
        // the GLA segment summaries have the kernelized modes' slot size
        if (N == 0) return la::write_start_state(a);
        const la::TcSegments sg = la::tc_segments_noalloc(B, H, N, d, dv);
        if (sg.G == 0) return LA_ERR_WORKSPACE;
        cudaError_t e;
        a.workspace = la::noalloc_scratch_address(&e);
        if (!a.workspace) return la::from_cuda(e);
        a.workspace_bytes = la::kNoAllocScratchBytes;
        return la::from_cuda(la::launch_prefill_tc_gla(a, sg));
    }
    if (!la::uses_tc_kernelized(c.dtype, c.mode)) {
        // paths that need no workspace run as la_prefill does; the bf16
        // gated delta rule's per-chunk operands grow with N and have no
        // fixed-size form
        if (la_prefill_workspace_bytes(B, H, N, d, dv, &c) != 0) return LA_ERR_UNSUPPORTED;
        return la::run_prefill(a);
    }
    if (N == 0) return la::write_start_state(a);
    if (la::tc_segments_noalloc(B, H, N, d, dv).G == 0) return LA_ERR_WORKSPACE;
    return la::from_cuda(la::launch_prefill_tc_kernelized_noalloc(a));
}

static la_status decode_common_checks(const void* q, const void* k, const void* v, float* S, void* out,
                                      int B, int H, int d, int dv, const la_config* cfg)
{
    if (!cfg) return LA_ERR_INVALID;
    if (B < 0 || H < 0) return LA_ERR_INVALID;
    if (cfg->dtype != LA_F32 && cfg->dtype != LA_BF16) return LA_ERR_INVALID;
    if (!la::head_ok(d) || !la::head_ok(dv)) return LA_ERR_UNSUPPORTED;
    if ((long long)B * H > 0 && (!q || !k || !v || !S || !out)) return LA_ERR_INVALID;
    if ((long long)B * H > 0x7fffffffLL) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

la_status la_decode_step(const void* q, const void* k, const void* v,
                         float* S, float* z, void* out,
                         int B, int H, int d, int dv, const la_config* cfg)
{
    la_status st = decode_common_checks(q, k, v, S, out, B, H, d, dv, cfg);
    if (st != LA_OK) return st;
    if (cfg->mode != LA_PLAIN) return LA_ERR_INVALID;
    if ((long long)B * H > 0 && !z) return LA_ERR_INVALID;
    if (!(cfg->eps >= 0.f)) return LA_ERR_INVALID;
    const void* ptrs[] = {q, k, v, S, z, out};
    for (const void* p : ptrs)
        if (!la::aligned16(p)) return LA_ERR_ALIGN;
    if ((long long)B * H == 0) return LA_OK;
    DecodeArgs a{};
    a.q = q; a.k = k; a.v = v; a.S = S; a.z = z; a.out = out;
    a.B = B; a.H = H; a.d = d; a.dv = dv; a.eps = cfg->eps; a.dtype = cfg->dtype;
    a.stream = static_cast<cudaStream_t>(cfg->stream);
    return la::from_cuda(la::launch_decode_kernelized(a));
}

la_status la_gated_delta_decode_step(const void* q, const void* k, const void* v,
                                     const float* alpha, const float* g,
                                     float* S, void* out,
                                     int B, int H, int d, int dv, const la_config* cfg)
{
    la_status st = decode_common_checks(q, k, v, S, out, B, H, d, dv, cfg);
    if (st != LA_OK) return st;
    if (cfg->mode != LA_GATED_DELTA) return LA_ERR_INVALID;
    if ((long long)B * H > 0 && (!alpha || !g)) return LA_ERR_INVALID;
    const void* ptrs[] = {q, k, v, alpha, g, S, out};
    for (const void* p : ptrs)
        if (!la::aligned16(p)) return LA_ERR_ALIGN;
    if ((long long)B * H == 0) return LA_OK;
    DecodeArgs a{};
    a.q = q; a.k = k; a.v = v; a.alpha = alpha; a.g = g; a.S = S; a.out = out;
    a.B = B; a.H = H; a.d = d; a.dv = dv; a.dtype = cfg->dtype;
    a.stream = static_cast<cudaStream_t>(cfg->stream);
    return la::from_cuda(la::launch_decode_gated_delta(a));
}

la_status la_causal_conv(const void* x, const float* weight, const void* cache, void* out, void* cache_out,
                         int B, int H, int N, int d, int w, const la_config* cfg)
{
    if (!cfg) return LA_ERR_INVALID;
    if (B < 0 || H < 0 || N < 0 || w < 1) return LA_ERR_INVALID;
    if (cfg->dtype != LA_F32 && cfg->dtype != LA_BF16) return LA_ERR_INVALID;
    if (!la::head_ok(d) || w > 8) return LA_ERR_UNSUPPORTED;
    const long long chains = (long long)B * H;
    if (chains == 0) return LA_OK;
    if (N > 0 && (!x || !weight || !out)) return LA_ERR_INVALID;
    const size_t es = cfg->dtype == LA_BF16 ? 2 : 4;
    const size_t cache_bytes = (size_t)chains * (w - 1) * d * es;
    if (la::overlap(cache_out, cache_bytes, cache, cache_bytes) ||
        la::overlap(cache_out, cache_bytes, x, (size_t)chains * N * d * es))
        return LA_ERR_INVALID;
    const void* ptrs[] = {x, weight, cache, out, cache_out};
    for (const void* p : ptrs)
        if (!la::aligned16(p)) return LA_ERR_ALIGN;
    if (N == 0 && !cache_out) return LA_OK;
    la::ConvArgs a{};
    a.x = x; a.weight = weight; a.cache = cache; a.y = out; a.cache_out = w > 1 ? cache_out : nullptr;
    a.B = B; a.H = H; a.N = N; a.d = d; a.w = w;
    a.dtype = cfg->dtype;
    a.stream = static_cast<cudaStream_t>(cfg->stream);
    if (a.N == 0 && !a.cache_out) return LA_OK;
    return la::from_cuda(la::launch_causal_conv(a));
}

la_status la_ssm_conv(const void* x, const float* weight, const float* bias, const void* cache, void* out,
                      void* cache_out, const int* seq_lens, int B, int N, int D, int w, int silu, long long x_batch,
                      long long x_row, const la_config* cfg)
{
    if (!cfg) return LA_ERR_INVALID;
    if (B < 0 || N < 0 || D < 0 || w < 1 || x_batch < 0 || x_row < 0) return LA_ERR_INVALID;
    if (cfg->dtype != LA_F32 && cfg->dtype != LA_BF16) return LA_ERR_INVALID;
    if (w > 8 || N > la::kMostRows) return LA_ERR_UNSUPPORTED;
    if (!la::lens_ok(seq_lens, B, N)) return LA_ERR_INVALID;
    if (B == 0 || D == 0) return LA_OK;
    if (N > 0 && (!x || !weight || !out)) return LA_ERR_INVALID;
    const size_t e = cfg->dtype == LA_BF16 ? 2 : 4;
    const void* rows[] = {x, cache, out, cache_out};
    for (const void* p : rows)
        if (!la::aligned_to(p, e)) return LA_ERR_ALIGN;
    if (!la::aligned16(weight) || !la::aligned16(bias)) return LA_ERR_ALIGN;
    // a run of tokens reads the rows before it, so out in place of x would change them; the caches may be one,
    // since a thread reads all it needs of them before it writes
    const size_t cache_bytes = (size_t)B * (w - 1) * D * e;
    const la::Region rx = la::region(x, e, D, {B, N, 1}, {x_batch, x_row, 0}), rw = la::dense(weight, (size_t)D * w * 4),
                     rb = la::dense(bias, (size_t)D * 4), rc = la::dense(cache, cache_bytes),
                     ro = la::dense(out, (size_t)B * N * D * e), rn = la::dense(cache_out, cache_bytes);
    for (const la::Region* r : {&rx, &rw, &rb})
        if (la::shared(ro, *r) || la::shared(rn, *r)) return LA_ERR_INVALID;
    if (la::shared(ro, rc) || la::shared(ro, rn) || (cache_out != cache && la::shared(rc, rn))) return LA_ERR_INVALID;
    if (w == 1) cache = cache_out = nullptr;
    if (N == 0 && !cache_out) return LA_OK;
    const int step = la::launch_group(seq_lens);
    for (int b0 = 0; b0 < B; b0 += step) {
        la::SsmConvArgs a{};
        const size_t rows0 = (size_t)b0 * D * e;
        auto move = [&](const void* p, size_t by) { return p ? static_cast<const char*>(p) + by : nullptr; };
        a.x = move(x, (size_t)b0 * x_batch * e);
        a.weight = weight;
        a.bias = bias;
        a.cache = move(cache, rows0 * (w - 1));
        a.out = const_cast<char*>(move(out, rows0 * N));
        a.cache_out = const_cast<char*>(move(cache_out, rows0 * (w - 1)));
        a.seq_lens = seq_lens ? seq_lens + b0 : nullptr;
        a.B = B - b0 < step ? B - b0 : step;
        a.N = N; a.D = D; a.w = w;
        a.silu = silu;
        a.x_batch = x_batch; a.x_row = x_row;
        a.dtype = cfg->dtype;
        a.stream = static_cast<cudaStream_t>(cfg->stream);
        const cudaError_t err = la::launch_ssm_conv(a);
        if (err != cudaSuccess) return LA_ERR_CUDA;
        la::stage_mark(0, a.stream);
    }
    return LA_OK;
}

size_t la_ssm_scan_workspace_bytes(int B, int N, int D, int G, int n)
{
    if (B <= 0 || N <= 0 || D <= 0 || G <= 0 || D % G != 0 || n < 1 || n > 64) return 0;
    return la::ssm_scan_workspace_bytes(B, N, D, G, n);
}

la_status la_ssm_scan(const void* x, const void* delta, const float* A, const void* Bm, const void* Cm,
                      const float* D_skip, const void* z, const float* delta_bias, void* out, float* h_out,
                      const int* seq_lens, int B, int N, int D, int G, int n, int delta_softplus,
                      const la_ssm_strides* strides, const la_config* cfg)
{
    if (N < 0) return LA_ERR_INVALID;
    const la_status st =
        la::check_ssm(x, delta, A, Bm, Cm, D_skip, z, delta_bias, out, h_out, N, B, D, G, n, strides, cfg);
    if (st != LA_OK) return st;
    if (N > la::kMostRows) return LA_ERR_UNSUPPORTED;
    if (!la::lens_ok(seq_lens, B, N)) return LA_ERR_INVALID;
    const size_t states = (size_t)B * D * n * sizeof(float);
    if (la::overlap(h_out, states, cfg->S0, states)) return LA_ERR_INVALID;
    const size_t need = la_ssm_scan_workspace_bytes(B, N, D, G, n);
    if (cfg->workspace_bytes < need || (need > 0 && !cfg->workspace)) return LA_ERR_WORKSPACE;
    if (B == 0 || D == 0) return LA_OK;
    la::SsmArgs all = la::ssm_args(x, delta, A, Bm, Cm, D_skip, z, delta_bias, out, h_out, B, N, D, G, n,
                                   delta_softplus, strides, cfg);
    if (la::ssm_shares(all, cfg->S0, cfg->workspace, need)) return LA_ERR_INVALID;
    cudaStream_t stream = static_cast<cudaStream_t>(cfg->stream);
    if (N == 0) {
        if (!h_out) return LA_OK;
        return la::from_cuda(cfg->S0 ? cudaMemcpyAsync(h_out, cfg->S0, states, cudaMemcpyDeviceToDevice, stream)
                                     : cudaMemsetAsync(h_out, 0, states, stream));
    }
    all.h0 = cfg->S0;
    all.seq_lens = seq_lens;
    la::ssm_scan_segments(B, N, D, G, n, &all.segs, &all.seg_len);
    const size_t per = need / B / sizeof(float);
    const int step = la::launch_group(seq_lens);
    for (int b0 = 0; b0 < B; b0 += step) {
        la::SsmArgs a = la::ssm_from(all, b0, B - b0 < step ? B - b0 : step);
        if (per) a.workspace = static_cast<float*>(cfg->workspace) + (size_t)b0 * per;
        const cudaError_t err = la::launch_ssm_scan(a);
        if (err != cudaSuccess) return LA_ERR_CUDA;
    }
    return LA_OK;
}

la_status la_ssm_step(const void* x, const void* delta, const float* A, const void* Bm, const void* Cm,
                      const float* D_skip, const void* z, const float* delta_bias, float* h, void* out, int B, int D,
                      int G, int n, int delta_softplus, const la_ssm_strides* strides, const la_config* cfg)
{
    const la_status st = la::check_ssm(x, delta, A, Bm, Cm, D_skip, z, delta_bias, out, h, 1, B, D, G, n, strides, cfg);
    if (st != LA_OK) return st;
    if (B == 0 || D == 0) return LA_OK;
    if (!h) return LA_ERR_INVALID;
    const la::SsmArgs a =
        la::ssm_args(x, delta, A, Bm, Cm, D_skip, z, delta_bias, out, h, B, 1, D, G, n, delta_softplus, strides, cfg);
    if (la::ssm_shares(a, nullptr, nullptr, 0)) return LA_ERR_INVALID;
    return la::from_cuda(la::launch_ssm_step(a));
}

la_status la_window_prefill(const void* q, const void* k, const void* v, void* out, void* k_cache, void* v_cache,
                            const int* pos, const int* seq_lens, int B, int Hq, int Hkv, int N, int d, int dv,
                            int window, int sinks, float scale, const la_window_strides* strides, const la_config* cfg)
{
    la::WindowArgs all;
    const la_status st = la::check_window(&all, q, k, v, out, k_cache, v_cache, pos, B, Hq, Hkv, N, d, dv, window,
                                          sinks, scale, strides, cfg);
    if (st != LA_OK) return st;
    if (pos && !k_cache) return LA_ERR_INVALID;
    if (!la::lens_ok(seq_lens, B, N)) return LA_ERR_INVALID;
    if ((long long)B * Hq * N == 0) return LA_OK;
    all.seq_lens = seq_lens;
    const int step = la::launch_group(seq_lens);
    for (int b0 = 0; b0 < B; b0 += step) {
        const la::WindowArgs a = la::window_from(all, b0, B - b0 < step ? B - b0 : step);
        // bf16 prompts run on the tensor cores; fp32 inputs keep fp32 arithmetic
        cudaError_t err = a.dtype == LA_BF16 ? la::launch_window_prefill_tc(a) : la::launch_window_prefill_simt(a);
        if (err == cudaSuccess) la::stage_mark(0, a.stream);
        if (err == cudaSuccess && a.k_cache) {
            err = la::launch_window_cache_update(a);
            if (err == cudaSuccess) la::stage_mark(1, a.stream);
        }
        if (err != cudaSuccess) return LA_ERR_CUDA;
    }
    return LA_OK;
}

la_status la_window_decode_step(const void* q, const void* k, const void* v, void* out, void* k_cache, void* v_cache,
                                const int* pos, int B, int Hq, int Hkv, int d, int dv, int window, int sinks,
                                float scale, const la_window_strides* strides, const la_config* cfg)
{
    la::WindowArgs all;
    const la_status st = la::check_window(&all, q, k, v, out, k_cache, v_cache, pos, B, Hq, Hkv, 1, d, dv, window,
                                          sinks, scale, strides, cfg);
    if (st != LA_OK) return st;
    if ((long long)B * Hq == 0) return LA_OK;
    if (!k_cache || !pos) return LA_ERR_INVALID;
    const int step = la::launch_group(nullptr);
    for (int b0 = 0; b0 < B; b0 += step) {
        const la::WindowArgs a = la::window_from(all, b0, B - b0 < step ? B - b0 : step);
        if (la::launch_window_decode(a) != cudaSuccess) return LA_ERR_CUDA;
        la::stage_mark(0, a.stream);
    }
    return LA_OK;
}

la_status la_set_stage_events(void* const* events, int n)
{
    if (n < 0 || n > la::kMaxStageEvents || (n > 0 && !events)) return LA_ERR_INVALID;
    for (int i = 0; i < n; ++i)
        if (!events[i]) return LA_ERR_INVALID;
    for (int i = 0; i < n; ++i) la::g_stage_events[i] = static_cast<cudaEvent_t>(events[i]);
    la::g_stage_count = n;
    return LA_OK;
}

la_status la_selftest_wait_timeout(void* stream)
{
    return la::from_cuda(la::launch_wait_timeout_selftest(static_cast<cudaStream_t>(stream)));
}

la_status la_prefill_check(const void* workspace, void* stream)
{
    (void)workspace;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(s) != cudaSuccess) return LA_ERR_CUDA;
    const unsigned int e1 = la::read_and_clear_device_error(s);
    const unsigned int e2 = la::read_and_clear_device_error_gdelta(s);
    const unsigned int e3 = la::read_and_clear_device_error_selftest(s);
    const unsigned int e4 = la::read_and_clear_device_error_gla(s);
    const unsigned int e5 = la::read_and_clear_device_error_window(s);
    if (e1 == 4u || e2 == 4u || e4 == 4u) return LA_ERR_UNSUPPORTED;
    if (e1 != 0 || e2 != 0 || e3 != 0 || e4 != 0 || e5 != 0) return LA_ERR_TIMEOUT;
    return LA_OK;
}

}  // extern "C"
