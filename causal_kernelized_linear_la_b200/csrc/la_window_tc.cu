// Sliding-window attention with sinks, bf16 prompts on the tensor cores
// (tcgen05 + TMEM + TMA).
//
//     S = Q K^T (fp32, TMEM),  P = 2^(S c - m c),  O += P V,  l += P 1,  o = O / l
// with c = scale log2 e and a reference m per query that only has to stay near
// the running maximum: O and l are rescaled when a tile's maximum exceeds m by
// more than 8 in log2 units, so P <= 2^8 and most tiles rescale nothing.
//
// A CTA takes 256 queries of one head as two tiles of 128 (the M of an MMA)
// and walks the key tiles of 128 that any of them sees: cache slots, the
// prompt's own sinks, the window's band (KeyWalk).  The two tiles alternate on
// the tensor pipe: while one tile's warps turn its scores into weights (one
// thread a query, the row in registers), the pipe runs the other tile's
// products.  Weights go back to TMEM as bf16, over the scores they came from,
// and are the A operand of P V from there, 64 keys at a time.
//   warps 0-3, 4-7  softmax of tile 0, 1; rescale; output
//   warp 8          TMA: Q once, then K and V tiles through a ring
//   warp 9          MMA issue; describes each key tile to the softmax warps
//   warp 10         zeroes the value rows of a tile that hold no token: padding
//                   and unfilled slots may hold NaN, and 0 * NaN is not 0
// A ring stage is refilled after the products that read it and after warp 10
// has seen it full: warp 10 follows every load, and a stage that passed two
// phases under it would look like one that has not been loaded yet.
// The weights are rounded to bf16 (half a step, 2^-8): the tensor cores take
// both operands of a product in one type.  l adds the weights before that
// rounding, in fp32.
//
// Bound: per 128 x 128 tile, 2 products of 128 x 128 x d (at d = 128 16
// instructions of 64 clocks) and 16384 exponentials (1024 clocks of the SFU).  A pair
// of tiles takes about 3700 clocks where the pipe needs 2060: a tile's own chain
// (load of the scores 350, maximum 250, exponentials 1100 and more while the
// other tile uses the SFU too, products 1024, hand-offs) is longer than what the
// other tile hides: the tensor pipe is active 52 % of the time, the SFU 52 %.  A
// 16384-token prompt (32 heads of 128, window 4096) takes 987 to 1008 us on
// different cards, 955 to 976 TFLOP/s at the 1000 W limit; a chunk of 4096 tokens
// behind 65540 cached slots 4.3 ms (1020 TFLOP/s).  Measured and not kept: two
// threads a query (1021 against 1014 us), an issuing warp a tile (1012), a
// quarter of the exponentials as polynomials on the FMA pipe (1033 to 1180).
#include <cudaTypedefs.h>

#include "f32x2.cuh"
#include "la_window.cuh"
#include "sm100.cuh"

namespace la {
namespace {

using namespace sm100;

constexpr int kM = 128;          // queries of a tile
constexpr int kKeys = 128;       // keys of a tile
constexpr int kSoftWarps = 8;
constexpr int kThreads = (kSoftWarps + 3) * 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;    // log2 units a tile's maximum may exceed the reference by

template <int D, int DV>
struct Plan {
    static constexpr int STAGES = 5;
    static constexpr int QB = kM * D * 2;                         // one query tile
    static constexpr int KB = kKeys * D * 2, VB = kKeys * DV * 2;
    static constexpr int STAGE = KB > VB ? KB : VB;
    static constexpr int OFF_RING = 2 * QB;
    static constexpr int OFF_BAR = OFF_RING + STAGES * STAGE;
    // full[S] empty[S] q_full s_full[2] p_full[2][2] o_done[2] clean[3] drain
    static constexpr int NBAR = 2 * STAGES + 13;
    static constexpr int OFF_DESC = OFF_BAR + NBAR * 8;           // [2] int2: the key tile behind each tile's scores
    static constexpr int OFF_TMEM = OFF_DESC + 16;
    static constexpr int BYTES = OFF_TMEM + 16 + 1024;
    static_assert(BYTES <= 232448, "shared memory plan exceeds the per-block limit");
    // TMEM columns: scores (and weights) of both tiles, outputs of both tiles
    static constexpr uint32_t T_S = 0, T_O = 256, T_COLS = 512;
};

// Tensor maps of one call, and which of their head / batch axes are real (an
// axis of stride 0 is mapped as one entry and read at coordinate 0).
struct Maps {
    CUtensorMap q, k, v, kc, vc;
    int qh, qb, kh, kb, vh, vb;
};

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar,
                                            uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem desc], kind::f16: A's row i is lane i, two bf16 of K a column.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t on;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(on));
    return on != 0;
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32])
{
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

enum TileFlags : int { kMasked = 1, kCacheTile = 2, kLastTile = 4 };

// grid: (heads, pairs of query tiles, sequences)
template <int D, int DV>
__global__ void __launch_bounds__(kThreads, 1)
window_prefill_tc(const __grid_constant__ Maps maps, const __grid_constant__ WindowArgs a,
                  const __grid_constant__ WindowLens lens)
{
    using P = Plan<D, DV>;
    // warp number and start come through a shuffle: the compiler then knows them to be the same in
    // every lane, and the issuing warp's descriptors and branches stay in the uniform registers that
    // tcgen05.mma takes them from (moving them there per instruction halved the issue rate)
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
    const int b = blockIdx.z, h = blockIdx.x, kvh = h / (a.Hq / a.Hkv);
    const int len = lens.use ? lens.n[b] : a.N;
    const int start = __shfl_sync(~0u, a.pos ? a.pos[b] : 0, 0);
    // later queries see at least as many keys: the longest walks start first
    const int q0 = ((int)gridDim.y - 1 - (int)blockIdx.y) * 2 * kM;
    if (start < 0 || q0 >= len) return;

    KeyWalk<kKeys> w;
    w.init(a.k_cache != nullptr, start, a.window, a.sinks, len, q0, min(len, q0 + 2 * kM));
    const int tiles = w.count();
    // tile g's queries [qa(g), qb(g)); tile 1 may be empty
    auto qa = [&](int g) { return q0 + g * kM; };
    auto qb = [&](int g) { return min(len, q0 + (g + 1) * kM); };
    // Which band tiles (by their number, first key / kKeys) a query tile sees,
    // and which it sees whole: ranges, so that the walk costs a few compares a
    // tile.  A tile of sinks is seen from anywhere behind it.
    int see0[2], see1[2], whole0[2], whole1[2];
    const int sink_any = (w.sinks_left() + kKeys - 1) / kKeys, sink_all = w.sinks_left() / kKeys;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        see0[g] = max(0, qa(g) - w.window + 1) / kKeys;
        see1[g] = qa(g) < len ? (qb(g) + kKeys - 1) / kKeys : 0;
        whole0[g] = (max(0, qb(g) - w.window) + kKeys - 1) / kKeys;
        whole1[g] = min(qa(g) + 1, len) / kKeys;
    }
    const int band_at = w.cache_tiles + w.sink_tiles;     // the walk's first band tile
    auto active = [&](int it, int g) {
        if (it < band_at) return qa(g) < len && w.any(it, qa(g), qb(g));
        const int n = w.band0 + it - band_at;
        return n < see1[g] && (n >= see0[g] || n < sink_any);
    };
    auto masked = [&](int it, int g) {
        if (it < band_at) return !w.all(it, qa(g), qb(g));
        const int n = w.band0 + it - band_at;
        return !(n < whole1[g] && (n >= whole0[g] || n < sink_all));
    };

    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = align1024(smem_raw);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + P::OFF_BAR);
    uint64_t* empty = full + P::STAGES;
    uint64_t* q_full = empty + P::STAGES;
    uint64_t* s_full = q_full + 1;     // [2] scores in TMEM
    uint64_t* p_full = s_full + 2;     // [2][2] weights of the first, the other 64 keys in TMEM, O rescaled
    uint64_t* o_done = p_full + 4;     // [2] P V complete
    uint64_t* clean = o_done + 2;      // [3] dead rows of the value tile are zero: the ring holds parts of three
    uint64_t* drain = clean + 3;       //     value tiles at most, so a barrier's phases are waited for in turn
    int2* desc = reinterpret_cast<int2*>(sm + P::OFF_DESC);    // [2] first key and TileFlags
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + P::OFF_TMEM);

    if (warp == kSoftWarps) {
        if (lane < 5) {
            const CUtensorMap* m = lane == 0 ? &maps.q : lane == 1 ? &maps.k : lane == 2 ? &maps.v : lane == 3 ? &maps.kc : &maps.vc;
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
        }
        if (lane == 0) {
            for (int s = 0; s < P::STAGES; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], 2);       // the products, and warp 10
            }
            mbar_init(q_full, 1);
            for (int g = 0; g < 2; ++g) {
                mbar_init(&s_full[g], 2);      // the product, and its tile's description
                mbar_init(&p_full[2 * g], 4);
                mbar_init(&p_full[2 * g + 1], 4);
                mbar_init(&o_done[g], 1);
            }
            for (int x = 0; x < 3; ++x) mbar_init(&clean[x], 1);
            mbar_init(drain, 1);
            fence_mbar_init();
            // Q is on its way before the block's set-up is done
            const uint64_t pol_q = policy_evict_first();
            const int nq = qa(1) < len ? 2 : 1;
            mbar_expect_tx(q_full, nq * P::QB);
            for (int g = 0; g < nq; ++g)
                for (int x = 0; x < D / 64; ++x)
                    tma_load_4d(sm + g * P::QB + x * (kM * 128), &maps.q, x * 64, qa(g), h * maps.qh, b * maps.qb, q_full,
                                pol_q);
        }
        __syncwarp();
    }
    if (warp == 0) tmem_alloc(tmem_slot, P::T_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = __shfl_sync(~0u, *tmem_slot, 0);

    if (warp == kSoftWarps) {
        // ---------------- TMA ----------------
        if (lane == 0) {
            const uint64_t pol_kv = policy_evict_last();   // heads share K and V
            int item = 0;
            bool ok = true;
            for (int it = 0; it < tiles && ok; ++it) {
                if (!active(it, 0) && !active(it, 1)) continue;
                const bool old = w.is_cache(it);
                const int row = w.base(it);
                for (int kv = 0; kv < 2 && ok; ++kv, ++item) {
                    const int s = item % P::STAGES;
                    if (item >= P::STAGES) ok = mbar_wait(&empty[s], (item / P::STAGES - 1) & 1, kErrMma);
                    if (!ok) break;
                    unsigned char* dst = sm + P::OFF_RING + s * P::STAGE;
                    mbar_expect_tx(&full[s], kv ? P::VB : P::KB);
                    const CUtensorMap* m = kv ? (old ? &maps.vc : &maps.v) : (old ? &maps.kc : &maps.k);
                    const int hc = old ? kvh : kvh * (kv ? maps.vh : maps.kh), bc = old ? b : b * (kv ? maps.vb : maps.kb);
                    for (int x = 0; x < (kv ? DV : D) / 64; ++x)
                        tma_load_4d(dst + x * (kKeys * 128), m, x * 64, row, hc, bc, &full[s], pol_kv);
                }
            }
            // no copy may be in flight when the block ends
            for (int i = max(0, item - P::STAGES); i < item; ++i)
                mbar_wait(&full[i % P::STAGES], (i / P::STAGES) & 1, kErrTmaLoad);
            mbar_wait(q_full, 0, kErrTmaLoad);
        }
    } else if (warp == kSoftWarps + 1) {
        // ---------------- MMA issue ----------------
        // The whole warp walks the tiles; one elected lane issues.  A wait that
        // gave up makes the later ones return at once: what is issued then
        // works on stale operands inside the CTA's own memory, and the error
        // word is set.
        const bool leader = elect_one();
        bool dead = false;
        auto wait = [&](uint64_t* bar, int phase, unsigned int site) {
            if (!dead) dead = !__all_sync(~0u, mbar_wait(bar, phase & 1, site));
        };
        // a negative scale negates Q (the descriptor's bit 13), so the maximum of the scores is what counts
        const uint32_t id_s = idesc_bf16_f32(kM, kKeys, 0, 0) | (a.scale < 0.f ? 1u << 13 : 0u), id_o = idesc_bf16_f32(kM, DV, 0, 1);
        const uint32_t q_at = smem_u32(sm), ring_at = q_at + P::OFF_RING;
        // a key tile to visit: its number, and per query tile whether and how
        struct Tile {
            int it, base;
            bool on[2];
            int flags[2];
        };
        auto next_tile = [&](int from) {
            Tile t{from, 0, {false, false}, {0, 0}};
            for (; t.it < tiles; ++t.it) {
                t.on[0] = active(t.it, 0);
                t.on[1] = active(t.it, 1);
                if (t.on[0] || t.on[1]) break;
            }
            if (t.it < tiles) {
                const bool old = w.is_cache(t.it);
                t.base = w.base(t.it);
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    // the tile of a query tile's last key is its last: keys behind it are in the future
                    t.flags[g] = (masked(t.it, g) ? kMasked : 0) | (old ? kCacheTile : 0) |
                                 (!old && t.base + kKeys >= qb(g) ? kLastTile : 0);
            }
            return t;
        };
        auto scores = [&](int g, const Tile& t, int item) {      // S_g = Q_g K^T
            const uint64_t dq = sdesc_sw128(q_at + g * P::QB, 16, 1024);
            const uint64_t dk = sdesc_sw128(ring_at + (item % P::STAGES) * P::STAGE, 16, 1024);
            if (leader) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t off = ((ks / 4) * (kKeys * 128) + (ks % 4) * 32) >> 4;
                    mma_bf16(tbase + P::T_S + g * kKeys, dq + off, dk + off, id_s, ks > 0);
                }
                mma_commit(&s_full[g]);
                desc[g] = make_int2(t.base, t.flags[g]);
                mbar_arrive(&s_full[g]);
            }
            __syncwarp();
        };
        auto loaded = [&](int item) { wait(&full[item % P::STAGES], item / P::STAGES, kErrTmaLoad); };
        auto release = [&](int item) {
            if (leader) mma_commit(&empty[item % P::STAGES]);
            __syncwarp();
        };
        Tile cur = next_tile(0);
        int done[2] = {0, 0}, item = 0, nv = 0;
        wait(q_full, 0, kErrTmaLoad);
        loaded(0);
        tc_fence_after();
#pragma unroll
        for (int g = 0; g < 2; ++g)
            if (cur.on[g]) scores(g, cur, 0);
        release(0);
        while (cur.it < tiles) {
            const Tile nx = next_tile(cur.it + 1);
            const bool more = nx.it < tiles;
            const int vi = item + 1, ki = item + 2;    // ring items: V of this tile, K of the next
            const uint64_t dv = sdesc_sw128(ring_at + (vi % P::STAGES) * P::STAGE, kKeys * 128, 1024);
            loaded(vi);
            wait(&clean[nv % 3], nv / 3, kErrMma);
            ++nv;
            if (more) loaded(ki);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                if (cur.on[g]) {
                    // O_g += P_g V, 64 keys at a time
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        wait(&p_full[2 * g + half], done[g], kErrMma);
                        tc_fence_after();
                        if (leader) {
#pragma unroll
                            for (int ks = half * 4; ks < half * 4 + 4; ++ks)
                                mma_bf16_ts(tbase + P::T_O + g * DV, tbase + P::T_S + g * kKeys + ks * 8,
                                            dv + ((ks * 2048) >> 4), id_o, done[g] > 0 || ks > 0);
                            if (half) mma_commit(&o_done[g]);
                        }
                        __syncwarp();
                    }
                    ++done[g];
                }
                if (more && nx.on[g]) scores(g, nx, ki);
            }
            release(vi);
            if (more) release(ki);
            cur = nx;
            item += 2;
        }
        // nothing in flight before TMEM is released
        if (leader) mma_commit(drain);
        __syncwarp();
        mbar_wait(drain, 0, kErrMma);
    } else if (warp == kSoftWarps + 2) {
        // ---------------- dead value rows ----------------
        bool ok = true;
        int item = 0, nv = 0;
        for (int it = 0; it < tiles && ok; ++it) {
            if (!active(it, 0) && !active(it, 1)) continue;
            // every load is waited for in turn, and its stage given back, by the whole warp
            ok = __all_sync(~0u, mbar_wait(&full[item % P::STAGES], (item / P::STAGES) & 1, kErrTmaLoad));
            if (ok && lane == 0) mbar_arrive(&empty[item % P::STAGES]);
            ++item;
            if (ok) ok = __all_sync(~0u, mbar_wait(&full[item % P::STAGES], (item / P::STAGES) & 1, kErrTmaLoad));
            const int live = w.live(it);
            if (ok && live < kKeys) {
                unsigned char* vt = sm + P::OFF_RING + (item % P::STAGES) * P::STAGE;
                const int first = max(live, 0), n = (kKeys - first) * 8;     // 16-byte pieces of a 64-column block
                for (int x = 0; x < DV / 64; ++x)
                    for (int e = lane; e < n; e += 32)
                        reinterpret_cast<uint4*>(vt + x * (kKeys * 128))[first * 8 + e] = make_uint4(0u, 0u, 0u, 0u);
                fence_async_smem();
            }
            __syncwarp();
            if (ok && lane == 0) {
                mbar_arrive(&clean[nv % 3]);
                mbar_arrive(&empty[item % P::STAGES]);
            }
            ++nv;
            ++item;
        }
    } else if (qa(warp >> 2) < len) {
        // ---------------- softmax ----------------
        const int g = warp >> 2, quad = warp & 3;
        const int row = qa(g) + quad * 32 + lane;
        // a zero scale weighs every visible key the same; it keeps masked keys at -inf
        const float c = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);
        const float slack = kSlack / c;
        float m = -INFINITY;
        f2 l[2] = {0, 0};    // sums of the weights of four classes of keys
        const uint32_t ts = tmem_addr(tbase, quad, P::T_S + g * kKeys), to = tmem_addr(tbase, quad, P::T_O + g * DV);
        int n = 0;          // tiles done
        bool ok = true;
        // a wait that gave up in one lane has given up for the warp: the lanes stay together
        auto wait = [&](uint64_t* bar, int phase) { return (bool)__all_sync(~0u, mbar_wait(bar, phase & 1, kErrMma)); };
        for (bool last = false; !last; ++n) {
            if (!wait(&s_full[g], n)) { ok = false; break; }
            tc_fence_after();
            const int2 tile = desc[g];
            last = tile.y & kLastTile;
            float s[4][32];
#pragma unroll
            for (int x = 0; x < 4; ++x) tmem_ld32(ts + x * 32, s[x]);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 4; ++x) tmem_regs_after_wait(s[x]);
            if (tile.y & kMasked) {
                const bool old = tile.y & kCacheTile;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t see = w.bits(old, row, tile.x + x * 32);
#pragma unroll
                    for (int j = 0; j < 32; ++j) s[x][j] = (see >> j) & 1u ? s[x][j] : -INFINITY;
                }
            }
            float t[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                t[x] = fmaxf(s[x][0], s[x][1]);
#pragma unroll
                for (int j = 2; j < 32; j += 2) t[x] = max3(t[x], s[x][j], s[x][j + 1]);
            }
            const float top = fmaxf(max3(t[0], t[1], t[2]), t[3]);
            const bool need = top > m + slack;       // also the first visible key: m = -inf
            if (__any_sync(~0u, need)) {
                const bool had = m != -INFINITY;
                const float f = need && had ? ex2_approx((m - top) * c) : 1.f;
                if (__any_sync(~0u, need && had)) {
                    // O holds the tiles before this one; a row that has seen nothing holds zeros
                    if (!wait(&o_done[g], n - 1)) { ok = false; break; }
                    tc_fence_after();
#pragma unroll 1
                    for (int x = 0; x < DV; x += 16) {
                        float o[16];
                        tmem_ld16(to + x, o);
                        tmem_ld_wait();
                        tmem_regs_after_wait(o);
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] *= f;
                        tmem_st16(to + x, o);
                    }
                }
                l[0] = mul2(l[0], pack2(f, f));
                l[1] = mul2(l[1], pack2(f, f));
                if (need) m = top;
            }
            const float off = m == -INFINITY ? 0.f : -m * c;
            const f2 c2 = pack2(c, c), off2 = pack2(off, off);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                uint32_t p[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const f2 y = fma2(pack2(s[x][2 * j], s[x][2 * j + 1]), c2, off2);
                    const float2 yv = unpack2(y);
                    const f2 e = pack2(ex2_approx(yv.x), ex2_approx(yv.y));
                    l[j % 2] = add2(l[j % 2], e);
                    const float2 v = unpack2(e);
                    p[j] = pack_bf16x2(v.x, v.y);
                }
                tmem_st16u(ts + x * 16, p);
                if (x % 2 == 1) {
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[2 * g + x / 2]);
                }
            }
        }
        if (ok && wait(&o_done[g], n - 1)) {
            tc_fence_after();
            const float2 l1 = unpack2(add2(l[0], l[1]));
            const float inv = 1.f / (l1.x + l1.y);     // every query sees itself
            __nv_bfloat16* op = (__nv_bfloat16*)a.out + b * a.st.out_batch + h * a.st.out_head + row * a.st.out_row;
#pragma unroll 1
            for (int x = 0; x < DV; x += 32) {
                float o[32];
                tmem_ld32(to + x, o);
                tmem_ld_wait();
                tmem_regs_after_wait(o);
                if (row < len) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float f[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = o[8 * j + i];
                        reinterpret_cast<uint4*>(op + x)[j] = pack8(f, inv);
                    }
                }
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tbase, P::T_COLS);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                       q == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p)
                   : nullptr;
    }();
    return fn;
}

// 4-D map [batch][head][row][inner] of a bf16 tensor, box 64 elements x 128
// rows, 128-byte swizzle; rows past `rows` read as zero.  An axis of stride 0
// (or of one entry) is mapped as one entry; *hs, *bs are its coordinate's factor.
bool map_4d(CUtensorMap* m, const void* base, int inner, int rows, int heads, int batch, long long row_stride,
            long long head_stride, long long batch_stride, int* hs, int* bs)
{
    auto fn = encode_fn();
    if (!fn) return false;
    *hs = head_stride > 0 && heads > 1;
    *bs = batch_stride > 0 && batch > 1;
    auto bytes = [&](long long s, bool real) { return (cuuint64_t)(real ? s * 2 : inner * 2); };
    cuuint64_t dims[4] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)(*hs ? heads : 1), (cuuint64_t)(*bs ? batch : 1)};
    cuuint64_t strides[3] = {bytes(row_stride, rows > 1), bytes(head_stride, *hs), bytes(batch_stride, *bs)};
    cuuint32_t box[4] = {64, 128, 1, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int DV>
cudaError_t launch(const WindowArgs& a)
{
    using P = Plan<D, DV>;
    Maps m;
    int ch, cb;   // a dense cache's coordinates of one-entry axes are 0 anyway
    if (!map_4d(&m.q, a.q, D, a.N, a.Hq, a.B, a.st.q_row, a.st.q_head, a.st.q_batch, &m.qh, &m.qb) ||
        !map_4d(&m.k, a.k, D, a.N, a.Hkv, a.B, a.st.k_row, a.st.k_head, a.st.k_batch, &m.kh, &m.kb) ||
        !map_4d(&m.v, a.v, DV, a.N, a.Hkv, a.B, a.st.v_row, a.st.v_head, a.st.v_batch, &m.vh, &m.vb))
        return cudaErrorInvalidValue;
    m.kc = m.k;
    m.vc = m.v;
    if (a.k_cache) {
        const long long cap = (long long)a.window + a.sinks;
        if (!map_4d(&m.kc, a.k_cache, D, (int)cap, a.Hkv, a.B, D, cap * D, cap * a.Hkv * D, &ch, &cb) ||
            !map_4d(&m.vc, a.v_cache, DV, (int)cap, a.Hkv, a.B, DV, cap * DV, cap * a.Hkv * DV, &ch, &cb))
            return cudaErrorInvalidValue;
    }
    auto kern = window_prefill_tc<D, DV>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, P::BYTES);
    if (e != cudaSuccess) return e;
    const int pairs = (a.N + 2 * kM - 1) / (2 * kM);
    if (pairs > 65535) return cudaErrorInvalidValue;
    kern<<<dim3(a.Hq, pairs, a.B), kThreads, P::BYTES, a.stream>>>(m, a, window_lens(a));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_prefill_tc(const WindowArgs& a)
{
    if (a.d == 64) return a.dv == 64 ? launch<64, 64>(a) : launch<64, 128>(a);
    return a.dv == 64 ? launch<128, 64>(a) : launch<128, 128>(a);
}

unsigned int read_and_clear_device_error_window(cudaStream_t stream)
{
    unsigned int v = 0;
    if (cudaMemcpyFromSymbolAsync(&v, sm100::g_device_error, sizeof(v), 0, cudaMemcpyDeviceToHost, stream) !=
        cudaSuccess)
        return 0;
    cudaStreamSynchronize(stream);
    if (v) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbolAsync(sm100::g_device_error, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
        cudaStreamSynchronize(stream);
    }
    return v;
}

}  // namespace la
