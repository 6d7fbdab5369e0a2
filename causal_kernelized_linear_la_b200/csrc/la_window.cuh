// Sliding-window attention with sinks: what the prompt kernels and the token
// step share -- the call's arguments, the rolling cache's slots and the walk
// over the key tiles a block of queries can see.
//
// The token at position p sees itself, the window - 1 tokens before it and the
// tokens at positions below `sinks`.  The cache has one slot a sink and
// `window` ring slots: position p lives in slot p (p < sinks) or
// sinks + (p - sinks) mod window, so the slots hold exactly the sinks and the
// last `window` other tokens.
#pragma once

#include "la_internal.cuh"

namespace la {

struct WindowArgs {
    const void* q;
    const void* k;
    const void* v;
    void* k_cache;          // [B, Hkv, sinks + window, d] or null
    void* v_cache;          // [B, Hkv, sinks + window, dv] or null
    const int* pos;         // device, [B] or null (0): tokens already in the cache; < 0: an idle sequence
    void* out;
    const int* seq_lens;    // host, or null
    int B, Hq, Hkv, N, d, dv;
    int window, sinks;
    float scale;
    la_window_strides st;
    la_dtype dtype;
    cudaStream_t stream;
};

struct WindowLens {
    int use;
    int n[kMaxSeqLens];
};

cudaError_t launch_window_prefill_simt(const WindowArgs& a);
cudaError_t launch_window_prefill_tc(const WindowArgs& a);
unsigned int read_and_clear_device_error_window(cudaStream_t stream);
cudaError_t launch_window_cache_update(const WindowArgs& a);
cudaError_t launch_window_decode(const WindowArgs& a);

__host__ inline WindowLens window_lens(const WindowArgs& a)
{
    WindowLens l{};
    l.use = a.seq_lens != nullptr;
    if (a.seq_lens)
        for (int b = 0; b < a.B; ++b) l.n[b] = a.seq_lens[b];
    return l;
}

// Position of ring slot r relative to the first new token (negative), for a
// ring of `window` slots that has taken `taken` tokens so far (taken > 0).
__device__ __forceinline__ int ring_age(int r, int last, int window)
{
    // last = (taken - 1) % window holds -1, the slots below it older ones, the
    // slots above it the turn before
    return r <= last ? -1 - (last - r) : -1 - (last - r + window);
}

// The key tiles (of T keys) that the queries [q0, q1) of one sequence can see,
// in this order: tiles of cache slots, tiles of the new tokens that are sinks,
// and the tiles of new tokens in the window's band.
template <int T>
struct KeyWalk {
    int start;               // position of the first new token
    int window, sinks, len;
    int q0, q1;
    int cache_tiles;         // tiles of cache slots to visit (the visible ones among them)
    int taken, last;         // tokens the ring has taken, slot of the newest
    int sink_tiles;          // leading tiles of new tokens, ahead of the band
    int band0, band1;        // band tiles [band0, band1)

    __device__ __forceinline__ void init(bool cached, int start_, int window_, int sinks_, int len_, int q0_, int q1_)
    {
        start = start_;
        window = window_;
        sinks = sinks_;
        len = len_;
        q0 = q0_;
        q1 = q1_;
        taken = start > sinks ? start - sinks : 0;
        last = taken > 0 ? (taken - 1) % window : 0;
        const int held = cached && start > 0 ? (start < sinks ? start : sinks + (taken < window ? taken : window)) : 0;
        // ring tokens are visible to queries up to window - 1 behind the newest
        const int reach = q0 >= window - 1 ? (held < sinks ? held : sinks) : held;
        cache_tiles = (reach + T - 1) / T;
        const int ns = start < sinks ? (sinks - start < len ? sinks - start : len) : 0;
        const int lo = q0 >= window ? q0 - window + 1 : 0;
        band0 = lo / T;
        band1 = (q1 + T - 1) / T;
        const int st = (ns + T - 1) / T;
        sink_tiles = st < band0 ? st : band0;
    }
    __device__ __forceinline__ int count() const { return cache_tiles + sink_tiles + (band1 - band0); }
    __device__ __forceinline__ bool is_cache(int i) const { return i < cache_tiles; }
    // first cache slot or first new token of tile i
    __device__ __forceinline__ int base(int i) const
    {
        if (i < cache_tiles) return i * T;
        i -= cache_tiles;
        return (i < sink_tiles ? i : band0 + i - sink_tiles) * T;
    }
    // cache slot s holds a token (of an earlier call)
    __device__ __forceinline__ bool slot_held(int s) const
    {
        return s < sinks ? s < start : s - sinks < taken && s - sinks < window;
    }
    __device__ __forceinline__ bool sees_slot(int i, int s) const
    {
        if (s < sinks) return s < start;
        const int r = s - sinks;
        return r < taken && r < window && i - ring_age(r, last, window) < window;
    }
    __device__ __forceinline__ bool sees_new(int i, int j) const
    {
        return j <= i && j < len && (i - j < window || j < sinks - start);
    }

    // The slots that query i sees, as three intervals of slot numbers: sinks,
    // ring tokens written in the ring's current turn, ring tokens of the turn
    // before.  (ring_age(r) > i - window solved for r on each side of `last`.)
    struct Span {
        int lo, hi;
    };
    __device__ __forceinline__ Span sink_slots() const { return {0, start < sinks ? start : sinks}; }
    __device__ __forceinline__ Span turn_slots(int i) const
    {
        const int lo = i - window + last + 2;
        return {sinks + (lo > 0 ? lo : 0), taken > 0 ? sinks + last + 1 : 0};
    }
    __device__ __forceinline__ Span past_slots(int i) const
    {
        const int lo = i + last + 2;
        return {sinks + (lo > last + 1 ? lo : last + 1), sinks + (taken < window ? taken : window)};
    }
    __device__ __forceinline__ int sinks_left() const { return start < sinks ? sinks - start : 0; }

    // some key of tile it is visible to some query of [qa, qb)
    __device__ __forceinline__ bool any(int it, int qa, int qb) const
    {
        const int b = base(it);
        if (!is_cache(it)) return b < qb && (b + T > qa - window + 1 || b < sinks_left());
        const Span s = sink_slots(), t = turn_slots(qa), p = past_slots(qa);   // the first query sees the most
        return b < s.hi || max(t.lo, b) < min(t.hi, b + T) || max(p.lo, b) < min(p.hi, b + T);
    }
    // every key of tile it is visible to every query of [qa, qb)
    __device__ __forceinline__ bool all(int it, int qa, int qb) const
    {
        const int b = base(it), e = b + T;
        if (!is_cache(it)) return e - 1 <= qa && e <= len && (b >= qb - window || e <= sinks_left());
        const Span t = turn_slots(qb - 1), p = past_slots(qb - 1);             // the last query sees the least
        return e <= sink_slots().hi || (b >= t.lo && e <= t.hi) || (b >= p.lo && e <= p.hi);
    }
    // cache slots in use: always a prefix of them
    __device__ __forceinline__ int held() const
    {
        return start < sinks ? start : sinks + (taken < window ? taken : window);
    }
    // keys of tile it, counted from its base, that hold a token: the rest may hold anything
    __device__ __forceinline__ int live(int it) const { return (is_cache(it) ? held() : len) - base(it); }
    // 32 keys from `key` on (a slot or a new token): bit c is set if query i sees key + c
    __device__ __forceinline__ static uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
    __device__ __forceinline__ static uint32_t within(Span s, int key) { return below(s.hi - key) & ~below(s.lo - key); }
    __device__ __forceinline__ uint32_t bits(bool old, int i, int key) const
    {
        if (old) return within(sink_slots(), key) | within(turn_slots(i), key) | within(past_slots(i), key);
        const int end = i < len ? i + 1 : len;
        return within({i - window + 1, end}, key) | within({0, min(end, sinks_left())}, key);
    }
};

}  // namespace la
