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
};

}  // namespace la
