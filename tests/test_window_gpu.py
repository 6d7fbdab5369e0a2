"""Sliding-window attention with sinks on the GPU: prompts and token steps over
the rolling cache, against the definition over absolute positions in float64,
element by element.

Tolerances come from the arithmetic.  With u = 2^-24 and r half a step of the
storage type (2^-8 bf16, u fp32): a score is a sum of d products, off by
e = (d + 4) u |scale| sum |q k|; with x = score - maximum in log2 units, the
weight 2^x is off by e ln-relative, by |x| 2^-23 from x's own rounding, and by
the exponential itself, 2^-21.  bf16 weights enter the value product rounded to
bf16 (2^-8), from exponentials good to 2^-12.  Numerator and denominator each
carry such errors, so with A = sum p |v| over the normalised weights
    |do| <= A (2 (e + |x|max 2^-23 + 2^-21) + (n + 4) u  [+ 2 * 2^-12 + 2^-8 for bf16]) + r |o|
"""
import numpy as np
import pytest
import torch

import causal_kernelized_linear_la_b200 as la

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def _f64(t):
    return t.detach().double().cpu().numpy()


def _ref(q, k, v, first, window, sinks, scale, dtype):
    """Queries at positions first.. over keys at positions 0..: (o, bound)."""
    i = np.arange(first, first + q.shape[0])[:, None]
    j = np.arange(k.shape[0])[None]
    see = (j <= i) & ((i - j < window) | (j < sinks))
    s = q @ k.T * scale
    e = (q.shape[1] + 4) * U * abs(scale) * (np.abs(q) @ np.abs(k).T).max(1, keepdims=True)
    s = np.where(see, s, -np.inf)
    x = s - s.max(1, keepdims=True)
    p = np.exp(x)
    p /= p.sum(1, keepdims=True)
    deep = np.where(see, -x, 0).max(1, keepdims=True) * 1.4427
    rel = 2 * (e + deep * 2.0 ** -23 + 2.0 ** -21) + (see.sum(1, keepdims=True) + 4) * U
    if dtype == torch.bfloat16:
        rel = rel + 2 * 2.0 ** -12 + 2.0 ** -8
    o = p @ v
    return o, (p @ np.abs(v)) * rel + HALF[dtype] * np.abs(o) + 1e-37


def _slot(p, window, sinks):
    return p if p < sinks else sinks + (p - sinks) % window


def _fill(cache, hist, upto, window, sinks):
    """The rolling cache after the tokens 0..upto-1 of hist [H, P, d]."""
    for p in range(upto):
        if p < sinks or p >= upto - window:
            cache[:, _slot(p, window, sinks)] = hist[:, p]


def _check(got, ref, tol, what):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} values off, worst by {np.nanmax(np.abs(got - ref) / tol):.2f} of the bound"


def _make(dtype, B, H, P, d, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(B, H, P, d, generator=g)).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,Hq,Hkv,N,d,dv,window,sinks,lens,fused", [
    (1, 1, 1, 1, 64, 64, 1, 0, None, False),              # one token
    (1, 2, 2, 65, 64, 64, 1, 0, None, False),             # sees itself only
    (2, 4, 2, 130, 128, 128, 40, 3, None, True),
    (1, 3, 1, 300, 64, 128, 1000, 0, None, False),        # window past the prompt: plain causal
    (1, 8, 1, 257, 128, 64, 64, 200, None, False),        # more sinks than a tile
    (3, 2, 2, 200, 64, 64, 63, 5, [200, 0, 77], True),    # ragged, one empty
    (2, 2, 1, 400, 128, 128, 129, 1, [1, 400], False),
    (1, 1, 1, 700, 128, 128, 256, 500, None, False),      # sinks reach into the band
    (1, 2, 2, 512, 128, 128, 128, 0, None, True),         # whole tiles
    (1, 4, 4, 1100, 64, 64, 300, 4, None, False),
    (130, 1, 1, 3, 64, 64, 2, 1, [i % 4 for i in range(130)], False),   # more sequences than one launch takes
])
def test_prefill(dtype, B, Hq, Hkv, N, d, dv, window, sinks, lens, fused):
    if fused:
        qkv = _make(dtype, B, N, Hq + 2 * Hkv, d, N).transpose(1, 2)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = _make(dtype, B, Hq, N, d, 1), _make(dtype, B, Hkv, N, d, 2), _make(dtype, B, Hkv, N, dv, 3)
    n_of = lens or [N] * B
    if fused:
        dev = qkv.transpose(1, 2).contiguous().cuda().transpose(1, 2)
        qd, kd, vd = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]
    else:
        qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    for b in range(B):
        for t in (qd, kd, vd):
            t[b, :, n_of[b]:] = float("nan")
    out = torch.full((B, N, Hq, dv), 7.0, dtype=dtype, device="cuda").transpose(1, 2) if fused else \
        torch.full((B, Hq, N, dv), 7.0, dtype=dtype, device="cuda")
    la.la_window_prefill(qd, kd, vd, window, sinks=sinks, seq_lens=lens, out=out)
    la.la_prefill_check()
    o, q, k, v = _f64(out), _f64(q), _f64(k), _f64(v)
    for b in range(B):
        n = n_of[b]
        for h in range(Hq):
            j = h // (Hq // Hkv)
            if n:
                ref, tol = _ref(q[b, h, :n], k[b, j, :n], v[b, j, :n], 0, window, sinks, d ** -0.5, dtype)
                _check(o[b, h, :n], ref, tol, f"sequence {b} head {h}")
            assert (o[b, h, n:] == 7.0).all()


def _with_cache(dtype, B, Hq, Hkv, N, d, dv, window, sinks, pos, lens, scale=None, decode=False):
    """One call behind caches filled to pos; everything a slot does not hold is NaN."""
    top = max(max(pos), 0) + N
    kh, vh = _make(dtype, B, Hkv, top, d, 5, 1.5), _make(dtype, B, Hkv, top, dv, 6)
    q = _make(dtype, B, Hq, N, d, 7, 1.5)
    cap = window + sinks
    kc = torch.full((B, Hkv, cap, d), float("nan"), dtype=dtype)
    vc = torch.full((B, Hkv, cap, dv), float("nan"), dtype=dtype)
    k, v = torch.full((B, Hkv, N, d), float("nan"), dtype=dtype), torch.full((B, Hkv, N, dv), float("nan"), dtype=dtype)
    want_k, want_v = kc.clone(), vc.clone()
    for b in range(B):
        p = max(pos[b], 0)
        n = lens[b] if pos[b] >= 0 else 0
        _fill(kc[b], kh[b], p, window, sinks)
        _fill(vc[b], vh[b], p, window, sinks)
        k[b, :, :lens[b]], v[b, :, :lens[b]] = kh[b, :, p:p + lens[b]], vh[b, :, p:p + lens[b]]
        _fill(want_k[b], kh[b], p, window, sinks)
        _fill(want_v[b], vh[b], p, window, sinks)
        for i in range(n):     # what a run of single tokens leaves behind
            want_k[b, :, _slot(p + i, window, sinks)] = kh[b, :, p + i]
            want_v[b, :, _slot(p + i, window, sinks)] = vh[b, :, p + i]
    kcd, vcd, posd = kc.cuda(), vc.cuda(), torch.tensor(pos, dtype=torch.int32, device="cuda")
    out = torch.full((B, Hq, N, dv), 7.0, dtype=dtype, device="cuda")
    if decode:
        la.la_window_decode_step(q[:, :, 0].contiguous().cuda(), k[:, :, 0].contiguous().cuda(),
                                 v[:, :, 0].contiguous().cuda(), kcd, vcd, posd, window, sinks=sinks, scale=scale,
                                 out=out[:, :, 0])
    else:
        la.la_window_prefill(q.cuda(), k.cuda(), v.cuda(), window, sinks=sinks, k_cache=kcd, v_cache=vcd, pos=posd,
                             seq_lens=lens, scale=scale, out=out)
    la.la_prefill_check()
    o = _f64(out)
    for b in range(B):
        n = lens[b] if pos[b] >= 0 else 0
        p = max(pos[b], 0)
        for h in range(Hq):
            j = h // (Hq // Hkv)
            if n:
                ref, tol = _ref(_f64(q[b, h, :n]), _f64(kh[b, j, :p + n]), _f64(vh[b, j, :p + n]), p, window, sinks,
                                d ** -0.5 if scale is None else scale, dtype)
                _check(o[b, h, :n], ref, tol, f"sequence {b} head {h}")
            assert (o[b, h, n:] == 7.0).all()
    same = lambda x, y: torch.equal(x.cpu().view(torch.uint8), y.view(torch.uint8))  # noqa: E731
    assert same(kcd, want_k) and same(vcd, want_v)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,Hq,Hkv,N,d,dv,window,sinks,pos,lens,scale", [
    (2, 2, 1, 70, 64, 64, 50, 3, [0, 400], [70, 70], None),
    (3, 4, 2, 33, 128, 128, 100, 4, [2, 5, 60], [33, 0, 20], 0.2),      # a cache that is still filling
    (2, 1, 1, 5, 128, 64, 7, 0, [6, 7], [5, 5], None),
    (2, 2, 2, 300, 64, 128, 64, 150, [100, 149], [300, 299], None),      # sinks still arriving
    (2, 8, 1, 200, 64, 64, 256, 2, [-1, 999], [200, 200], None),         # one idle sequence
    (1, 2, 2, 260, 128, 128, 130, 130, [520], [260], -0.1),
    (2, 1, 1, 1, 64, 64, 300, 1, [300, 301], [1, 1], None),
])
def test_prefill_behind_the_cache(dtype, B, Hq, Hkv, N, d, dv, window, sinks, pos, lens, scale):
    _with_cache(dtype, B, Hq, Hkv, N, d, dv, window, sinks, pos, lens, scale)


@pytest.mark.parametrize("N", [40000, 300])
def test_prefill_behind_a_long_cache(N):
    """A chunk behind a full cache of 512 tiles: its later queries see none of the
    hundreds of tiles between the sinks and the window's edge, which every walking
    warp passes over on its own.  Sampled rows against the definition."""
    d, window, sinks, pos0 = 64, 65536, 4, 65536 + 4 + 1000      # the ring has wrapped
    g = torch.Generator(device="cuda").manual_seed(N)
    r = lambda n: torch.randn(1, 1, n, d, generator=g, device="cuda").bfloat16()  # noqa: E731
    kh, vh, q = r(pos0 + N), r(pos0 + N), r(N)
    p = torch.arange(pos0, device="cuda")
    p = p[(p < sinks) | (p >= pos0 - window)]
    slot = torch.where(p < sinks, p, sinks + (p - sinks) % window)
    kc = torch.zeros(1, 1, window + sinks, d, device="cuda", dtype=torch.bfloat16)
    vc = torch.zeros_like(kc)
    kc[:, :, slot], vc[:, :, slot] = kh[:, :, p], vh[:, :, p]
    o = la.la_window_prefill(q, kh[:, :, pos0:], vh[:, :, pos0:], window, sinks=sinks, k_cache=kc, v_cache=vc,
                             pos=torch.tensor([pos0], dtype=torch.int32, device="cuda"))
    la.la_prefill_check()
    o, q, kh, vh = (_f64(t)[0, 0] for t in (o, q, kh, vh))
    for i in sorted({0, 1, 127, 128, 255, 256, N // 2, N - 257, N - 129, N - 1} & set(range(N))):
        ref, tol = _ref(q[i:i + 1], kh[:pos0 + i + 1], vh[:pos0 + i + 1], pos0 + i, window, sinks, d ** -0.5, torch.bfloat16)
        _check(o[i:i + 1], ref, tol, f"query {i}")
    i = np.arange(pos0, pos0 + N)
    held = np.concatenate([np.arange(sinks), i[-window:]])
    at = torch.from_numpy(np.where(held < sinks, held, sinks + (held - sinks) % window)).cuda()
    assert np.array_equal(_f64(kc)[0, 0][at.cpu()], kh[held]) and np.array_equal(_f64(vc)[0, 0][at.cpu()], vh[held])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,Hq,Hkv,d,dv,window,sinks,pos", [
    (1, 1, 1, 64, 64, 1, 0, [0]),
    (3, 4, 4, 128, 128, 40, 4, [0, 3, 4]),
    (4, 8, 2, 64, 128, 100, 3, [50, 102, 103, 777]),
    (3, 6, 2, 128, 64, 33, 0, [-1, 32, 33]),            # one idle sequence
    (2, 16, 1, 128, 128, 700, 5, [704, 2000]),          # sixteen heads a kv head, several splits
    (2, 10, 2, 64, 64, 1500, 200, [150, 1699]),
    (2, 40, 2, 128, 128, 130, 1, [129, 131]),
])
def test_decode(dtype, B, Hq, Hkv, d, dv, window, sinks, pos):
    _with_cache(dtype, B, Hq, Hkv, 1, d, dv, window, sinks, pos, [1] * B, decode=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompt_pieces_then_tokens(dtype):
    """A prompt in pieces and then token by token, as a server runs it: every
    output within the bound of the whole sequence's definition."""
    B, Hq, Hkv, d, window, sinks, pieces, steps = 2, 4, 2, 64, 48, 4, (60, 1, 30), 70
    total = sum(pieces) + steps
    q, k, v = _make(dtype, B, Hq, total, d, 11), _make(dtype, B, Hkv, total, d, 12), _make(dtype, B, Hkv, total, d, 13)
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    kc = torch.zeros(B, Hkv, window + sinks, d, dtype=dtype, device="cuda")
    vc, pos = torch.zeros_like(kc), torch.zeros(B, dtype=torch.int32, device="cuda")
    parts, t = [], 0
    for n in pieces:
        parts.append(la.la_window_prefill(qd[:, :, t:t + n], kd[:, :, t:t + n], vd[:, :, t:t + n], window, sinks=sinks,
                                          k_cache=kc, v_cache=vc, pos=pos))
        pos += n
        t += n
    for _ in range(steps):
        parts.append(la.la_window_decode_step(qd[:, :, t], kd[:, :, t], vd[:, :, t], kc, vc, pos, window,
                                              sinks=sinks)[:, :, None])
        pos += 1
        t += 1
    la.la_prefill_check()
    o = _f64(torch.cat(parts, 2))
    for b in range(B):
        for h in range(Hq):
            ref, tol = _ref(_f64(q[b, h]), _f64(k[b, h // 2]), _f64(v[b, h // 2]), 0, window, sinks, d ** -0.5, dtype)
            _check(o[b, h], ref, tol, f"sequence {b} head {h}")


def test_refusals():
    z = lambda *s, **kw: torch.zeros(*s, device="cuda", dtype=kw.get("dtype", torch.bfloat16))  # noqa: E731
    q, k = z(2, 4, 8, 64), z(2, 2, 8, 64)
    kc, pos = z(2, 2, 20, 64), z(2, dtype=torch.int32)
    vc = kc.clone()

    def code(f):
        with pytest.raises(la.LaError) as e:
            f()
        return e.value.code

    assert code(lambda: la.la_window_prefill(q, k, k, 0)) == la.LA_ERR_INVALID
    assert code(lambda: la.la_window_prefill(q, k, k, 4, sinks=-1)) == la.LA_ERR_INVALID
    assert code(lambda: la.la_window_prefill(q, k, k, 4, scale=float("nan"))) == la.LA_ERR_INVALID
    assert code(lambda: la.la_window_prefill(q, k, k, 4, pos=pos)) == la.LA_ERR_INVALID          # pos without a cache
    assert code(lambda: la.la_window_prefill(q, k, k, 16, sinks=4, k_cache=kc)) == la.LA_ERR_INVALID   # half a cache
    assert code(lambda: la.la_window_prefill(q, k, k, 16, sinks=4, k_cache=kc, v_cache=kc)) == la.LA_ERR_INVALID
    assert code(lambda: la.la_window_prefill(q, k, k, 4, seq_lens=[8, 9])) == la.LA_ERR_INVALID
    assert code(lambda: la.la_window_prefill(z(2, 4, 8, 32), z(2, 2, 8, 32), z(2, 2, 8, 32), 4)) == la.LA_ERR_UNSUPPORTED
    odd = z(2, 4, 8, 68)[..., :64]
    assert code(lambda: la.la_window_prefill(odd, k, k, 4)) == la.LA_ERR_ALIGN
    three = z(2, 3, 8, 64)
    assert code(lambda: la.la_window_prefill(q, three, three, 4)) == la.LA_ERR_INVALID           # 4 heads over 3
    with pytest.raises(ValueError):
        la.la_window_prefill(q, k, k.float(), 4)
    with pytest.raises(ValueError):
        la.la_window_prefill(q, k, k, 4, sinks=4, k_cache=kc, v_cache=vc)                        # cache of another size
    with pytest.raises(TypeError):
        la.la_window_prefill(q.half(), k.half(), k.half(), 4)
    with pytest.raises(ValueError):
        la.la_window_decode_step(q[:, :, 0], k[:, :, 0], k[:, :, 0], kc, vc, pos.long(), 16, sinks=4)
    with pytest.raises(ValueError):
        la.la_window_decode_step(q[:, :, 0], k[:, :, 0], k[:, :, 0], kc, vc, pos.cpu(), 16, sinks=4)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_outputs_beside_and_over_q(dtype):
    """out as a part of the buffer that q, k and v are parts of, and out in q's place:
    the bits of an out of its own."""
    B, N, H, Hkv, d, window, sinks, lens = 2, 300, 4, 2, 64, 70, 3, [300, 111]
    g = torch.Generator().manual_seed(21)
    base = torch.randn(B, N, 2 * H + 2 * Hkv, d, generator=g).to(dtype).cuda()

    def parts(t):
        t = t.transpose(1, 2)
        return t[:, :H], t[:, H:H + Hkv], t[:, H + Hkv:H + 2 * Hkv], t[:, H + 2 * Hkv:]
    q, k, v, _ = parts(base)
    want = torch.full((B, H, N, d), 7.0, dtype=dtype, device="cuda")
    la.la_window_prefill(q, k, v, window, sinks=sinks, seq_lens=lens, out=want)
    one = base.clone()
    q1, k1, v1, o1 = parts(one)
    o1.fill_(7.0)
    la.la_window_prefill(q1, k1, v1, window, sinks=sinks, seq_lens=lens, out=o1)
    assert torch.equal(o1, want) and all(torch.equal(x, y) for x, y in zip((q1, k1, v1), (q, k, v)))
    two = base.clone()
    q2, k2, v2, _ = parts(two)
    la.la_window_prefill(q2, k2, v2, window, sinks=sinks, seq_lens=lens, out=q2)
    for b, n in enumerate(lens):
        assert torch.equal(q2[b, :, :n], want[b, :, :n]) and torch.equal(q2[b, :, n:], q[b, :, n:])
    # one token, q's heads over several CTAs of a cluster
    cap = 2000
    kc, vc = torch.randn(B, Hkv, cap, d, generator=g).to(dtype).cuda(), torch.randn(B, Hkv, cap, d, generator=g).to(dtype).cuda()
    pos = torch.tensor([5000, 70], dtype=torch.int32, device="cuda")
    q1, k1, v1 = q[:, :, 0].contiguous(), k[:, :, 0].contiguous(), v[:, :, 0].contiguous()
    kc2, vc2 = kc.clone(), vc.clone()
    want = la.la_window_decode_step(q1, k1, v1, kc, vc, pos, cap - 4, sinks=4)
    got = la.la_window_decode_step(q1, k1, v1, kc2, vc2, pos, cap - 4, sinks=4, out=q1)
    assert got is q1 and torch.equal(q1, want)
    la.la_prefill_check()
    # out over k, over a cache, over rows of q that are not its own: refused, nothing written
    keep = two.clone()
    for out in (two.transpose(1, 2)[:, 1:1 + H], two.transpose(1, 2)[:, H:2 * H]):
        with pytest.raises(la.LaError) as e:
            la.la_window_prefill(q2, k2, v2, window, sinks=sinks, out=out)
        assert e.value.code == la.LA_ERR_INVALID
    with pytest.raises(la.LaError) as e:
        la.la_window_decode_step(want, k1, v1, kc, vc, pos, cap - 4, sinks=4, out=kc.view(-1)[:B * H * d].view(B, H, d))
    assert e.value.code == la.LA_ERR_INVALID
    torch.cuda.synchronize()
    assert torch.equal(two, keep)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cap,pos", [(44, 30), (44, 43), (44, 200), (1500, 700), (1500, 9000)])
def test_decode_infinite_value_in_the_last_slot(dtype, cap, pos):
    """An infinite value that the token sees makes its column of the output infinite, with
    its sign, and no other: also in the last slot in use, which ends inside a block of slots."""
    B, Hq, Hkv, d, sinks = 1, 8, 2, 64, 4
    g = torch.Generator().manual_seed(cap + pos)
    r = lambda *s: (0.3 * torch.randn(*s, generator=g)).to(dtype).cuda()  # noqa: E731
    q, k, v, kc, vc = r(B, Hq, d), r(B, Hkv, d), r(B, Hkv, d), r(B, Hkv, cap, d), r(B, Hkv, cap, d)
    window, used = cap - sinks, min(pos + 1, cap)
    posd = torch.tensor([pos], dtype=torch.int32, device="cuda")
    want = la.la_window_decode_step(q, k, v, kc.clone(), vc.clone(), posd, window, sinks=sinks)
    last = v if _slot(pos, window, sinks) == used - 1 else vc[:, :, used - 1]
    last[:, 0, 5], last[:, 1, 63] = float("inf"), float("-inf")
    got = la.la_window_decode_step(q, k, v, kc.clone(), vc.clone(), posd, window, sinks=sinks)
    hit = torch.zeros(B, Hq, d, dtype=torch.bool, device="cuda")
    hit[:, :4, 5] = hit[:, 4:, 63] = True
    assert (got[:, :4, 5] == float("inf")).all() and (got[:, 4:, 63] == float("-inf")).all()
    assert torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("B,Hq,Hkv,d,dv,window,sinks,pos", [
    (2, 16, 2, 128, 128, 700, 5, [704, 2000]),
    (40, 32, 8, 64, 64, 400, 4, [100 + 7 * b for b in range(40)]),
    (80, 16, 8, 64, 128, 97, 3, [50 + b for b in range(80)]),
])
def test_decode_keeps_the_weights(B, Hq, Hkv, d, dv, window, sinks, pos):
    """bf16 token steps take each weight as two bf16 parts: the upper one cut off, so the rest is
    below 2^-7 of it, and that rest rounded by 2^-8 of itself.  2^-15 of the weights is what is
    lost, where one rounding would take 2^-8; the other terms are those of fp32 inputs."""
    g = torch.Generator().manual_seed(B)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    cap = window + sinks
    q, k, v, kc, vc = r(B, Hq, d), r(B, Hkv, d), r(B, Hkv, dv), r(B, Hkv, cap, d), r(B, Hkv, cap, dv)
    o = la.la_window_decode_step(q, k, v, kc, vc, torch.tensor(pos, dtype=torch.int32, device="cuda"), window, sinks=sinks)
    o, q, kc, vc = _f64(o), _f64(q), _f64(kc), _f64(vc)
    for b in range(B):
        used = min(pos[b] + 1, cap)       # the slots in use are all seen, in any order
        for h in range(Hq):
            K, V = kc[b, h // (Hq // Hkv), :used], vc[b, h // (Hq // Hkv), :used]
            ref, tol = _ref(q[b, h:h + 1], K, V, used - 1, used, 0, d ** -0.5, torch.float32)
            spread, _ = _ref(q[b, h:h + 1], K, np.abs(V), used - 1, used, 0, d ** -0.5, torch.float32)
            _check(o[b, h:h + 1], ref, tol + 2.0 ** -15 * spread + 2.0 ** -8 * np.abs(ref), f"sequence {b} head {h}")
