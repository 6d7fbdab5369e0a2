"""Selective state-space layer on the GPU: convolution, prompt scan and token
step against their definitions in float64, element by element.

Tolerances come from the arithmetic, not from runs.  With u = 2^-24 (half an
fp32 step, relative) and r = half a step of the storage type (2^-8 for bf16,
u for fp32):

* convolution: w products and a bias summed in fp32 are off by at most
  (w + 1) u times the sum of their magnitudes S; SiLU has slope at most 1.1 and
  its own arithmetic is good to 2^-19 relative (an exponential of up to 2^-21
  where |y| is below 16, a reciprocal, a product); the result is rounded once.
* recurrence: the reference carries a bound E on the state's error beside the
  state.  A step size is off by at most q = 2^-20 (1 + |v|) relative, with v
  the biased raw value (softplus of a sum); without softplus by 2 u.  Its
  decay a = exp(dt A) is off by 2^-22 + |dt A| (q + 3 u) relative (2^x to
  2^-22, its argument by a constant's, a product's and dt's error), the
  written term by q + 3 u, and each of the two sums by u:
      E <- a E + |a h| (2^-22 + |dt A| (q + 3 u) + u) + |dt x B| (q + 4 u) + u |h|
  and to second order a factor 1.01.  y sums n products of C and h (each off by |C| E and
  (n + 4) u relative), adds D x, and is gated and rounded as above.
* segments of a long sequence take exp(A sum dt) for their decay: one more
  2^-22 + |A sum dt| 2^-20 relative per segment, which the bound of the tokens
  inside it covers (each token has 2^-22 and |dt A| 2^-20 of its own).
"""
import numpy as np
import pytest
import torch

import causal_kernelized_linear_la_b200 as la

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def _silu(y):
    return y / (1 + np.exp(-y))


def _conv_ref(x, w, bias, cache, silu, r):
    """One sequence: (y, its error bound, new cache), all float64."""
    N, D = x.shape
    W = w.shape[1]
    xh = np.concatenate([cache, x])
    y = np.zeros((N, D))
    mag = np.zeros((N, D))
    for i in range(W):
        y += w[:, i] * xh[i:i + N]
        mag += np.abs(w[:, i] * xh[i:i + N])
    if bias is not None:
        y += bias
        mag += np.abs(bias)
    err = (W + 1) * U * mag
    if silu:
        y = _silu(y)
        err = 1.1 * err + 2.0 ** -19 * np.abs(y)
    return y, 1.01 * err + r * np.abs(y) + 1e-37, xh[N:]


def _f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _check(got, ref, tol, what):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} values off, worst by {np.nanmax(np.abs(got - ref) / tol):.2f} of the bound"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,N,D,w,bias,silu,cache,strided,lens", [
    (2, 300, 64, 4, True, True, True, True, None),
    (1, 1, 4096, 4, True, True, True, True, None),          # one new token
    (3, 41, 8, 8, False, True, True, False, [41, 0, 5]),
    (2, 33, 5, 3, True, False, False, True, [1, 33]),       # rows off 16 bytes
    (2, 7, 1, 1, True, True, False, False, None),           # no history at all
    (4, 2, 24, 5, False, False, True, False, [2, 1, 0, 2]), # shorter than the history
    (1, 1000, 1023, 2, True, True, True, True, None),
    (130, 3, 16, 4, True, True, True, False, [i % 4 for i in range(130)]),   # more sequences than one launch takes
])
def test_conv(dtype, B, N, D, w, bias, silu, cache, strided, lens):
    g = torch.Generator().manual_seed(N * 31 + D)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = rand(B, N, 2 * D if strided else D).to(dtype)
    wt, bs = rand(D, w) / w ** 0.5, rand(D) if bias else None
    c0 = rand(B, w - 1, D).to(dtype) if cache else None
    n_of = lens or [N] * B
    xd = x.cuda()
    for b in range(B):
        xd[b, n_of[b]:] = float("nan")      # padding may hold anything
    out = torch.full((B, N, D), 7.0, dtype=dtype, device="cuda")
    y, c1 = la.la_ssm_conv(xd[..., D:] if strided else xd, wt.cuda(), None if bs is None else bs.cuda(),
                           None if c0 is None else c0.cuda(), silu=silu, seq_lens=lens, out=out)
    torch.cuda.synchronize()
    y, c1 = _f64(y), _f64(c1)
    x64 = _f64(x)[..., D:] if strided else _f64(x)
    for b in range(B):
        n = n_of[b]
        past = _f64(c0)[b] if cache else np.zeros((w - 1, D))
        ref, tol, kept = _conv_ref(x64[b, :n], _f64(wt), _f64(bs), past, silu, HALF[dtype])
        _check(y[b, :n], ref, tol, f"sequence {b}")
        assert (y[b, n:] == 7.0).all()       # padding rows stay as they were
        assert np.array_equal(c1[b], kept)   # copies of inputs


def test_conv_cache_in_place_and_continuation():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2, 77, 40, generator=g).to(torch.bfloat16).cuda()
    wt, c0 = torch.randn(40, 4, generator=g).cuda(), torch.randn(2, 3, 40, generator=g).to(torch.bfloat16).cuda()
    y_all, c_all = la.la_ssm_conv(x, wt, cache=c0)
    c = c0.clone()
    parts = []
    for t0, t1 in ((0, 50), (50, 51), (51, 53), (53, 77)):
        y, same = la.la_ssm_conv(x[:, t0:t1], wt, cache=c, cache_out=c)
        assert same is c
        parts.append(y)
    assert torch.equal(torch.cat(parts, 1), y_all) and torch.equal(c, c_all)
    # no tokens: the cache is passed on
    _, c2 = la.la_ssm_conv(x[:, :0], wt, cache=c0)
    assert torch.equal(c2, c0)


def _scan_ref(x, delta, A, Bm, Cm, D, z, bias, softplus, h0, r):
    """One sequence: y, bound on y, final state, bound on the state (float64)."""
    N, ch = x.shape
    n = A.shape[1]
    per = ch // Bm.shape[1]
    h = np.zeros((ch, n)) if h0 is None else h0.copy()
    E = np.zeros((ch, n))
    ys, tols = np.zeros((N, ch)), np.zeros((N, ch))
    for t in range(N):
        v = delta[t] + (0 if bias is None else bias)
        dt = np.logaddexp(v, 0) if softplus else v
        q = (2.0 ** -20 * (1 + np.abs(v)) if softplus else np.full(ch, 2 * U))[:, None]
        Bt, Ct = np.repeat(Bm[t], per, 0), np.repeat(Cm[t], per, 0)
        rate = dt[:, None] * A
        a = np.exp(rate)
        add = (dt * x[t])[:, None] * Bt
        E = a * E + np.abs(a * h) * (2.0 ** -22 + np.abs(rate) * (q + 3 * U) + U) + np.abs(add) * (q + 4 * U)
        h = a * h + add
        E = E + U * np.abs(h)
        y = (Ct * h).sum(-1)
        err = (np.abs(Ct) * E).sum(-1) + (n + 4) * U * np.abs(Ct * h).sum(-1)
        if D is not None:
            y = y + D * x[t]
            err = err + 2 * U * np.abs(D * x[t])
        if z is not None:
            s = _silu(z[t])
            y, err = y * s, err * np.abs(s) + 2.0 ** -19 * np.abs(y * s)
        ys[t], tols[t] = y, 1.01 * err + r * np.abs(y) + 1e-37
    return ys, tols, h, 1.01 * E + 1e-37


def _scan_inputs(dtype, B, N, ch, n, G, softplus, skip, gate, start, strided, seed, rows=True):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    lead = (B, N) if rows else (B,)
    wide = 2 * ch + 1 if strided else ch
    x = rand(*lead, wide).to(dtype)
    z = rand(*lead, wide).to(dtype) if gate else None
    delta = (rand(*lead, wide) if softplus else 0.05 * rand(*lead, wide).abs()).to(dtype)
    bc = rand(*lead, 2 * G * n + (3 if strided else 0)).to(dtype)
    part = lambda t: None if t is None else t[..., wide - ch:]  # noqa: E731
    p = dict(x=part(x), delta=part(delta), z=part(z),
             B=bc[..., :G * n].unflatten(-1, (G, n)), C=bc[..., G * n:2 * G * n].unflatten(-1, (G, n)),
             A=-torch.rand(ch, n, generator=g) * 4 - 0.01, D=rand(ch) if skip else None,
             delta_bias=rand(ch) - 3 if softplus else None)
    p["h"] = rand(B, ch, n) if start else None
    return p


def _view_cuda(t):
    """The same view of a copy of the whole underlying tensor on the GPU."""
    if t is None:
        return None
    base = t if t._base is None else t._base
    return base.cuda().as_strided(t.size(), t.stride(), t.storage_offset())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,N,ch,n,G,softplus,skip,gate,start,strided,lens", [
    (2, 70, 64, 16, 1, True, True, True, True, False, None),
    (1, 1, 33, 16, 1, True, True, True, False, True, None),
    (3, 65, 96, 8, 3, True, False, True, True, False, [65, 0, 32]),
    (2, 40, 10, 5, 2, False, True, False, False, True, [7, 40]),     # odd states, groups off every boundary
    (1, 96, 1, 1, 1, True, False, False, True, False, None),
    (2, 33, 40, 32, 1, True, True, True, True, True, None),
    (1, 64, 36, 64, 1, False, True, True, False, False, None),
    (1, 50, 34, 47, 1, True, True, True, True, False, None),
    (1, 1500, 32, 16, 1, True, True, True, True, False, None),       # several segments
    (2, 2100, 16, 4, 1, True, True, True, False, True, [2100, 700]), # segments past a sequence's end
    (131, 2, 4, 2, 1, False, False, True, True, False, [i % 3 for i in range(131)]),
])
def test_scan(dtype, B, N, ch, n, G, softplus, skip, gate, start, strided, lens):
    p = _scan_inputs(dtype, B, N, ch, n, G, softplus, skip, gate, start, strided, seed=N + ch)
    n_of = lens or [N] * B
    d = {k: _view_cuda(v) for k, v in p.items()}
    for b in range(B):
        for k in ("x", "delta", "z", "B", "C"):
            if d[k] is not None:
                d[k][b, n_of[b]:] = float("nan")
    out = torch.full((B, N, ch), 7.0, dtype=dtype, device="cuda")
    y, h = la.la_ssm_scan(d["x"], d["delta"], d["A"], d["B"], d["C"], D=d["D"], z=d["z"], delta_bias=d["delta_bias"],
                          delta_softplus=softplus, h0=d["h"], seq_lens=lens, out=out)
    torch.cuda.synchronize()
    y, h = _f64(y), _f64(h)
    q = {k: _f64(v) for k, v in p.items()}
    for b in range(B):
        m = n_of[b]
        at = lambda k: None if q[k] is None else q[k][b, :m]  # noqa: E731
        ry, ty, rh, th = _scan_ref(at("x"), at("delta"), q["A"], at("B"), at("C"), q["D"], at("z"), q["delta_bias"],
                                   softplus, None if q["h"] is None else q["h"][b], HALF[dtype])
        _check(h[b], rh, th, f"state of sequence {b}")
        _check(y[b, :m], ry, ty, f"sequence {b}")
        assert (y[b, m:] == 7.0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,ch,n,G,softplus,skip,gate,strided", [
    (3, 64, 16, 1, True, True, True, False),
    (2, 33, 4, 1, True, False, True, True),
    (1, 1, 1, 1, False, False, False, False),
    (5, 40, 8, 2, True, True, False, True),
    (2, 35, 32, 1, True, True, True, False),
    (2, 70, 64, 1, False, True, True, True),
    (3, 31, 5, 1, True, True, True, False),
    (2, 66, 47, 3, True, True, True, True),
    (2, 34, 10, 2, True, True, True, True),
    (2, 34, 18, 1, True, True, True, True),
    (2, 9, 12, 1, True, True, True, True),
])
def test_step(dtype, B, ch, n, G, softplus, skip, gate, strided):
    p = _scan_inputs(dtype, B, 1, ch, n, G, softplus, skip, gate, True, strided, seed=ch + n, rows=False)
    d = {k: _view_cuda(v) for k, v in p.items()}
    y = la.la_ssm_step(d["x"], d["delta"], d["A"], d["B"], d["C"], d["h"], D=d["D"], z=d["z"],
                       delta_bias=d["delta_bias"], delta_softplus=softplus)
    torch.cuda.synchronize()
    y, h = _f64(y), _f64(d["h"])
    q = {k: _f64(v) for k, v in p.items()}
    for b in range(B):
        at = lambda k: None if q[k] is None else q[k][b:b + 1]  # noqa: E731
        ry, ty, rh, th = _scan_ref(at("x"), at("delta"), q["A"], at("B"), at("C"), q["D"], at("z"), q["delta_bias"],
                                   softplus, q["h"][b], HALF[dtype])
        _check(h[b], rh, th, f"state of sequence {b}")
        _check(y[b:b + 1], ry, ty, f"sequence {b}")


def test_refusals():
    dev = dict(device="cuda", dtype=torch.bfloat16)
    x, w = torch.zeros(2, 8, 16, **dev), torch.zeros(16, 4, device="cuda")
    c = torch.zeros(2, 3, 16, **dev)
    with pytest.raises(ValueError):
        la.la_ssm_conv(x, w, cache=c[:, :2])
    with pytest.raises(ValueError):
        la.la_ssm_conv(x.transpose(1, 2), w)
    with pytest.raises(ValueError, match="seq_lens"):
        la.la_ssm_conv(x, w, seq_lens=[8])
    with pytest.raises(la.LaError) as e:
        la.la_ssm_conv(x, w, seq_lens=[8, 9])
    assert e.value.code == la.LA_ERR_INVALID
    with pytest.raises(la.LaError):                       # more than eight taps
        la.la_ssm_conv(x, torch.zeros(16, 9, device="cuda"))
    with pytest.raises(ValueError):
        la.la_ssm_conv(x.cpu(), w)
    A, bc = -torch.ones(16, 4, device="cuda"), torch.zeros(2, 8, 4, **dev)
    with pytest.raises(TypeError):
        la.la_ssm_scan(*(t.half() for t in (x, x)), A, bc.half(), bc.half())
    with pytest.raises(ValueError):
        la.la_ssm_scan(x, x[:, :7], A, bc, bc)
    with pytest.raises(ValueError):
        la.la_ssm_scan(x, x, A, bc, bc.float())
    with pytest.raises(ValueError):
        la.la_ssm_scan(x, x, A, torch.zeros(2, 8, 3, 4, **dev), torch.zeros(2, 8, 3, 4, **dev))   # 3 groups of 16
    h = torch.zeros(2, 16, 4, device="cuda")
    with pytest.raises(la.LaError) as e:
        la.la_ssm_scan(x, x, A, bc, bc, h0=h, h_out=h)
    assert e.value.code == la.LA_ERR_INVALID
    big = torch.zeros(2, 8, 65, **dev)
    with pytest.raises(la.LaError) as e:
        la.la_ssm_scan(x, x, -torch.ones(16, 65, device="cuda"), big, big)
    assert e.value.code == la.LA_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        la.la_ssm_step(x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0], h.bfloat16())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [16, 61])
def test_scan_rows_of_any_alignment(dtype, n):
    """How rows reach the kernel does not change a bit: whole 16-byte rows, rows on
    4 bytes and rows on one element, over more tiles than a kernel holds at once."""
    N, ch, lens = 700, 1921, [700, 413]
    p = _scan_inputs(dtype, 2, N, ch, n, 1, True, True, True, True, False, seed=3)
    assert la.la_ssm_scan_workspace_bytes(2, N, ch, 1, n) == 0
    fixed = {k: p[k].cuda() for k in ("A", "D", "delta_bias")}

    def rows(t, width, first):
        base = torch.full((*t.shape[:2], width), float("nan"), dtype=dtype, device="cuda")
        base[..., first:first + t.shape[-1]] = t.cuda()
        return base[..., first:first + t.shape[-1]]
    got = []
    for width, first in ((1928, 0), (1930, 2), (1927, 3)):
        x, delta, z = (rows(p[k], width, first) for k in ("x", "delta", "z"))
        B, C = (rows(p[k].flatten(2), width % 8 + 64, first) for k in ("B", "C"))
        got.append(la.la_ssm_scan(x, delta, B=B, C=C, z=z, h0=p["h"].cuda(), delta_softplus=True, seq_lens=lens, **fixed))
    for y, h in got[1:]:
        assert all(torch.equal(y[b, :t], got[0][0][b, :t]) for b, t in enumerate(lens))
        assert torch.equal(h, got[0][1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,N,ch,n,G,lens", [
    (2, 1500, 64, 16, 2, [1500, 700]),     # several segments
    (1, 300, 1921, 5, 1, None),            # rows off 4 bytes
    (1, 200, 2048, 16, 1, None),
])
def test_out_in_an_inputs_place(dtype, B, N, ch, n, G, lens):
    """out may be x, delta or z itself: the bits of an out of its own, for prompts and tokens."""
    p = {k: _view_cuda(v) for k, v in _scan_inputs(dtype, B, N, ch, n, G, True, True, True, True, False, seed=N).items()}
    assert (la.la_ssm_scan_workspace_bytes(B, N, ch, G, n) > 0) == (N == 1500)

    def scan(out, q):
        return la.la_ssm_scan(q["x"], q["delta"], q["A"], q["B"], q["C"], D=q["D"], z=q["z"], delta_bias=q["delta_bias"],
                              delta_softplus=True, h0=q["h"], seq_lens=lens, out=out)

    def step(out, q):
        h = q["h"].clone()
        return la.la_ssm_step(*(q[k][:, 0] if k != "A" else q[k] for k in ("x", "delta", "A", "B", "C")), h, D=q["D"],
                              z=q["z"][:, 0], delta_bias=q["delta_bias"], delta_softplus=True, out=out), h
    want = scan(torch.zeros(B, N, ch, dtype=dtype, device="cuda"), p)
    want1 = step(torch.zeros(B, ch, dtype=dtype, device="cuda"), p)
    for name in ("x", "delta", "z"):
        q = {**p, name: p[name].clone()}
        y, h = scan(q[name], q)
        for b in range(B):
            m = N if lens is None else lens[b]
            assert torch.equal(y[b, :m], want[0][b, :m]) and torch.equal(y[b, m:], p[name][b, m:])
        assert y is q[name] and torch.equal(h, want[1])
        q = {**p, name: p[name][:, :1].clone()}
        got = step(q[name][:, 0], q)
        assert torch.equal(got[0], want1[0]) and torch.equal(got[1], want1[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_conv_outputs_between_the_rows_of_x(dtype):
    """One buffer of a sequence's rows, the output of the sequence, its cache: the bits of buffers of their own."""
    B, N, D, w = 1, 50, 24, 4
    g = torch.Generator().manual_seed(4)
    wt = torch.randn(D, w, generator=g).cuda()
    base = torch.randn(2 * N * D + 3 * D + N, generator=g).to(dtype).cuda()
    x = base[:N * D].view(1, N, D)
    out, cache = base[N * D:2 * N * D].view(1, N, D), base[2 * N * D:2 * N * D + 3 * D].view(1, 3, D)
    keep, want = base.clone(), la.la_ssm_conv(x.clone(), wt, cache=cache.clone())
    la.la_ssm_conv(x, wt, cache=cache, out=out, cache_out=cache)
    assert torch.equal(out, want[0]) and torch.equal(cache, want[1]) and torch.equal(x, keep[:N * D].view(1, N, D))
    # two sequences far apart, out in the gap behind the first one
    far = torch.randn(2, 2 * (N * D) + 8 * D, generator=g).to(dtype).cuda()
    x = far[:, :N * D].view(2, N, D)
    gap = far.view(-1)[N * D:N * D + 2 * 10 * D].view(2, 10, D)
    want = la.la_ssm_conv(x[:, 3:13].clone(), wt)
    got = la.la_ssm_conv(x[:, 3:13], wt, out=gap)
    assert torch.equal(got[0], want[0])
    with pytest.raises(la.LaError) as e:
        la.la_ssm_conv(x, wt, out=far.view(-1)[:2 * N * D].view(2, N, D))
    assert e.value.code == la.LA_ERR_INVALID


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,N,ch,lens", [(2, 40, 32, [40, 7]), (1, 1500, 32, None)])     # one segment, several
def test_scan_of_states_that_keep_nothing(dtype, B, N, ch, lens):
    """A rate of minus infinity decays by 0, as any rate does whose decay is below the smallest number:
    the same bits, also where a sequence ends inside a tile."""
    p = {k: _view_cuda(v) for k, v in _scan_inputs(dtype, B, N, ch, 6, 1, True, True, True, True, False, seed=8).items()}
    got = []
    for rate in (-float("inf"), -1e30):
        A = p["A"].clone()
        A[::3, 1:4] = rate
        got.append(la.la_ssm_scan(p["x"], p["delta"], A, p["B"], p["C"], D=p["D"], z=p["z"], delta_bias=p["delta_bias"],
                                  delta_softplus=True, h0=p["h"], seq_lens=lens))
    (y0, h0), (y1, h1) = got
    assert torch.isfinite(h1).all() and torch.equal(h0, h1)
    assert all(torch.equal(y0[b, :n], y1[b, :n]) for b, n in enumerate(lens or [N] * B))
