"""The state-space and sliding-window kernels at sizes where their launch rules
choose what serves large calls: runs of tokens longer than a thread's ring of
copies, several sequences a thread, many (sequence, kv head) units of one token.
Against the definitions in float64 on the GPU, element by element, with the
bounds that tests/test_ssm_gpu.py and tests/test_window_gpu.py derive; and rows
that several heads or sequences share."""
import pytest
import torch

import causal_kernelized_linear_la_b200 as la

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
DTYPES = [torch.bfloat16, torch.float32]


def _check(got, ref, tol, what):
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} values off, first at {bad.nonzero()[0].tolist()}"


def _conv_ref(x, w, bias, cache, r):
    """One sequence [N, D]: (y, bound, new cache) of a convolution with SiLU, in float64."""
    W, N = w.shape[1], x.shape[0]
    xh = torch.cat([cache, x]).double()
    y, mag = bias.double().expand(N, -1).clone(), bias.double().abs().expand(N, -1).clone()
    for i in range(W):
        term = w[:, i].double() * xh[i:i + N]
        y += term
        mag += term.abs()
    err = (W + 1) * U * mag
    y = y * torch.sigmoid(y)
    err = 1.1 * err + 2.0 ** -19 * y.abs()
    return y, 1.01 * err + r * y.abs() + 1e-37, torch.cat([cache, x])[N:]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,N,D,w,lens", [
    (1, 20011, 4096, 4, None),               # runs of 128 tokens, the last one short
    (2, 10007, 4096, 8, [10007, 5003]),      # a sequence that ends inside a run
    (1, 4999, 4096, 5, None),                # runs of 32
    (1, 9999, 4096, 1, None),                # no history; runs of 64
    (1, 20011, 1023, 3, None),               # one channel a thread
    (2, 20011, 519, 8, [77, 20011]),
])
def test_conv_long_runs(dtype, B, N, D, w, lens):
    g = torch.Generator(device="cuda").manual_seed(N + D + w)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, wt, bias, c0 = r(B, N, D).to(dtype), r(D, w) / w ** 0.5, r(D), r(B, w - 1, D).to(dtype)
    n_of = lens or [N] * B
    xd, cache = x.clone(), c0.clone()
    for b in range(B):
        xd[b, n_of[b]:] = float("nan")
    out = torch.full_like(x, 7.0)
    la.la_ssm_conv(xd, wt, bias, cache, seq_lens=lens, out=out, cache_out=cache)
    for b, n in enumerate(n_of):
        ref, tol, kept = _conv_ref(x[b, :n], wt, bias, c0[b], HALF[dtype])
        _check(out[b, :n], ref, tol, f"sequence {b}")
        assert (out[b, n:] == 7.0).all() and torch.equal(cache[b], kept)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,D,w,lens", [
    (257, 4096, 4, None),                                     # four sequences a thread, one left over
    (259, 4096, 8, None),
    (127, 4096, 4, [int(i % 3 > 0) for i in range(127)]),     # some without a token
    (259, 4096, 3, [int(i % 4 > 0) for i in range(259)]),     # two launches of 128 and one of 3
    (130, 1023, 5, None),                                     # one channel a thread
    (301, 1023, 1, None),
])
def test_conv_tokens_of_many_sequences(dtype, B, D, w, lens):
    g = torch.Generator(device="cuda").manual_seed(B + D + w)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, wt, bias, c0 = r(B, 1, 2 * D).to(dtype)[..., D:], r(D, w) / w ** 0.5, r(D), r(B, w - 1, D).to(dtype)
    out, cache = torch.full((B, 1, D), 7.0, dtype=dtype, device="cuda"), c0.clone()
    la.la_ssm_conv(x, wt, bias, cache, seq_lens=lens, out=out, cache_out=cache)
    # w rows a sequence: each is a sequence's only token
    xh = torch.cat([c0, x], 1).double()
    mag = (wt.double().T * xh).abs().sum(1) + bias.double().abs()
    y = (wt.double().T * xh).sum(1) + bias.double()
    y = y * torch.sigmoid(y)
    tol = 1.01 * (1.1 * (w + 1) * U * mag + 2.0 ** -19 * y.abs()) + HALF[dtype] * y.abs() + 1e-37
    on = torch.tensor(lens or [1] * B, device="cuda").bool()
    _check(out[on, 0], y[on], tol[on], "tokens")
    assert (out[~on] == 7.0).all()
    kept = torch.where(on[:, None, None], torch.cat([c0, x], 1)[:, 1:], c0)
    assert torch.equal(cache, kept)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,Hq,Hkv,d,dv,window,sinks", [
    (80, 16, 8, 64, 128, 97, 3),         # 640 units: a CTA each
    (40, 32, 8, 128, 128, 700, 5),       # 320 units: two CTAs each
    (40, 16, 8, 128, 64, 2099, 1),       # four CTAs each
    (13, 80, 8, 64, 64, 600, 0),         # ten heads a kv head: a full and a short chunk of heads
    (20, 8, 8, 64, 64, 1000, 7),         # 160 units: eight warps a CTA
    (50, 4, 2, 128, 128, 1201, 2),       # 100 units, two CTAs each
    (3, 32, 8, 128, 128, 5000, 4),       # few units: a cluster of eight
])
def test_decode_of_many_sequences(dtype, B, Hq, Hkv, d, dv, window, sinks):
    cap, group = window + sinks, Hq // Hkv
    g = torch.Generator(device="cuda").manual_seed(B + window)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    q, k, v, kc, vc = r(B, Hq, d) * 2, r(B, Hkv, d), r(B, Hkv, dv), r(B, Hkv, cap, d), r(B, Hkv, cap, dv)
    pos = [0, cap - 1, cap, 3 * cap + 11, sinks, window // 2, cap - 2, 15, 16, 1 << 30]
    pos = [-1 if b == 1 else pos[b % len(pos)] if b < 20 else (b * 7919) % (2 * cap) for b in range(B)]
    for b, p in enumerate(pos):
        kc[b, :, max(p, 0):], vc[b, :, max(p, 0):] = float("nan"), float("nan")    # slots not filled yet
    want_k, want_v = kc.clone(), vc.clone()
    out = torch.full((B, Hq, dv), 7.0, dtype=dtype, device="cuda")
    la.la_window_decode_step(q, k, v, kc, vc, torch.tensor(pos, dtype=torch.int32, device="cuda"), window, sinks=sinks,
                             out=out)
    la.la_prefill_check()
    for b, p in enumerate(pos):
        if p < 0:
            assert (out[b] == 7.0).all()
            continue
        slot = p if p < sinks else sinks + (p - sinks) % window
        want_k[b, :, slot], want_v[b, :, slot] = k[b], v[b]
        used = min(p + 1, cap)
        K, V = (t[b, :, :used].double().repeat_interleave(group, 0) for t in (want_k, want_v))
        Q, scale = q[b].double()[:, None], d ** -0.5
        s = (Q @ K.mT)[:, 0] * scale
        e = (d + 4) * U * scale * (Q.abs() @ K.abs().mT)[:, 0].amax(1, keepdim=True)
        x = s - s.amax(1, keepdim=True)
        w = torch.softmax(s, 1)
        rel = 2 * (e - x.amin(1, keepdim=True) * 1.4427 * 2.0 ** -23 + 2.0 ** -21) + (used + 4) * U
        if dtype == torch.bfloat16:
            rel = rel + 2 * 2.0 ** -12 + 2.0 ** -8
        ref = (w[:, None] @ V)[:, 0]
        _check(out[b], ref, (w[:, None] @ V.abs())[:, 0] * rel + HALF[dtype] * ref.abs() + 1e-37, f"sequence {b} at {p}")
    same = lambda x, y: torch.equal(x.view(torch.uint8), y.view(torch.uint8))  # noqa: E731
    assert same(kc, want_k) and same(vc, want_v)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("share", ["heads of q", "heads of k", "heads of v", "sequences of q", "sequences of k and v", "all"])
def test_rows_shared_by_heads_and_sequences(dtype, share):
    """Expanded q, k or v (stride 0): the bits of a copy with rows for every head and sequence."""
    B, Hq, Hkv, N, d, dv, window, sinks = 3, 4, 2, 300, 64, 128, 90, 2
    g = torch.Generator(device="cuda").manual_seed(len(share))
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731

    def make(name, H, cols):
        one_head = share == "all" or share == f"heads of {name}"
        one_batch = share == "all" or (share.startswith("sequences") and name in share.split("of ")[1].split(" and "))
        return r(1 if one_batch else B, 1 if one_head else H, N, cols).expand(B, H, N, cols)
    q, k, v = make("q", Hq, d), make("k", Hkv, d), make("v", Hkv, dv)
    assert any(0 in t.stride() for t in (q, k, v))
    kc, vc = r(B, Hkv, window + sinks, d), r(B, Hkv, window + sinks, dv)
    pos = torch.tensor([0, 50, 1000], dtype=torch.int32, device="cuda")
    lens = [300, 290, 1]
    got, want = [], []
    for out, (a, b, c) in ((got, (q, k, v)), (want, (q.contiguous(), k.contiguous(), v.contiguous()))):
        kc1, vc1 = kc.clone(), vc.clone()
        o = torch.full((B, Hq, N, dv), 7.0, dtype=dtype, device="cuda")
        out += [la.la_window_prefill(a, b, c, window, sinks=sinks),
                la.la_window_prefill(a, b, c, window, sinks=sinks, k_cache=kc1, v_cache=vc1, pos=pos, seq_lens=lens, out=o),
                kc1, vc1]
        kc2, vc2 = kc.clone(), vc.clone()
        out += [la.la_window_decode_step(a[:, :, 7], b[:, :, 7], c[:, :, 7], kc2, vc2, pos, window, sinks=sinks), kc2, vc2]
    la.la_prefill_check()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("dtype", DTYPES)
def test_state_space_rows_shared_by_sequences_and_tokens(dtype):
    """Expanded inputs (stride 0 over sequences or tokens): the bits of copies."""
    B, N, ch, n, G, w = 3, 70, 48, 6, 2, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, delta, z = r(1, N, ch).expand(B, N, ch), r(B, 1, ch).expand(B, N, ch), r(1, 1, ch).expand(B, N, ch)
    Bm, Cm = r(1, N, G, n).expand(B, N, G, n), r(B, 1, G, n).expand(B, N, G, n)
    A, D, bias = -torch.rand(ch, n, device="cuda") - 0.1, torch.randn(ch, device="cuda"), torch.randn(ch, device="cuda") - 2
    wt, lens = torch.randn(ch, w, device="cuda"), [70, 3, 41]
    got, want = [], []
    for out, f in ((got, lambda t: t), (want, lambda t: t.contiguous())):
        y = torch.full((B, N, ch), 7.0, dtype=dtype, device="cuda")
        out += la.la_ssm_scan(f(x), f(delta), A, f(Bm), f(Cm), D=D, z=f(z), delta_bias=bias, delta_softplus=True,
                              seq_lens=lens, out=y)
        h = torch.ones(B, ch, n, device="cuda")
        out += [la.la_ssm_step(f(x)[:, 5], f(delta)[:, 5], A, f(Bm)[:, 5], f(Cm)[:, 5], h, D=D, z=f(z)[:, 5],
                               delta_bias=bias, delta_softplus=True), h]
        y = torch.full((B, N, ch), 7.0, dtype=dtype, device="cuda")
        out += la.la_ssm_conv(f(x), wt, seq_lens=lens, out=y)
        out += la.la_ssm_conv(f(delta), wt)
        out += la.la_ssm_conv(f(z)[:, :1], wt)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", DTYPES)
def test_more_sequences_than_a_grid_holds(dtype):
    """32768 sequences go in one launch: what the first and the last ones get is what they get alone."""
    B, N, ch, n, d, window = 32768 + 5, 3, 8, 4, 64, 2
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, delta, bc = r(B, N, ch), r(B, N, ch).abs(), r(B, N, n)
    A, h0, wt = -torch.rand(ch, n, device="cuda"), torch.randn(B, ch, n, device="cuda"), torch.randn(ch, 4, device="cuda")
    q, k, v, kc, vc = r(B, 1, N, d), r(B, 1, N, d), r(B, 1, N, d), r(B, 1, window, d), r(B, 1, window, d)
    pos = torch.arange(B, dtype=torch.int32, device="cuda") % 5

    def run(s):
        k1, v1, k2, v2, h = kc[s].clone(), vc[s].clone(), kc[s].clone(), vc[s].clone(), h0[s].clone()
        return [*la.la_ssm_conv(x[s], wt), *la.la_ssm_scan(x[s], delta[s], A, bc[s], bc[s], h0=h0[s]),
                la.la_ssm_step(x[s, 0], delta[s, 0], A, bc[s, 0], bc[s, 0], h), h,
                la.la_window_prefill(q[s], k[s], v[s], window, k_cache=k1, v_cache=v1, pos=pos[s]), k1, v1,
                la.la_window_decode_step(q[s, :, 0], k[s, :, 0], v[s, :, 0], k2, v2, pos[s], window), k2, v2]
    whole = run(slice(0, B))
    for s in (slice(0, 7), slice(B - 9, B)):
        assert all(torch.equal(a[s], b) for a, b in zip(whole, run(s)))
    la.la_prefill_check()


def test_offsets_past_32_bits():
    """More than 2^31 elements in x, and in a cache: the last rows, and the first, are the right ones."""
    N, D = (1 << 31) // 4096 + 300, 4096
    x = torch.empty(1, N, D, dtype=torch.bfloat16, device="cuda").normal_()
    wt, bias = torch.randn(D, 4, device="cuda"), torch.randn(D, device="cuda")
    out, cache = la.la_ssm_conv(x, wt, bias)
    for t0, t1 in ((0, 50), (N - 700, N)):
        before = torch.zeros(3, D, dtype=x.dtype, device="cuda") if t0 == 0 else x[0, t0 - 3:t0]
        ref, tol, kept = _conv_ref(x[0, t0:t1], wt, bias, before, HALF[x.dtype])
        _check(out[0, t0:t1], ref, tol, f"tokens from {t0}")
    assert torch.equal(cache[0], kept)
    n, ch = 16, 4096
    bc = torch.randn(1, N, n, device="cuda").bfloat16()
    A = -torch.ones(ch, n, device="cuda") * 40                # a state that forgets within a few tokens
    y, h = la.la_ssm_scan(x, x.abs_(), A, bc, bc, delta_bias=torch.ones(ch, device="cuda"), out=out)
    tail = la.la_ssm_scan(x[:, N - 64:], x[:, N - 64:], A, bc[:, N - 64:], bc[:, N - 64:],
                          delta_bias=torch.ones(ch, device="cuda"))
    assert torch.equal(y[:, N - 32:], tail[0][:, 32:]) and torch.equal(h, tail[1])     # exp(-40 * 32) = 0
    del x, out, y
    torch.cuda.empty_cache()
    d, cap = 128, (1 << 31) // 128 + 1000
    kc = torch.zeros(1, 1, cap, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc).normal_()
    q = torch.zeros(1, 1, 1, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 8.0
    far = torch.tensor([cap + 12345], dtype=torch.int32, device="cuda")       # the new token lands in a slot below
    slot = (cap + 12345) % cap
    for at in (0, cap // 2, cap - 700, cap - 1):
        kc[0, 0, at, 0] = 200.0               # the score that outweighs 2^24 others: 8 * 200 * d^-0.5 = 141
        got = la.la_window_decode_step(q[:, :, 0], q[:, :, 0] * 0, q[:, :, 0], kc, vc, far, cap)
        assert torch.equal(got[0, 0], vc[0, 0, at]), at
        if at == cap - 1:
            got = la.la_window_prefill(q, q * 0, q, cap, k_cache=kc, v_cache=vc, pos=far)
            assert torch.equal(got[0, 0, 0], vc[0, 0, at])
        kc[0, 0, at, 0] = 0.0
    assert torch.equal(vc[0, 0, slot], q[0, 0, 0]) and not kc[0, 0, slot].any()
    la.la_prefill_check()
