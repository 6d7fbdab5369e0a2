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
