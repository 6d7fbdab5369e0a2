"""The state-space and sliding-window entry points as a server runs them: a
layer's convolution, prompt scan and token steps in a row; captured into CUDA
graphs and replayed; on another stream; the same bits on every call; causality
under hostile futures; one profiling event a kernel."""
import numpy as np
import pytest
import torch

import causal_kernelized_linear_la_b200 as la

from tests.test_ssm_gpu import HALF, _check, _f64, _scan_ref

pytestmark = pytest.mark.gpu


def _layer(dtype, B, N, ch, n, seed=0):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    xz = rand(B, N, 2 * ch).to(dtype).cuda()
    p = dict(x=xz[..., :ch], z=xz[..., ch:], delta=(rand(B, N, ch) * 0.5).to(dtype).cuda(),
             bc=rand(B, N, 2 * n).to(dtype).cuda(), w=rand(ch, 4).cuda() / 2, wb=rand(ch).cuda() / 4,
             A=-torch.rand(ch, n, generator=g).cuda() * 4 - 0.01, D=rand(ch).cuda(), db=rand(ch).cuda() - 3)
    return p


def _scan_kw(p):
    return dict(D=p["D"], delta_bias=p["db"], delta_softplus=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_layer_prompt_in_pieces_then_tokens(dtype):
    """Pieces of a prompt, then single tokens, with the cache and the state
    carried on: every y within the recurrence's bound over the whole sequence,
    whose input is what the convolution returned."""
    B, ch, n, pieces, steps = 2, 48, 16, (70, 1, 33), 6
    N = sum(pieces) + steps
    p = _layer(dtype, B, N, ch, n)
    cache = torch.zeros(B, 3, ch, dtype=dtype, device="cuda")
    h, t, us, ys = torch.zeros(B, ch, n, device="cuda"), 0, [], []
    for k in pieces:
        s = slice(t, t + k)
        u, _ = la.la_ssm_conv(p["x"][:, s], p["w"], bias=p["wb"], cache=cache, cache_out=cache)
        y, h = la.la_ssm_scan(u, p["delta"][:, s], p["A"], p["bc"][:, s, :n], p["bc"][:, s, n:], z=p["z"][:, s], h0=h,
                              **_scan_kw(p))
        us.append(u)
        ys.append(y)
        t += k
    for _ in range(steps):
        u, _ = la.la_ssm_conv(p["x"][:, t:t + 1], p["w"], bias=p["wb"], cache=cache, cache_out=cache)
        y = la.la_ssm_step(u[:, 0], p["delta"][:, t], p["A"], p["bc"][:, t, :n], p["bc"][:, t, n:], h, z=p["z"][:, t],
                           **_scan_kw(p))
        us.append(u)
        ys.append(y[:, None])
        t += 1
    torch.cuda.synchronize()
    u_all, y_all = torch.cat(us, 1), torch.cat(ys, 1)
    # the convolution in pieces is the convolution of the whole: the same sums in the same order
    whole, last = la.la_ssm_conv(p["x"], p["w"], bias=p["wb"])
    assert torch.equal(u_all, whole) and torch.equal(last, cache)
    for b in range(B):
        ref, tol, rh, th = _scan_ref(_f64(u_all[b]), _f64(p["delta"][b]), _f64(p["A"]), _f64(p["bc"][b, :, None, :n]),
                                     _f64(p["bc"][b, :, None, n:]), _f64(p["D"]), _f64(p["z"][b]), _f64(p["db"]), True,
                                     None, HALF[dtype])
        _check(_f64(y_all[b]), ref, tol, f"sequence {b}")
        _check(_f64(h[b]), rh, th, f"state {b}")


def _calls(dtype):
    """name -> (call into fixed buffers, the buffers it writes)"""
    B, N, ch, n, d, W, S = 2, 1500, 64, 16, 64, 100, 4
    p = _layer(dtype, B, N, ch, n, seed=5)
    g = torch.Generator().manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    q, k, v = r(B, 4, N, d), r(B, 2, N, d), r(B, 2, N, d)
    kc0, vc0 = r(B, 2, W + S, d), r(B, 2, W + S, d)
    kc, vc = kc0.clone(), vc0.clone()
    pos = torch.tensor([300, 7], dtype=torch.int32, device="cuda")
    e = lambda *s, dt=dtype: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    u, c1, y, h1 = e(B, N, ch), e(B, 3, ch), e(B, N, ch), e(B, ch, n, dt=torch.float32)
    ws = torch.empty(max(16, la.la_ssm_scan_workspace_bytes(B, N, ch, 1, n)), dtype=torch.uint8, device="cuda")
    assert la.la_ssm_scan_workspace_bytes(B, N, ch, 1, n) > 0       # the segmented form
    h2, y2, o, o2 = e(B, ch, n, dt=torch.float32), e(B, ch), e(B, 4, N, d), e(B, 4, d)

    def scan(stream=None):
        la.la_ssm_scan(p["x"], p["delta"], p["A"], p["bc"][..., :n], p["bc"][..., n:], z=p["z"], out=y, h_out=h1,
                       workspace=ws, stream=stream, **_scan_kw(p))

    def step(stream=None):
        la.la_ssm_step(p["x"][:, 3], p["delta"][:, 3], p["A"], p["bc"][:, 3, :n], p["bc"][:, 3, n:], h2, z=p["z"][:, 3],
                       out=y2, stream=stream, **_scan_kw(p))

    def window(stream=None):
        la.la_window_prefill(q, k, v, W, sinks=S, k_cache=kc, v_cache=vc, pos=pos, out=o, stream=stream)

    def decode(stream=None):
        la.la_window_decode_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], kc, vc, pos, W, sinks=S, out=o2, stream=stream)

    def reset():
        h2.fill_(0.25)
        kc.copy_(kc0)
        vc.copy_(vc0)

    return {
        "conv": (lambda stream=None: la.la_ssm_conv(p["x"], p["w"], bias=p["wb"], out=u, cache_out=c1, stream=stream), [u, c1]),
        "scan": (scan, [y, h1]), "step": (step, [y2, h2]), "window": (window, [o, kc, vc]), "decode": (decode, [o2, kc, vc]),
    }, reset, [p["x"], p["delta"], q, k]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", ["conv", "scan", "step", "window", "decode"])
def test_graph_stream_and_bits(name, dtype):
    calls, reset, inputs = _calls(dtype)
    call, bufs = calls[name]
    reset()
    call()
    torch.cuda.synchronize()
    ref = [t.clone() for t in bufs]
    for _ in range(3):                                  # the same bits on every call
        reset()
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, bufs))
    side = torch.cuda.Stream()                          # on a stream that is not the current one
    reset()
    bufs[0].zero_()
    torch.cuda.synchronize()
    call(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, bufs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    reset()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, bufs))
    for t in inputs:                                    # a replay reads the buffers' new contents
        t.copy_(t.flip(0))
    reset()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in bufs]
    reset()
    call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, bufs))
    assert not torch.equal(got[0], ref[0])
    la.la_prefill_check()


def test_outputs_made_on_the_given_stream():
    """Outputs that the binding allocates belong to the stream of the call."""
    calls, _, _ = _calls(torch.bfloat16)
    side = torch.cuda.Stream()
    q = torch.randn(1, 2, 300, 64, device="cuda").bfloat16()
    want = la.la_window_prefill(q, q, q, 50, sinks=2)
    x, w = torch.randn(2, 300, 64, device="cuda").bfloat16(), torch.randn(64, 4, device="cuda")
    want_u, _ = la.la_ssm_conv(x, w)
    torch.cuda.synchronize()
    for _ in range(20):
        junk = torch.full((1, 2, 300, 64), float("nan"), device="cuda", dtype=torch.bfloat16)
        del junk
        got = la.la_window_prefill(q, q, q, 50, sinks=2, stream=side)
        u, _ = la.la_ssm_conv(x, w, stream=side)
        junk = torch.full((1, 2, 300, 64), float("nan"), device="cuda", dtype=torch.bfloat16)
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(u, want_u)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_window_futures_do_not_matter(dtype):
    """Rows before a change of keys (to NaN and infinities, which they do not
    see) and values (finite) keep their bits, in and across tiles."""
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    q, k, v = r(1, 2, 500, 64), r(1, 2, 500, 64), r(1, 2, 500, 64)
    ref = la.la_window_prefill(q, k, v, 150, sinks=3)
    for cut in (1, 77, 128, 300, 499):
        k2, v2 = k.clone(), v.clone()
        k2[:, :, cut:] = float("nan")
        k2[:, :, cut + 1:] = float("inf")
        v2[:, :, cut:] = 1e30
        got = la.la_window_prefill(q, k2, v2, 150, sinks=3)
        assert torch.equal(got[:, :, :cut], ref[:, :, :cut]), cut
    # a token that has left the window and is no sink: likewise
    k2, v2 = k.clone(), v.clone()
    k2[:, :, 100:200], v2[:, :, 100:200] = float("nan"), -1e30
    got = la.la_window_prefill(q, k2, v2, 150, sinks=3)
    assert torch.equal(got[:, :, 349:], ref[:, :, 349:]) and torch.equal(got[:, :, :100], ref[:, :, :100])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scan_futures_do_not_matter(dtype):
    p = _layer(dtype, 1, 200, 40, 16, seed=3)
    run = lambda q: la.la_ssm_scan(q["x"], q["delta"], q["A"], q["bc"][..., :16], q["bc"][..., 16:], z=q["z"], **_scan_kw(q))[0]  # noqa: E731
    ref = run(p)
    for cut in (1, 31, 33, 150):
        q = {k: v.clone() for k, v in p.items()}
        for k in ("x", "delta", "z", "bc"):
            q[k][:, cut:] = float("nan")
        assert torch.equal(run(q)[:, :cut], ref[:, :cut]), cut


def test_large_and_extreme_values():
    """Scores far apart (a row dominated by one key), equal scores, a zero
    scale, and step sizes that forget everything."""
    q = torch.zeros(1, 1, 200, 64, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(1, 1, 200, 64, device="cuda").bfloat16()
    o = la.la_window_prefill(q, q, v, 200)                    # all weights equal: a running mean
    want = v.double().cumsum(2) / torch.arange(1, 201, device="cuda").double()[:, None]
    mag = v.double().abs().cumsum(2) / torch.arange(1, 201, device="cuda").double()[:, None]
    assert ((o.double() - want).abs() <= mag * 2.0 ** -8 + want.abs() * 2.0 ** -8).all()
    k = torch.randn(1, 1, 200, 64, device="cuda").bfloat16()
    assert torch.equal(la.la_window_prefill(k, k, v, 200, scale=0.0), o)
    big = (k.float() * 60).bfloat16()                         # scores of thousands: each query's best key wins
    o = la.la_window_prefill(big, big, v, 200)
    s = (big.double() @ big.double().transpose(-1, -2) / 8).masked_fill(
        torch.ones(200, 200, device="cuda").triu(1).bool(), float("-inf"))
    p = torch.softmax(s, -1)
    assert torch.isfinite(o.float()).all()
    # score errors of (d + 4) u sum |q k| scale move a weight by that many e-folds
    e = 68 * 2.0 ** -24 * (big.double().abs() @ big.double().abs().transpose(-1, -2) / 8).amax(-1, keepdim=True)
    tol = (p @ v.double().abs()) * (2 * e + 2.0 ** -7 + 2.0 ** -11) + 2.0 ** -8 * (p @ v.double()).abs()
    assert ((o.double() - p @ v.double()).abs() <= tol).all()
    x = torch.randn(1, 64, 8, device="cuda")
    bc = torch.randn(1, 64, 4, device="cuda")
    A = -torch.ones(8, 4, device="cuda")
    dt = torch.full_like(x, 200.0)                            # exp(-200) = 0 in fp32: y_t = dt x_t B.C
    y, h = la.la_ssm_scan(x, dt, A, bc, bc)
    want = 200.0 * x.double() * (bc.double() ** 2).sum(-1, keepdim=True)
    assert torch.allclose(y.double(), want, rtol=10 * 2.0 ** -24, atol=0)
    y, h = la.la_ssm_scan(x, torch.zeros_like(x), A, bc, bc)  # nothing is written
    assert (y == 0).all() and (h == 0).all()
    h0 = torch.randn(1, 8, 4, device="cuda")
    _, h = la.la_ssm_scan(x, torch.zeros_like(x), A, bc, bc, h0=h0)      # and nothing forgotten: every decay is 1
    assert torch.equal(h, h0)
    la.la_ssm_step(x[:, 0], torch.zeros_like(x[:, 0]), A, bc[:, 0], bc[:, 0], h)
    assert torch.equal(h, h0)


@pytest.mark.parametrize("segments", [False, True])
def test_slow_states_keep_their_precision(segments):
    """Decays near 1 over thousands of tokens: a bias of the exponential adds
    up token by token.  With u = 2^-24: a decay's mean error is at most 0.06 u
    for these exponents (between -0.0022 and 0 in log2 units), so N tokens shift
    the state by at most 0.06 N u; the scatter of decay, product and sum is at
    most 2 u a token and independent, so about 2 u sqrt(N) together.  At N =
    4096 that is (246 + 128) u of the state's norm; 8 u sqrt(N) = 512 u are allowed."""
    g = torch.Generator().manual_seed(1)
    ch, n, N = (32 if segments else 4096), 8, 4096
    assert (la.la_ssm_scan_workspace_bytes(1, N, ch, 1, n) > 0) == segments
    x = torch.randn(1, N, ch, generator=g).cuda()
    dt = (0.0005 + 0.001 * torch.rand(1, N, ch, generator=g)).cuda()
    bc = torch.randn(1, N, n, generator=g).cuda()
    A = -(0.2 + 0.8 * torch.rand(ch, n, generator=g)).cuda()
    h0 = torch.randn(1, ch, n, generator=g).cuda() * 10
    _, h = la.la_ssm_scan(x, dt, A, bc, bc, h0=h0)
    ref = h0.double()[0]
    for t in range(N):
        k = dt[0, t].double()[:, None]
        ref = torch.exp(k * A.double()) * ref + k * x[0, t].double()[:, None] * bc[0, t].double()
    err = ((h[0].double() - ref).norm() / ref.norm()).item()
    assert err <= 4 * 2 * 2.0 ** -24 * N ** 0.5, err


def test_one_event_a_kernel():
    calls, reset, _ = _calls(torch.bfloat16)
    events = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    for name, kernels in (("conv", 1), ("scan", 2), ("step", 1), ("window", 2), ("decode", 1)):
        reset()
        for e in events:
            e.record()
        torch.cuda.synchronize()
        start = torch.cuda.Event(enable_timing=True)
        la.la_set_stage_events(events)
        try:
            start.record()
            calls[name][0]()
        finally:
            la.la_set_stage_events(None)
        torch.cuda.synchronize()
        # events of kernels that ran lie behind the start, the others before it
        assert [start.elapsed_time(e) >= 0 for e in events] == [i < kernels for i in range(3)], name


def test_silu_in_fp32():
    """One tap of weight one: out = silu(x).  Steps of u = 2^-24: the SFU's 2^x 4
    (two places), its first-order correction and product 2, 1 + h 1, the
    reciprocal after its Newton step 1, two products 2: 10 u together."""
    x = torch.cat([torch.linspace(-80, 80, 200001), torch.logspace(-30, 0, 5000), -torch.logspace(-30, 0, 5000)])
    x = x[:x.numel() // 8 * 8].view(1, -1, 8).cuda()
    y, _ = la.la_ssm_conv(x, torch.ones(8, 1, device="cuda"))
    want = torch.nn.functional.silu(x.double())
    assert ((y.double() - want).abs() <= 10 * 2.0 ** -24 * want.abs()).all()
    far = torch.tensor([float("inf"), 1e30, -1e4, -120.0, 0.0, -0.0, float("nan"), 100.0], device="cuda").view(1, 1, 8)
    y, _ = la.la_ssm_conv(far, torch.ones(8, 1, device="cuda"))
    y = y.flatten().tolist()
    assert y[0] == float("inf") and y[1] == far[0, 0, 1].item() and y[2:6] == [0, 0, 0, 0] and y[6] != y[6] and y[7] == 100


def test_event_of_a_batch_of_several_launches():
    """More sequences with lengths than one launch takes: the event lies behind the last launch.
    The first 128 sequences hold one token each, the others all the work."""
    B, N, ch, n = 256, 2048, 256, 16
    lens = [1] * 128 + [N] * 128
    r = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    x, bc, w = r(B, N, ch), r(B, N, n), torch.randn(ch, 4, device="cuda")
    delta, A = torch.rand(B, N, ch, device="cuda").bfloat16(), -torch.rand(ch, n, device="cuda")
    q = r(B, 2, N, 64)
    u, y, o = torch.empty_like(x), torch.empty_like(x), torch.empty_like(q)
    for name, call in (("conv", lambda: la.la_ssm_conv(x, w, seq_lens=lens, out=u)),
                       ("scan", lambda: la.la_ssm_scan(x, delta, A, bc, bc, seq_lens=lens, out=y)),
                       ("window", lambda: la.la_window_prefill(q, q, q, 256, seq_lens=lens, out=o))):
        call()
        start, mark, end = (torch.cuda.Event(enable_timing=True) for _ in range(3))
        mark.record()
        torch.cuda.synchronize()
        la.la_set_stage_events([mark])
        try:
            torch.cuda._sleep(20_000_000)        # the launches queue up behind it: no host time between them
            start.record()
            call()
            end.record()
        finally:
            la.la_set_stage_events(None)
        torch.cuda.synchronize()
        assert start.elapsed_time(mark) > 0.5 * start.elapsed_time(end), name


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_empty_calls(dtype):
    """No sequences, no tokens, no channels, sequences of length zero: nothing but what the formulas leave."""
    r = lambda *s: torch.randn(*s, device="cuda").to(dtype)  # noqa: E731
    A, w, h0 = -torch.rand(16, 4, device="cuda"), torch.randn(16, 4, device="cuda"), torch.randn(2, 16, 4, device="cuda")
    for B, N, lens in ((0, 5, None), (2, 0, None), (2, 5, [0, 0])):
        x, bc, c0 = r(B, N, 16), r(B, N, 4), r(B, 3, 16)
        out = torch.full_like(x, 7.0)
        y, h = la.la_ssm_scan(x, x, A, bc, bc, h0=h0[:B].contiguous(), seq_lens=lens, out=out)
        assert torch.equal(h, h0[:B]) and (y == 7.0).all()
        y, h = la.la_ssm_scan(x, x, A, bc, bc, seq_lens=lens, out=out)
        assert not h.any() and (y == 7.0).all()
        u, c = la.la_ssm_conv(x, w, cache=c0, seq_lens=lens, out=out)
        assert torch.equal(c, c0) and (u == 7.0).all()
        q, kc = r(B, 2, N, 64), r(B, 2, 9, 64)
        vc, o = r(B, 2, 9, 64), torch.full((B, 2, N, 64), 7.0, dtype=dtype, device="cuda")
        k0, v0, pos = kc.clone(), vc.clone(), torch.full((B,), 6, dtype=torch.int32, device="cuda")
        la.la_window_prefill(q, q, q, 8, sinks=1, k_cache=kc, v_cache=vc, pos=pos, seq_lens=lens, out=o)
        assert (o == 7.0).all() and torch.equal(kc, k0) and torch.equal(vc, v0)
    x, bc = r(0, 16), r(0, 4)
    assert la.la_ssm_step(x, x, A, bc, bc, h0[:0]).shape == (0, 16)
    e = r(0, 2, 64)
    assert la.la_window_decode_step(e, e, e, r(0, 2, 9, 64), r(0, 2, 9, 64), torch.zeros(0, dtype=torch.int32, device="cuda"),
                                    8, sinks=1).shape == (0, 2, 64)
    x = r(2, 5, 0)
    y, h = la.la_ssm_scan(x, x, A[:0], r(2, 5, 4), r(2, 5, 4))
    assert y.shape == (2, 5, 0) and h.shape == (2, 0, 4)
    u, c = la.la_ssm_conv(x, w[:0])
    assert u.shape == (2, 5, 0) and c.shape == (2, 3, 0)
    torch.cuda.synchronize()
    la.la_prefill_check()
