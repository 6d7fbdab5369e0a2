"""State-space and sliding-window entry points: argument checks that return
before any CUDA call, host-only queries, and the binding's own checks (no GPU
needed; the pointers below are never dereferenced)."""
import ctypes

import pytest
import torch

import causal_kernelized_linear_la_b200 as la
from causal_kernelized_linear_la_b200 import LaConfig, LaSsmStrides, LaWindowStrides

P = 1 << 20
C = ctypes.c_void_p


def _cfg(dtype=la.LA_BF16, S0=None, ws=None, wsb=0):
    return LaConfig(dtype, 0, 0.0, None, S0, None, ws, wsb)


def _conv(x=P, w_=P, bias=None, cache=None, out=P, cache_out=None, lens=None, B=1, N=8, D=16, w=4, xb=128, xt=16, cfg=None):
    arr = None if lens is None else (ctypes.c_int * len(lens))(*lens)
    c = _cfg() if cfg is None else cfg
    return la.lib().la_ssm_conv(C(x), C(w_), C(bias), C(cache), C(out), C(cache_out), arr, B, N, D, w, 1, xb, xt,
                                ctypes.byref(c))


def test_conv_refusals():
    assert _conv(B=-1) == la.LA_ERR_INVALID
    assert _conv(N=-1) == la.LA_ERR_INVALID
    assert _conv(w=0) == la.LA_ERR_INVALID
    assert _conv(w=9) == la.LA_ERR_UNSUPPORTED
    assert _conv(xt=-1) == la.LA_ERR_INVALID
    assert _conv(N=(1 << 30) + 1) == la.LA_ERR_UNSUPPORTED
    assert _conv(x=0) == la.LA_ERR_INVALID
    assert _conv(out=0) == la.LA_ERR_INVALID
    assert _conv(cfg=_cfg(dtype=5)) == la.LA_ERR_INVALID
    assert _conv(lens=[9]) == la.LA_ERR_INVALID
    assert _conv(lens=[-1]) == la.LA_ERR_INVALID
    assert _conv(x=P + 1) == la.LA_ERR_ALIGN                       # off its elements
    assert _conv(w_=P + 4) == la.LA_ERR_ALIGN
    assert _conv(cache=P, cache_out=P + 16) == la.LA_ERR_INVALID   # overlaps the cache in part
    assert _conv(cache_out=P + 32) == la.LA_ERR_INVALID            # overlaps x
    # the last row of a strided x: 7 * 64 + 16 elements
    assert _conv(xt=64, cache_out=P + 2 * (7 * 64 + 8)) == la.LA_ERR_INVALID
    assert _conv(B=0) == la.LA_OK
    assert _conv(D=0) == la.LA_OK
    assert _conv(N=0, x=0, w_=0, out=0) == la.LA_OK                # no tokens and no cache to pass on


def _scan(x=P, A=P, h_out=2 * P, lens=None, B=1, N=8, D=16, G=1, n=4, st=None, cfg=None, z=None, out=P):
    arr = None if lens is None else (ctypes.c_int * len(lens))(*lens)
    c = _cfg() if cfg is None else cfg
    return la.lib().la_ssm_scan(C(x), C(P), C(A), C(P), C(P), None, C(z), None, C(out), C(h_out), arr, B, N, D, G, n, 1,
                                None if st is None else ctypes.byref(st), ctypes.byref(c))


def test_scan_refusals():
    assert _scan(B=-1) == la.LA_ERR_INVALID
    assert _scan(N=-1) == la.LA_ERR_INVALID
    assert _scan(n=0) == la.LA_ERR_INVALID
    assert _scan(n=65) == la.LA_ERR_UNSUPPORTED
    assert _scan(N=(1 << 30) + 1) == la.LA_ERR_UNSUPPORTED
    assert _scan(G=3) == la.LA_ERR_INVALID                         # 16 channels in 3 groups
    assert _scan(G=0) == la.LA_ERR_INVALID
    assert _scan(x=0) == la.LA_ERR_INVALID
    assert _scan(cfg=_cfg(dtype=3)) == la.LA_ERR_INVALID
    assert _scan(A=P + 4) == la.LA_ERR_ALIGN
    assert _scan(z=P + 1) == la.LA_ERR_ALIGN
    assert _scan(h_out=2 * P + 8) == la.LA_ERR_ALIGN
    assert _scan(lens=[9]) == la.LA_ERR_INVALID
    assert _scan(st=LaSsmStrides(128, -16)) == la.LA_ERR_INVALID
    assert _scan(cfg=_cfg(S0=2 * P)) == la.LA_ERR_INVALID          # final states over the start states
    assert _scan(cfg=_cfg(S0=2 * P + 16)) == la.LA_ERR_INVALID
    assert _scan(N=100000) == la.LA_ERR_WORKSPACE                  # few channels: several segments
    assert _scan(B=0) == la.LA_OK
    assert _scan(D=0, G=0) == la.LA_OK


def test_scan_workspace():
    ws = la.la_ssm_scan_workspace_bytes
    assert ws(1, 8192, 4096, 1, 16) == 0                # enough channels for every SM: one segment
    assert ws(1, 0, 512, 1, 16) == 0 and ws(0, 8, 512, 1, 16) == 0
    assert ws(1, 64, 32, 1, 16) == 0                    # too short to cut
    # one summary of 32 channels x (16 states + a sum) fp32 a segment and tile; whole tiles of
    # 32 channels, so narrower layers take the same
    n = ws(1, 32768, 512, 1, 16)
    assert n > 0 and n % (16 * 32 * 17 * 4) == 0
    assert ws(1, 32768, 500, 1, 16) == n
    assert ws(2, 32768, 512, 1, 16) % (2 * 16 * 32 * 17 * 4) == 0
    # the caller of a smaller batch never needs more than it was told
    for N in (255, 256, 257, 4095, 32768, 100001):
        assert ws(1, N, 40, 2, 5) % (2 * 32 * 9 * 4) == 0


def _step(h=P, x=P, cfg=None, B=1, D=16, n=4, G=1):
    c = _cfg() if cfg is None else cfg
    return la.lib().la_ssm_step(C(x), C(P), C(P), C(P), C(P), None, None, None, C(h), C(P), B, D, G, n, 1, None,
                                ctypes.byref(c))


def test_step_refusals():
    assert _step(h=0) == la.LA_ERR_INVALID
    assert _step(h=P + 8) == la.LA_ERR_ALIGN
    assert _step(n=65) == la.LA_ERR_UNSUPPORTED
    assert _step(G=5) == la.LA_ERR_INVALID
    assert _step(x=0) == la.LA_ERR_INVALID
    assert _step(B=0, h=0) == la.LA_OK


FAR = 1 << 40


def _window(q=P, k=2 * P, v=3 * P, out=4 * P, kc=None, vc=None, pos=None, lens=None, B=1, Hq=2, Hkv=1, N=8, d=64, dv=64,
            window=4, sinks=1, scale=0.1, st=None, cfg=None):
    arr = None if lens is None else (ctypes.c_int * len(lens))(*lens)
    c = _cfg() if cfg is None else cfg
    return la.lib().la_window_prefill(C(q), C(k), C(v), C(out), C(kc), C(vc), C(pos), arr, B, Hq, Hkv, N, d, dv, window,
                                      sinks, scale, None if st is None else ctypes.byref(st), ctypes.byref(c))


def test_window_refusals():
    bad, unsup, align = la.LA_ERR_INVALID, la.LA_ERR_UNSUPPORTED, la.LA_ERR_ALIGN
    assert _window(B=-1) == bad
    assert _window(window=0) == bad
    assert _window(sinks=-1) == bad
    assert _window(Hq=3, Hkv=2) == bad
    assert _window(Hkv=0) == bad
    assert _window(d=96) == unsup
    assert _window(dv=32) == unsup
    assert _window(N=65535 * 256 + 1) == unsup
    assert _window(scale=float("nan")) == bad
    assert _window(scale=float("inf")) == bad
    assert _window(cfg=_cfg(dtype=9)) == bad
    assert _window(q=0) == bad
    assert _window(kc=FAR) == bad                               # half a cache
    assert _window(pos=P) == bad                                # positions without a cache
    assert _window(kc=FAR, vc=FAR + 64) == bad                  # the caches overlap
    assert _window(kc=FAR, vc=2 * P) == bad                     # a cache over k
    assert _window(kc=FAR, vc=FAR << 1, window=1 << 30) == unsup
    assert _window(out=2 * P + 64) == bad                       # out over k
    assert _window(q=P + 8) == align
    assert _window(kc=FAR + 8, vc=FAR << 1) == align
    assert _window(kc=FAR, vc=FAR << 1, pos=P + 2) == align
    assert _window(lens=[9]) == bad
    dense = [1024, 512, 64] * 4
    assert _window(st=LaWindowStrides(*dense[:2], 68, *dense[3:])) == align     # rows off 16 bytes
    assert _window(st=LaWindowStrides(*dense[:2], 32, *dense[3:])) == bad       # rows that share memory
    assert _window(st=LaWindowStrides(-1024, *dense[1:])) == bad
    assert _window(B=0) == la.LA_OK
    assert _window(N=0, q=0, k=0, v=0, out=0) == la.LA_OK


def test_decode_refusals():
    def call(kc=FAR, vc=FAR << 1, pos=P, window=4, q=P):
        c = _cfg()
        return la.lib().la_window_decode_step(C(q), C(2 * P), C(3 * P), C(4 * P), C(kc), C(vc), C(pos), 1, 2, 1, 64, 64,
                                              window, 1, 0.1, None, ctypes.byref(c))
    assert call(kc=0, vc=0) == la.LA_ERR_INVALID
    assert call(pos=0) == la.LA_ERR_INVALID
    assert call(vc=0) == la.LA_ERR_INVALID
    assert call(window=0) == la.LA_ERR_INVALID
    assert call(q=P + 2) == la.LA_ERR_ALIGN


def test_binding_checks():
    x, w = torch.zeros(2, 8, 16), torch.zeros(16, 4)
    with pytest.raises(ValueError, match="CUDA"):
        la.la_ssm_conv(x, w)
    with pytest.raises(ValueError, match="weight"):
        la.la_ssm_conv(x, torch.zeros(15, 4))
    with pytest.raises(ValueError, match="cache"):
        la.la_ssm_conv(x, w, cache=torch.zeros(2, 4, 16))
    with pytest.raises(ValueError, match="contiguous"):
        la.la_ssm_conv(x.transpose(1, 2), torch.zeros(8, 4))
    A, bc = torch.zeros(16, 4), torch.zeros(2, 8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        la.la_ssm_scan(x, x, A, bc, bc)
    with pytest.raises(ValueError, match="groups"):
        la.la_ssm_scan(x, x, A, torch.zeros(2, 8, 3, 4), bc)
    with pytest.raises(ValueError, match="C must"):
        la.la_ssm_scan(x, x, A, bc, bc[:, :7])
    with pytest.raises(ValueError, match="A must"):
        la.la_ssm_scan(x, x, A[:, :3], bc, bc)
    with pytest.raises(ValueError, match="dtype"):
        la.la_ssm_scan(x, x.bfloat16(), A, bc, bc)
    with pytest.raises(ValueError, match="h must"):
        la.la_ssm_step(x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0], torch.zeros(2, 16, 5))
    q, k = torch.zeros(1, 2, 8, 64), torch.zeros(1, 1, 8, 64)
    with pytest.raises(ValueError, match="CUDA"):
        la.la_window_prefill(q, k, k, 4)
    with pytest.raises(ValueError, match="32 bits"):
        la.la_window_prefill(q, k, k, (1 << 32) + 4)      # would wrap to 4
    with pytest.raises(ValueError, match="do not fit"):
        la.la_window_prefill(q, k, k[:, :, :7], 4)
    with pytest.raises(ValueError, match="k_cache"):
        la.la_window_prefill(q, k, k, 4, k_cache=torch.zeros(1, 1, 5, 64), v_cache=torch.zeros(1, 1, 4, 64))
    with pytest.raises(ValueError, match="pos"):
        la.la_window_decode_step(q[:, :, 0], k[:, :, 0], k[:, :, 0], torch.zeros(1, 1, 4, 64), torch.zeros(1, 1, 4, 64),
                                 torch.zeros(1), 4)


def test_outputs_that_share_memory_are_refused():
    dense = [1024, 512, 64] * 4
    assert _window(Hq=2, Hkv=1, st=LaWindowStrides(*dense[:10], 0, 64)) == la.LA_ERR_INVALID     # heads of out
    assert _window(B=2, st=LaWindowStrides(*dense[:9], 0, 512, 64)) == la.LA_ERR_INVALID         # sequences of out
    x, A, bc = torch.zeros(1, 4096, 32), torch.zeros(32, 16), torch.zeros(1, 4096, 16)
    need = la.la_ssm_scan_workspace_bytes(1, 4096, 32, 1, 16)
    assert need > 0
    with pytest.raises(ValueError, match="workspace"):        # many bytes by its shape, one in memory
        la.la_ssm_scan(x, x, A, bc, bc, workspace=torch.zeros(1, dtype=torch.uint8).expand(need))


def test_conv_out_over_its_inputs():
    assert _conv(x=P, out=P) == la.LA_ERR_INVALID                              # in place of x
    assert _conv(x=P, out=P + 128, B=1) == la.LA_ERR_INVALID                   # behind its first rows
    assert _conv(x=P, out=2 * P, cache=2 * P + 32) == la.LA_ERR_INVALID
    assert _conv(x=P, out=2 * P, cache_out=2 * P + 32) == la.LA_ERR_INVALID


def test_window_outputs_over_other_arguments():
    """The layout decides, not whether strides are given: the binding always gives them."""
    bad = la.LA_ERR_INVALID
    dense = LaWindowStrides(1024, 512, 64, 512, 512, 64, 512, 512, 64, 1024, 512, 64)
    for st in (None, dense):
        assert _window(out=2 * P + 64, st=st) == bad                # over k
        assert _window(out=3 * P - 64, st=st) == bad                # its last rows over v's first
        assert _window(out=P + 128, st=st) == bad                   # over q, a row on
        assert _window(kc=FAR, vc=FAR << 1, out=FAR + 128, st=st) == bad
        assert _window(kc=FAR, vc=FAR << 1, out=(FAR << 1) + 128, st=st) == bad
        assert _window(kc=FAR, vc=FAR << 1, q=FAR, st=st) == bad    # q inside a cache
        assert _window(kc=FAR, vc=FAR << 1, pos=4 * P + 16, st=st) == bad      # positions inside out
        assert _window(kc=FAR, vc=FAR << 1, pos=FAR + 16, st=st) == bad        # ... inside a cache
    # out over q with another order of rows and heads
    assert _window(out=P, st=LaWindowStrides(1024, 512, 64, 512, 512, 64, 512, 512, 64, 1024, 64, 128)) == bad
    # heads (sequences) of out that are neither equal nor apart
    assert _window(st=LaWindowStrides(1024, 512, 64, 512, 512, 64, 512, 512, 64, 1024, 8, 64)) == bad
    assert _window(B=2, st=LaWindowStrides(1024, 512, 64, 512, 512, 64, 512, 512, 64, 64, 512, 64)) == bad
    # one buffer of 8 rows of 64 x (2 q, 1 k, 1 v): out on k's columns
    packed = LaWindowStrides(2048, 64, 256, 2048, 64, 256, 2048, 64, 256, 2048, 64, 256)
    assert _window(q=P, k=P + 256, v=P + 384, out=P + 128, st=packed) == bad


def test_decode_outputs_over_other_arguments():
    def call(q=P, out=4 * P, pos=5 * P, Hq=2, st=None):
        c = _cfg()
        return la.lib().la_window_decode_step(C(q), C(2 * P), C(3 * P), C(out), C(FAR), C(FAR << 1), C(pos), 1, Hq, 1, 64,
                                              64, 4, 1, 0.1, None if st is None else ctypes.byref(st), ctypes.byref(c))
    for st in (None, LaWindowStrides(128, 64, 0, 64, 64, 0, 64, 64, 0, 128, 64, 0)):
        for kw in (dict(out=2 * P), dict(out=3 * P - 128), dict(out=FAR + 128), dict(out=(FAR << 1) + 512), dict(q=FAR),
                   dict(out=P + 128), dict(pos=FAR), dict(pos=4 * P + 16)):
            assert call(st=st, **kw) == la.LA_ERR_INVALID, kw


def _ssm(step, x=P, delta=2 * P, A=3 * P, Bm=4 * P, Cm=5 * P, D=6 * P, z=7 * P, bias=8 * P, out=9 * P, h=10 * P, S0=None,
         ws=None, wsb=0, N=40, st=None):
    B, ch, G, n = 2, 32, 1, 16
    c = _cfg(S0=S0, ws=ws, wsb=wsb)
    st = None if st is None else ctypes.byref(st)
    ptrs = [C(p) for p in (x, delta, A, Bm, Cm, D, z, bias)]
    if step:
        return la.lib().la_ssm_step(*ptrs, C(h), C(out), B, ch, G, n, 1, st, ctypes.byref(c))
    return la.lib().la_ssm_scan(*ptrs, C(out), C(h), None, B, N, ch, G, n, 1, st, ctypes.byref(c))


@pytest.mark.parametrize("step", [False, True])
def test_ssm_outputs_over_other_arguments(step):
    """Two sequences of 32 channels and 16 states: rows of 64 bytes, states of 2048 bytes a sequence."""
    bad = la.LA_ERR_INVALID
    for arg in ("Bm", "Cm", "A", "D", "bias", "h"):
        at = dict(Bm=4, Cm=5, A=3, D=6, bias=8, h=10)[arg] * P
        assert _ssm(step, out=at) == bad, arg                       # out over it ...
        assert _ssm(step, out=at - 64) == bad, arg                  # ... by its last row
        if arg != "h":
            assert _ssm(step, h=at) == bad, arg
            assert _ssm(step, h=at - 4080) == bad, arg
    for arg in ("x", "delta", "z"):
        at = dict(x=1, delta=2, z=7)[arg] * P
        assert _ssm(step, out=at + 64) == bad, arg                  # a row on
        assert _ssm(step, out=at - 2) == bad, arg
        assert _ssm(step, h=at) == bad, arg
    # in x's place, but x has other strides
    wide = LaSsmStrides(80 * 32, 64, 40 * 32, 32, 40 * 32, 32, 40 * 16, 16, 40 * 16, 16)
    assert _ssm(step, out=P, st=wide) == bad
    # every sequence reads the first one's rows, out has rows of its own
    one = LaSsmStrides(0, 32, 40 * 32, 32, 40 * 32, 32, 40 * 16, 16, 40 * 16, 16)
    assert _ssm(step, out=P, st=one) == bad


def test_scan_workspace_over_other_arguments():
    N = 4096
    need = la.la_ssm_scan_workspace_bytes(2, N, 32, 1, 16)
    assert need > 0
    far = 1 << 40
    assert _ssm(False, N=N, ws=None, wsb=need) == la.LA_ERR_WORKSPACE          # bytes of no workspace
    apart = dict(x=far, delta=2 * far, A=3 * far, Bm=4 * far, Cm=5 * far, D=6 * far, z=7 * far, bias=8 * far, out=9 * far,
                 h=10 * far, S0=11 * far)
    for arg, at in apart.items():
        assert _ssm(False, N=N, **apart, ws=at, wsb=need) == la.LA_ERR_INVALID, arg
        assert _ssm(False, N=N, **apart, ws=at - need + 16, wsb=need) == la.LA_ERR_INVALID, arg
    assert _ssm(False, N=N, **{**apart, "S0": apart["out"] + 64}, ws=far // 2, wsb=need) == la.LA_ERR_INVALID


def test_conv_outputs_over_a_strided_x():
    bad = la.LA_ERR_INVALID
    # one sequence of 8 rows of 16 in rows of 64 elements: out (256 bytes) over some of them
    for at in (P, P + 128, P + 2 * 7 * 64 - 224, P - 240):
        assert _conv(out=at, w_=2 * P, xt=64) == bad
    # two sequences 1024 elements apart: out over the second, or cache_out over its last row
    assert _conv(B=2, out=P + 2 * (1024 + 7 * 64), w_=2 * P, xt=64, xb=1024) == bad
    assert _conv(B=2, out=3 * P, cache_out=P + 2 * (1024 + 7 * 64) + 30, w_=2 * P, xt=64, xb=1024) == bad
    # the filter and the bias are read by every thread
    assert _conv(x=4 * P, out=P + 128, w_=P) == bad
    assert _conv(x=4 * P, out=P + 32, w_=2 * P, bias=P) == bad
    assert _conv(x=4 * P, out=5 * P, w_=P, cache_out=P + 240) == bad
    assert _conv(x=4 * P, out=5 * P, w_=2 * P, bias=P, cache_out=P + 32) == bad
