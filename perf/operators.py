"""Measured cases of the constant-memory token mixers beside linear attention.

Five operators.  Three form a selective state-space layer:

* ``conv``: short causal convolution over the tokens of [B, N, D] rows, with
  bias, SiLU and a cache of the last w - 1 inputs (N = 1: one new token),
* ``scan``: h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t,  y_t = C_t h_t + D x_t,
  times SiLU(z_t), for prompts,
* ``step``: the same recurrence for one token a sequence, the state updated in place.

Two are softmax attention whose context is bounded: query i sees key j when
j <= i and (i - j < window or j < sinks):

* ``window``: prompts, from an empty start or behind a rolling cache,
* ``decode``: one token a sequence against the rolling cache, which takes the
  token's key and value in place.

``run`` computes a case in elementary torch operations in 32 bits, or, with
``own`` set, by the library's calls.  ``exact`` evaluates the definitions in
64 bits, token by token or head by head.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # the convolution of a long prompt, its input one half of a gated projection's output
        dict(name="conv prompt", op="conv", dtype="bf16", B=1, N=32768, D=4096, w=4, bias=True, silu=True, cache=True,
             half=True, lens=""),
        # the convolution of one new token in a serving batch: a latency-bound call
        dict(name="conv token", op="conv", dtype="bf16", B=256, N=1, D=4096, w=4, bias=True, silu=True, cache=True,
             half=True, lens=""),
        # a long prompt of one user through a wide layer
        dict(name="scan prompt", op="scan", dtype="bf16", B=1, N=8192, D=4096, n=16, G=1, softplus=True, skip=True,
             gate=True, start=False, half=True, lens=""),
        # a padded batch of fp32 continuations, odd lengths and an odd width
        dict(name="scan ragged f32", op="scan", dtype="f32", B=4, N=1000, D=1025, n=16, G=1, softplus=True, skip=True,
             gate=True, start=True, half=False, lens="1000,517,64,1"),
        # a very long prompt through a narrow layer: few channels, many tokens
        dict(name="scan narrow long", op="scan", dtype="bf16", B=1, N=32768, D=512, n=16, G=1, softplus=True,
             skip=True, gate=True, start=True, half=True, lens=""),
        # one new token of a single user
        dict(name="step one user", op="step", dtype="bf16", B=1, D=4096, n=16, G=1, softplus=True, skip=True,
             gate=True, half=True),
        # one new token of each of 256 resident sequences
        dict(name="step batch", op="step", dtype="bf16", B=256, D=4096, n=16, G=1, softplus=True, skip=True, gate=True,
             half=True),
        # a long prompt of one user, grouped heads
        dict(name="window prompt", op="window", dtype="bf16", B=1, Hq=32, Hkv=8, N=16384, d=128, dv=128, window=4096,
             sinks=4, cached=False, pos="", fused=True, lens=""),
        # a padded batch of short prompts, small heads and a short window
        dict(name="window ragged", op="window", dtype="bf16", B=4, Hq=8, Hkv=8, N=4096, d=64, dv=64, window=512,
             sinks=16, cached=False, pos="", fused=False, lens="4096,3000,700,65"),
        # a chunk of new tokens behind the rolling cache of sequences of different ages
        dict(name="window chunk", op="window", dtype="bf16", B=2, Hq=16, Hkv=4, N=777, d=128, dv=128, window=2048,
             sinks=4, cached=True, pos="5000,300", fused=True, lens="777,500"),
        # one new token of a single user
        dict(name="decode one user", op="decode", dtype="bf16", B=1, Hq=32, Hkv=8, d=128, dv=128, window=4096, sinks=4,
             pos="9000"),
        # one new token of each sequence of a serving batch
        dict(name="decode batch", op="decode", dtype="bf16", B=64, Hq=32, Hkv=8, d=128, dv=128, window=4096, sinks=4,
             pos=""),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, B, N):
    if B == 1 or rng.random() < 0.4:
        return ""
    return ",".join(str(N if b == 0 else rng.randint(0, N)) for b in range(B))


def draw(rng):
    op = rng.choice(["conv", "scan", "step", "window", "decode"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    width = lambda top: rng.choice([_log(rng, 1, top), 8 * _log(rng, 4, top // 8), 64 * _log(rng, 1, top // 64)])  # noqa: E731
    if op == "conv":
        B, D = _log(rng, 1, 64), width(4096)
        N = rng.choice([1, _log(rng, 1, max(1, min(32768, (1 << 25) // (B * D))))])
        return dict(op=op, dtype=dtype, B=B, N=N, D=D, w=rng.randint(1, 8), bias=rng.random() < 0.7,
                    silu=rng.random() < 0.7, cache=rng.random() < 0.6, half=rng.random() < 0.5, lens=_lens(rng, B, N))
    if op == "scan":
        B, n = _log(rng, 1, 8), rng.choice([16, 16, rng.randint(1, 64)])
        G = rng.choice([1, 1, 2, 4])
        D = G * max(1, width(4096) // G)
        N = _log(rng, 1, max(2, min(16384, (1 << 28) // (B * D * n))))
        return dict(op=op, dtype=dtype, B=B, N=N, D=D, n=n, G=G, softplus=rng.random() < 0.7, skip=rng.random() < 0.7,
                    gate=rng.random() < 0.7, start=rng.random() < 0.5, half=rng.random() < 0.5, lens=_lens(rng, B, N))
    if op == "step":
        B, n, G = _log(rng, 1, 256), rng.choice([16, 16, rng.randint(1, 64)]), rng.choice([1, 1, 2])
        return dict(op=op, dtype=dtype, B=B, D=G * max(1, width(4096) // G), n=n, G=G, softplus=rng.random() < 0.7,
                    skip=rng.random() < 0.7, gate=rng.random() < 0.7, half=rng.random() < 0.5)
    heads = rng.choice([1, 2, 4, 8])
    group, d, dv = rng.choice([1, 2, 4, 8, 3]), rng.choice([64, 128]), rng.choice([64, 128])
    window, sinks = _log(rng, 1, 4096), rng.choice([0, 4, rng.randint(0, 200)])
    if op == "window":
        B = _log(rng, 1, 8)
        top = (1 << 28 if dtype == "f32" else 1 << 30) // (B * heads * group * (min(window, 4096) + 256))
        N = _log(rng, 1, max(2, min(8192, top)))
        cached = rng.random() < 0.5
        pos = ",".join(str(rng.choice([0, rng.randint(0, sinks + window), _log(rng, 1, 10 ** 6)])) for _ in range(B))
        return dict(op=op, dtype=dtype, B=B, Hq=heads * group, Hkv=heads, N=N, d=d, dv=dv, window=window, sinks=sinks,
                    cached=cached, pos=pos if cached else "", fused=d == dv and rng.random() < 0.5,
                    lens=_lens(rng, B, N))
    B = _log(rng, 1, 64)
    pos = ",".join(str(rng.choice([0, rng.randint(0, sinks + window), _log(rng, 1, 10 ** 6)])) for _ in range(B))
    return dict(op=op, dtype=dtype, B=B, Hq=heads * group, Hkv=heads, d=d, dv=dv, window=window, sinks=sinks, pos=pos)


def _ints(text, B, default):
    return [int(t) for t in text.split(",")] if text else [default] * B


def _seen(p, window, sinks):
    """How many keys the query at position p sees."""
    return min(p + 1, sinks) + max(0, min(p + 1 - sinks, window))


def _pos(case):
    if case["pos"]:
        return _ints(case["pos"], case["B"], 0)
    # a serving batch: sequences of many ages, most of them past the window
    return [0 if case["op"] == "window" else 2000 + 517 * b for b in range(case["B"])]


def work(case):
    e, op, B = ESIZE[case["dtype"]], case["op"], case["B"]
    if op == "conv":
        rows = sum(_ints(case["lens"], B, case["N"]))
        D, w = case["D"], case["w"]
        return {"bytes": 2 * rows * D * e + (w + 1) * D * 4 + (2 if case["cache"] else 1) * B * (w - 1) * D * e,
                "flops": 2 * rows * D * w}
    if op in ("scan", "step"):
        rows = sum(_ints(case["lens"], B, case["N"])) if op == "scan" else B
        D, n = case["D"], case["n"]
        state = B * D * n * 4 * (1 if op == "scan" and not case["start"] else 2)
        return {"bytes": rows * (D * (4 if case["gate"] else 3) + 2 * case["G"] * n) * e + state + D * n * 4,
                "flops": rows * D * (7 * n + 4)}
    pos, Hq, Hkv, d, dv = _pos(case), case["Hq"], case["Hkv"], case["d"], case["dv"]
    if op == "window":
        lens = _ints(case["lens"], B, case["N"])
        pairs = sum(sum(_seen(p + i, case["window"], case["sinks"]) for i in range(n)) for p, n in zip(pos, lens))
        rows = sum(lens) * (Hq + Hkv)
        if case["cached"]:
            kept = [(min(p, case["sinks"] + case["window"]), min(n, case["sinks"] + case["window"])) for p, n in zip(pos, lens)]
            rows += Hkv * sum(a + b for a, b in kept)
        return {"bytes": rows * (d + dv) * e, "flops": 2 * Hq * pairs * (d + dv)}
    pairs = sum(_seen(p, case["window"], case["sinks"]) for p in pos)
    return {"bytes": (Hkv * (pairs + B) + B * Hq) * (d + dv) * e, "flops": 2 * Hq * pairs * (d + dv)}


# ---------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    dev, dt, op, B = "cuda", DTYPES[case["dtype"]], case["op"], case["B"]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    s = dict(case)
    if op == "conv":
        N, D, w = case["N"], case["D"], case["w"]
        # x is the first half of a [B, N, 2D] projection, the gate the second
        x = normal(B, N, 2 * D if case["half"] else D).to(dt)
        s["x"] = x[..., :D]
        s["weight"] = normal(D, w) / math.sqrt(w)
        s["bias"] = 0.1 * normal(D) if case["bias"] else None
        s["cache"] = normal(B, w - 1, D).to(dt) if case["cache"] else None
        s["cache_out"] = torch.zeros(B, w - 1, D, device=dev, dtype=dt)
        s["out"] = torch.zeros(B, N, D, device=dev, dtype=dt)
        s["lens"] = _ints(case["lens"], B, N) if case["lens"] else None
        return s
    if op in ("scan", "step"):
        rows = (B, case["N"]) if op == "scan" else (B,)
        D, n, G = case["D"], case["n"], case["G"]
        # the inputs of the recurrence: x behind the convolution's SiLU, the step
        # sizes' raw values, B and C slices of one projection, the gate half of another
        x = normal(*rows, D)
        s["x"] = (x * torch.sigmoid(x)).to(dt)
        s["delta"] = (0.5 * normal(*rows, D)).to(dt)
        bc = normal(*rows, 2 * G * n).to(dt)
        s["B_"] = bc[..., :G * n].unflatten(-1, (G, n))
        s["C"] = bc[..., G * n:].unflatten(-1, (G, n))
        if not case["half"]:
            s["B_"], s["C"] = s["B_"].contiguous(), s["C"].contiguous()
        z = normal(*rows, 2 * D if case["half"] else D).to(dt)
        s["z"] = z[..., z.shape[-1] - D:] if case["gate"] else None
        # steps of 0.001 to 0.1 and decay rates of 1 to n, as such layers start from
        steps = torch.exp(torch.rand(D, generator=gen, device=dev) * math.log(100.0) + math.log(0.001))
        s["delta_bias"] = steps + torch.log(-torch.expm1(-steps)) if case["softplus"] else None
        if not case["softplus"]:
            s["delta"] = (steps * torch.exp(0.5 * normal(*rows, D))).to(dt)
        s["A"] = -torch.arange(1, n + 1, device=dev).float() * torch.exp(0.1 * normal(D, n))
        s["D_"] = 1.0 + 0.1 * normal(D) if case["skip"] else None
        s["h"] = normal(B, D, n) if op == "step" or case["start"] else None
        s["out"] = torch.zeros(*rows, D, device=dev, dtype=dt)
        if op == "scan":
            s["h_out"] = torch.zeros(B, D, n, device=dev)
            s["lens"] = _ints(case["lens"], B, case["N"]) if case["lens"] else None
        return s
    Hq, Hkv, d, dv, cap = case["Hq"], case["Hkv"], case["d"], case["dv"], case["window"] + case["sinks"]
    s["pos_host"] = _pos(case)
    s["pos"] = torch.tensor(s["pos_host"], dtype=torch.int32, device=dev)
    if op == "decode" or case["cached"]:
        s["k_cache"], s["v_cache"] = normal(B, Hkv, cap, d).to(dt), normal(B, Hkv, cap, dv).to(dt)
    else:
        s["k_cache"] = s["v_cache"] = s["pos"] = None
    if op == "decode":
        s["q"], s["k"], s["v"] = normal(B, Hq, d).to(dt), normal(B, Hkv, d).to(dt), normal(B, Hkv, dv).to(dt)
        s["out"] = torch.zeros(B, Hq, dv, device=dev, dtype=dt)
        return s
    N = case["N"]
    if case["fused"]:
        # heads side by side in each token's row, as one projection writes them
        qkv = normal(B, N, Hq + 2 * Hkv, d).to(dt).transpose(1, 2)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["out"] = torch.zeros(B, N, Hq, dv, device=dev, dtype=dt).transpose(1, 2)
    else:
        s["q"], s["k"], s["v"] = normal(B, Hq, N, d).to(dt), normal(B, Hkv, N, d).to(dt), normal(B, Hkv, N, dv).to(dt)
        s["out"] = torch.zeros(B, Hq, N, dv, device=dev, dtype=dt)
    s["lens"] = _ints(case["lens"], B, N) if case["lens"] else None
    return s


# ---------------------------------------------------------------------------
# the plain forms

def _lengths(s, device):
    n = s["N"]
    return torch.tensor(s["lens"] if s["lens"] else [n] * s["B"], device=device)


def _plain_conv(s):
    x, w, B, N = s["x"], s["w"], s["B"], s["N"]
    past = s["cache"] if s["cache"] is not None else torch.zeros(B, w - 1, s["D"], device=x.device, dtype=x.dtype)
    lens = _lengths(s, x.device)
    rows = torch.cat([past, x], 1)
    xh = rows.float().unfold(1, w, 1)                        # [B, N, D, w]
    y = (xh * s["weight"]).sum(-1)
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["silu"]:
        y = y * torch.sigmoid(y)
    keep = torch.arange(N, device=x.device) < lens[:, None]
    out = torch.where(keep[..., None], y.to(x.dtype), s["out"])
    at = lens[:, None] + torch.arange(w - 1, device=x.device)    # the last w - 1 rows of each sequence
    return out, torch.gather(rows, 1, at[..., None].expand(-1, -1, s["D"]))


def _scan_inputs(s):
    delta = s["delta"].float()
    if s["delta_bias"] is not None:
        delta = delta + s["delta_bias"]
    if s["softplus"]:
        delta = torch.where(delta > 20, delta, torch.log1p(torch.exp(delta.clamp(max=20))))
    per = s["D"] // s["G"]
    return delta, s["B_"].float().repeat_interleave(per, -2), s["C"].float().repeat_interleave(per, -2)


def _scan_output(s, y):
    if s["D_"] is not None:
        y = y + s["D_"] * s["x"].float()
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    return y.to(s["x"].dtype)


def _plain_scan(s):
    x, N = s["x"], s["N"]
    lens = _lengths(s, x.device)
    keep = torch.arange(N, device=x.device) < lens[:, None]
    delta, Bm, Cm = _scan_inputs(s)
    delta = torch.where(keep[..., None], delta, 0.0)
    a = torch.exp(delta[..., None] * s["A"])                 # [B, N, D, n]
    h = (delta * x.float())[..., None] * Bm
    if s["h"] is not None:
        h[:, 0] += a[:, 0] * s["h"]
    # prefix combination of the steps (a, h) in doubling spans
    span = 1
    while span < N:
        h[:, span:] += a[:, span:] * h[:, :-span].clone()
        a[:, span:] = a[:, span:] * a[:, :-span].clone()
        span *= 2
    y = _scan_output(s, (h * Cm).sum(-1))
    h_out = h[torch.arange(s["B"], device=x.device), (lens - 1).clamp(min=0)]
    start = s["h"] if s["h"] is not None else torch.zeros_like(h_out)
    return torch.where(keep[..., None], y, s["out"]), torch.where((lens > 0)[:, None, None], h_out, start)


def _plain_step(s):
    delta, Bm, Cm = _scan_inputs(s)
    a = torch.exp(delta[..., None] * s["A"])
    s["h"].mul_(a).add_((delta * s["x"].float())[..., None] * Bm)
    return _scan_output(s, (s["h"] * Cm).sum(-1)), s["h"]


def _slot(p, window, sinks):
    return torch.where(p < sinks, p, sinks + (p - sinks) % window)


def _slot_positions(s, device):
    """Position held by each cache slot of each sequence, -1 where it is empty."""
    pos = torch.tensor(s["pos_host"], device=device)[:, None]
    slot = torch.arange(s["window"] + s["sinks"], device=device)
    ring = pos - 1 - (pos - 1 - slot) % s["window"]          # the latest position before pos in this ring slot
    at = torch.where(slot < s["sinks"], slot, ring)
    return torch.where((at < pos) & (at >= torch.minimum(slot, torch.tensor(s["sinks"], device=device))), at, -1)


def _attend(q, k, v, mask, scale):
    """softmax(scale q k^T) v over the keys that mask keeps: q [..., g, rows, d],
    k, v [..., keys, .] shared by the g heads, mask [..., 1, rows, keys]."""
    g, rows = q.shape[-3:-1]
    score = torch.matmul(q.flatten(-3, -2), k.transpose(-1, -2)).unflatten(-2, (g, rows)) * scale
    score = torch.where(mask, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True).clamp(min=1e-30)
    return torch.matmul(p.flatten(-3, -2), v).unflatten(-2, (g, rows)) / total


def _plain_window(s):
    dev, dt, B, N, Hq, Hkv = s["q"].device, s["q"].dtype, s["B"], s["N"], s["Hq"], s["Hkv"]
    W, S, d, dv = s["window"], s["sinks"], s["d"], s["dv"]
    lens, start = _lengths(s, dev), torch.tensor(s["pos_host"], device=dev)
    cached = s["k_cache"] is not None
    cap = W + S if cached else 0
    new = torch.where(torch.arange(N, device=dev) < lens[:, None], start[:, None] + torch.arange(N, device=dev), -1)
    at = torch.cat([_slot_positions(s, dev), new], 1) if cached else new
    k = torch.cat([s["k_cache"], s["k"]], 2) if cached else s["k"]
    v = torch.cat([s["v_cache"], s["v"]], 2) if cached else s["v"]
    # blocks of queries; each sees the cache, the prompt's first tokens and a band
    blk = min(N, 512)
    nb = -(-N // blk)
    first = torch.arange(nb, device=dev)[:, None] * blk
    band = first + torch.arange(-min(W, N) + 1, blk, device=dev)
    ns = min(S, N)
    idx = torch.cat([torch.arange(cap + ns, device=dev).expand(nb, -1), cap + band.clamp(0, N - 1)], 1)
    kpos = at[:, idx]                                          # [B, nb, keys]
    in_band = torch.cat([torch.zeros(nb, cap + ns, dtype=torch.bool, device=dev), (band >= 0) & (band < N)], 1)
    # the prompt's own sinks come from the first list, everything else of it from the band
    old = torch.arange(idx.shape[1], device=dev) < cap
    usable = (kpos >= 0) & (old | torch.where(in_band, kpos >= S, (kpos < S) & (torch.arange(idx.shape[1], device=dev) < cap + ns)))
    row = (first + torch.arange(blk, device=dev)).clamp(max=N - 1)
    qpos = start[:, None, None] + row                          # [B, nb, blk]
    see = (kpos[:, :, None] <= qpos[..., None]) & ((qpos[..., None] - kpos[:, :, None] < W) | (kpos[:, :, None] < S))
    mask = (see & usable[:, :, None])[:, None, :, None]        # [B, 1, nb, 1, blk, keys]
    g = Hq // Hkv
    qb = s["q"].float().unflatten(1, (Hkv, g))[:, :, :, row].permute(0, 1, 3, 2, 4, 5)     # [B, Hkv, nb, g, blk, d]
    kb, vb = k.float()[:, :, idx], v.float()[:, :, idx]                                    # [B, Hkv, nb, keys, .]
    o = _attend(qb, kb, vb, mask, 1.0 / math.sqrt(d))
    o = o.permute(0, 1, 3, 2, 4, 5).reshape(B, Hq, nb * blk, dv)[:, :, :N].to(dt)
    keep = (torch.arange(N, device=dev) < lens[:, None])[:, None, :, None]
    o = torch.where(keep, o, s["out"])
    if not cached:
        return o
    # the cache keeps the sinks and the last `window` other tokens
    stays = (new >= 0) & ((new < S) | (new >= (start + lens)[:, None] - W))
    b, i = stays.nonzero(as_tuple=True)
    slot = _slot(new[b, i], W, S)
    s["k_cache"][b, :, slot] = s["k"][b, :, i]
    s["v_cache"][b, :, slot] = s["v"][b, :, i]
    return o, s["k_cache"], s["v_cache"]


def _plain_decode(s):
    dev, B, Hkv, W, S = s["q"].device, s["B"], s["Hkv"], s["window"], s["sinks"]
    pos = s["pos"].long()
    b = torch.arange(B, device=dev)
    slot = _slot(pos, W, S)
    s["k_cache"][b, :, slot] = s["k"]
    s["v_cache"][b, :, slot] = s["v"]
    at = _slot_positions({**s, "pos_host": [p + 1 for p in s["pos_host"]]}, dev)
    q = s["q"].float().unflatten(1, (Hkv, -1))[..., None, :]
    mask = (at >= 0)[:, None, None, None]
    o = _attend(q, s["k_cache"].float(), s["v_cache"].float(), mask, 1.0 / math.sqrt(s["d"]))
    return o.reshape(B, s["Hq"], s["dv"]).to(s["q"].dtype), s["k_cache"], s["v_cache"]


def _own_run(s):
    import causal_kernelized_linear_la_b200 as la
    op = s["op"]
    if op == "conv":
        return la.la_ssm_conv(s["x"], s["weight"], bias=s["bias"], cache=s["cache"], silu=s["silu"],
                              seq_lens=s["lens"], out=s["out"], cache_out=s["cache_out"])
    if op == "scan":
        return la.la_ssm_scan(s["x"], s["delta"], s["A"], s["B_"], s["C"], D=s["D_"], z=s["z"],
                              delta_bias=s["delta_bias"], delta_softplus=s["softplus"], h0=s["h"], seq_lens=s["lens"],
                              out=s["out"], h_out=s["h_out"])
    if op == "step":
        y = la.la_ssm_step(s["x"], s["delta"], s["A"], s["B_"], s["C"], s["h"], D=s["D_"], z=s["z"],
                           delta_bias=s["delta_bias"], delta_softplus=s["softplus"], out=s["out"])
        return y, s["h"]
    if op == "window":
        o = la.la_window_prefill(s["q"], s["k"], s["v"], s["window"], sinks=s["sinks"], k_cache=s["k_cache"],
                                 v_cache=s["v_cache"], pos=s["pos"], seq_lens=s["lens"], out=s["out"])
        return (o, s["k_cache"], s["v_cache"]) if s["cached"] else o
    o = la.la_window_decode_step(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["pos"], s["window"],
                                 sinks=s["sinks"], out=s["out"])
    return o, s["k_cache"], s["v_cache"]


def run(state):
    if own:
        return _own_run(state)
    return {"conv": _plain_conv, "scan": _plain_scan, "step": _plain_step, "window": _plain_window,
            "decode": _plain_decode}[state["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_conv(s):
    B, N, D, w = s["B"], s["N"], s["D"], s["w"]
    dev = s["x"].device
    out, kept = s["out"].double(), torch.zeros(B, w - 1, D, device=dev, dtype=torch.float64)
    for b in range(B):
        n = s["lens"][b] if s["lens"] else N
        past = s["cache"][b].double() if s["cache"] is not None else kept[b] * 0
        rows = torch.cat([past, s["x"][b, :n].double()])
        y = torch.zeros(n, D, device=dev, dtype=torch.float64)
        for i in range(w):
            y += s["weight"][:, i].double() * rows[i:i + n]
        if s["bias"] is not None:
            y += s["bias"].double()
        out[b, :n] = y / (1 + torch.exp(-y)) if s["silu"] else y
        kept[b] = rows[rows.shape[0] - (w - 1):]
    return out, kept


def _exact_recurrence(s, h, x, delta, Bm, Cm, z):
    """One token: the new state and the output."""
    if s["delta_bias"] is not None:
        delta = delta + s["delta_bias"].double()
    if s["softplus"]:
        delta = torch.logaddexp(delta, torch.zeros_like(delta))
    per = s["D"] // s["G"]
    h = torch.exp(delta[..., None] * s["A"].double()) * h + (delta * x)[..., None] * Bm.repeat_interleave(per, -2)
    y = torch.einsum("bcs,bcs->bc", h, Cm.repeat_interleave(per, -2))
    if s["D_"] is not None:
        y = y + s["D_"].double() * x
    if z is not None:
        y = y * z / (1 + torch.exp(-z))
    return h, y


def _exact_scan(s):
    B, N = s["B"], s["N"]
    lens = s["lens"] if s["lens"] else [N] * B
    h = s["h"].double() if s["h"] is not None else torch.zeros(B, s["D"], s["n"], device=s["x"].device, dtype=torch.float64)
    out = s["out"].double()
    for t in range(max(lens)):
        on = [b for b in range(B) if lens[b] > t]
        sel = slice(None) if len(on) == B else on
        z = s["z"][sel, t].double() if s["z"] is not None else None
        h[sel], out[sel, t] = _exact_recurrence(s, h[sel], s["x"][sel, t].double(), s["delta"][sel, t].double(),
                                                s["B_"][sel, t].double(), s["C"][sel, t].double(), z)
    return out, h


def _exact_step(s):
    h, y = _exact_recurrence(s, s["h"].double(), s["x"].double(), s["delta"].double(), s["B_"].double(),
                             s["C"].double(), s["z"].double() if s["z"] is not None else None)
    return y, h


def _exact_attention(q, qpos, k, v, kpos, window, sinks):
    """One head: queries at qpos over keys at kpos, in slices of queries."""
    o = torch.zeros(q.shape[0], v.shape[1], device=q.device, dtype=torch.float64)
    for i in range(0, q.shape[0], 2048):
        p = qpos[i:i + 2048, None]
        see = (kpos >= 0) & (kpos <= p) & ((kpos > p - window) | (kpos < sinks))
        w = (q[i:i + 2048].double() @ k.double().T / math.sqrt(q.shape[1])).masked_fill(~see, -math.inf)
        o[i:i + 2048] = torch.softmax(w, -1) @ v.double()
    return o


def _exact_bounded(s):
    """Both attention operators: decode is a prompt of one token."""
    one = s["op"] == "decode"
    dev, W, S, g = s["q"].device, s["window"], s["sinks"], s["Hq"] // s["Hkv"]
    q, k, v = (t[:, :, None] if one else t for t in (s["q"], s["k"], s["v"]))
    out = (s["out"][:, :, None] if one else s["out"]).double()
    cached = s["k_cache"] is not None
    kc, vc = (s["k_cache"].double(), s["v_cache"].double()) if cached else (None, None)
    for b, p0 in enumerate(s["pos_host"]):
        n = 1 if one else s["lens"][b] if s["lens"] else s["N"]
        kpos = torch.arange(p0, p0 + n, device=dev)
        place = {}
        if cached:
            held = [p for p in list(range(min(S, p0))) + list(range(max(S, p0 - W), p0))]
            slots = torch.tensor([p if p < S else S + (p - S) % W for p in held], device=dev, dtype=torch.long)
            allpos = torch.cat([torch.tensor(held, device=dev, dtype=torch.long), kpos])
            for i in range(n):
                place[p0 + i if p0 + i < S else S + (p0 + i - S) % W] = i
        else:
            allpos = kpos
        for j in range(s["Hkv"]):
            keys, vals = k[b, j, :n], v[b, j, :n]
            if cached:
                keys, vals = torch.cat([s["k_cache"][b, j, slots], keys]), torch.cat([s["v_cache"][b, j, slots], vals])
            for h in range(j * g, j * g + g):
                out[b, h, :n] = _exact_attention(q[b, h, :n], kpos, keys, vals, allpos, W, S)
        if place:
            to, src = (torch.tensor(list(t), device=dev) for t in (place.keys(), place.values()))
            kc[b, :, to], vc[b, :, to] = k[b, :, src].double(), v[b, :, src].double()
    out = out[:, :, 0] if one else out
    return (out, kc, vc) if cached else out


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "step": _exact_step, "window": _exact_bounded,
            "decode": _exact_bounded}[case["op"]](s)
