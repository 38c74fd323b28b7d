"""Cases of the operators around a 4-bit key/value cache.

Four operators of a video world model's block, between its quantized linears:

* ``attention``   queries over a paged cache of keys and values held in NVFP4;
* ``cache``       new keys and values quantised into that cache as they are
  written, and read back;
* ``rotary``      rotary positions with one to three axes on queries and keys;
* ``gated_norm``  the gated residual of a block fused with the norm behind its
  output and the modulated norm in front of the next block.

``run`` computes them either in plain torch operations (``own`` is False; in 32
bits, angles in 64) or through this package's operators (``own`` is True);
``exact`` gives the same results from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------
def _attention(name, B, T, Hq, Hkv, D, L, page, ragged, absent, causal):
    return {"name": name, "op": "attention", "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "L": L, "page": page,
            "ragged": ragged, "absent": absent, "causal": causal}


def _cache(name, M, H, D, page, dtype):
    return {"name": name, "op": "cache", "M": M, "H": H, "D": D, "page": page, "dtype": dtype}


def _rotary(name, M, Hq, Hk, D, axes, interleaved, dtype, far):
    return {"name": name, "op": "rotary", "M": M, "Hq": Hq, "Hk": Hk, "D": D, "axes": axes, "interleaved": interleaved,
            "dtype": dtype, "far": far}


def _gated(name, M, C, rows, kind, post, gate, x, h, y):
    return {"name": name, "op": "gated_norm", "M": M, "C": C, "rows": rows, "kind": kind, "post": post, "gate": gate,
            "x": x, "h": h, "y": y}


def listed():
    return [
        # one robot, one new token, a short history: the latency of a call
        _attention("attn4_token", 1, 1, 8, 1, 64, 317, 16, False, False, True),
        # a serving batch that decodes one token each over long histories
        _attention("attn4_decode", 64, 1, 32, 8, 128, 8192, 64, True, False, True),
        # sampled action chunks over an observation with an evicted camera
        _attention("attn4_chunk", 8, 50, 16, 4, 128, 2090, 16, False, True, False),
        # one KV head of width 256, few rows over a long history
        _attention("attn4_wide_head", 2, 13, 8, 1, 256, 5131, 32, True, True, True),
        # the largest: a latent frame of 30 x 52 tokens, with and without
        # guidance, that sees the seven frames before it and itself
        _attention("attn4_frame", 2, 1560, 16, 16, 128, 12480, 64, False, False, False),
        # one token of each sequence of a batch
        _cache("cache_step", 64, 8, 128, 64, "bf16"),
        # eight latent frames at once
        _cache("cache_frames", 12480, 16, 128, 64, "bf16"),
        # the queries and key of an action chunk, positions along one axis
        _rotary("rotary_chunk", 400, 16, 4, 128, 1, False, "bf16", False),
        # eight latent frames: time, height and width
        _rotary("rotary_frames", 12480, 16, 16, 128, 3, True, "bf16", False),
        # 64 action tokens of one sample, 16-bit residual stream
        _gated("gated_step", 64, 2048, 1, "rms", True, True, "bf16", "bf16", "bf16"),
        # a width that is no multiple of eight, 32-bit throughout
        _gated("gated_odd", 777, 1155, 3, "layer", False, True, "f32", "f32", "f32"),
        # four latent frames of two samples at the video width, 32-bit residual
        # stream, modulated frame by frame
        _gated("gated_frames", 12480, 5120, 8, "layer", False, True, "f32", "bf16", "bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["attention", "attention", "cache", "rotary", "gated_norm"])
    top = [work(c) for c in listed() if c["op"] == op]
    top = {k: max(w[k] for w in top) for k in ("bytes", "flops")}
    while True:
        if op == "attention":
            Hkv = rng.choice([1, 2, 4, 5, 8])
            case = {"op": op, "B": _log_int(rng, 1, 64), "T": rng.choice([1, 1, _log_int(rng, 1, 64), _log_int(rng, 1, 1560)]),
                    "Hq": Hkv * rng.choice([1, 2, 3, 4, 7, 8]), "Hkv": Hkv, "D": rng.choice([64, 128, 128, 256]),
                    "L": _log_int(rng, 1, 16384), "page": rng.choice([16, 32, 64, 128]), "ragged": rng.random() < 0.5,
                    "absent": rng.random() < 0.5, "causal": rng.random() < 0.5}
        elif op == "cache":
            case = {"op": op, "M": _log_int(rng, 1, 12480), "H": rng.choice([1, 2, 4, 5, 8, 16]),
                    "D": rng.choice([64, 128, 128, 256]), "page": rng.choice([16, 32, 64, 128]),
                    "dtype": rng.choice(["bf16", "bf16", "f32"])}
        elif op == "rotary":
            case = {"op": op, "M": _log_int(rng, 1, 12480), "Hq": rng.choice([1, 4, 5, 8, 16, 32]), "Hk": rng.choice([1, 2, 4, 8, 16]),
                    "D": rng.choice([64, 72, 128, 128, 256]), "axes": rng.choice([1, 2, 3]), "interleaved": rng.random() < 0.5,
                    "dtype": rng.choice(["bf16", "bf16", "f32"]), "far": rng.random() < 0.3}
        else:
            rows = rng.choice([1, 1, 2, 3, 8])
            case = {"op": op, "M": rows * _log_int(rng, 1, 4096), "C": rng.choice([_log_int(rng, 64, 8192), 8 * _log_int(rng, 8, 1024)]),
                    "rows": rows, "kind": rng.choice(["layer", "rms"]), "post": rng.random() < 0.5,
                    "gate": rng.random() < 0.7, "x": rng.choice(["bf16", "f32"]), "h": rng.choice(["bf16", "bf16", "f32"]),
                    "y": rng.choice(["bf16", "bf16", "f32"])}
        w = work(case)
        if sum(w[k] / top[k] for k in top) <= 1.0:     # no dearer than the largest of its kind
            return case


# ----------------------------------------------------------------------------
# What a pass cannot do without
# ----------------------------------------------------------------------------
def _lens(c):
    """Keys of each sequence: all L, or between half and all."""
    if not c["ragged"]:
        return [c["L"]] * c["B"]
    return [c["L"] - (b * 137) % (c["L"] // 2 + 1) for b in range(c["B"])]


def _pages(c):
    return -(-c["L"] // c["page"])


def _present(c):
    """Which pages of a sequence's history are held: an evicted camera's are not."""
    P = _pages(c)
    return [not (c["absent"] and P * 3 // 8 <= p < P // 2) for p in range(P)]


def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    c = case
    if c["op"] == "attention":
        present, page, T = _present(c), c["page"], c["T"]
        below = [0]                                    # held keys below a page's start
        for p in present:
            below.append(below[-1] + page * p)

        def held(n):                                   # held keys among the first n
            p, r = divmod(max(0, n), page)
            return below[p] + (r if r and present[p] else 0)

        seen = keys = 0
        for n in _lens(c):
            keys += held(n)
            seen += sum(held(n - T + t + 1) for t in range(T)) if c["causal"] else T * held(n)
        row = c["D"] // 2 + c["D"] // 16
        return {"bytes": 2 * keys * c["Hkv"] * row + 2 * 2 * c["B"] * T * c["Hq"] * c["D"],
                "flops": 4 * c["Hq"] * c["D"] * seen}
    if c["op"] == "cache":
        n = 2 * c["M"] * c["H"] * c["D"]
        return {"bytes": n * _size(c["dtype"]) * 2 + n // 2 + n // 16, "flops": 8 * n}
    if c["op"] == "rotary":
        n = c["M"] * (c["Hq"] + c["Hk"]) * c["D"]
        return {"bytes": 2 * n * _size(c["dtype"]) + 4 * c["M"] * c["axes"], "flops": 3 * n}
    n = c["M"] * c["C"]
    return {"bytes": n * (2 * _size(c["x"]) + _size(c["h"]) + _size(c["y"])), "flops": 12 * n}


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
# the static scale of a cache, a power of two above amax / (6 * 448)
K_SCALE, V_SCALE = 2.0 ** -8, 2.0 ** -9
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _quantise(x, g):
    """(E2M1 codes, E4M3 codes) of x in blocks of 16: e = E4M3(amax / 6 / g), c = E2M1(x / (e g))."""
    b = x.float().view(*x.shape[:-1], x.shape[-1] // 16, 16)
    v = (b.abs().amax(-1, keepdim=True) / 6.0) / g
    E = torch.clamp(torch.frexp(v)[1] - 1, min=-6)
    e = (E + 6) * 8 + torch.round(torch.ldexp(v, 3 - E)).int()
    e = torch.where(v > 0, torch.clamp(e, max=126), 0)
    s = _e4m3(e) * g
    u = torch.where(s > 0, b / torch.where(s > 0, s, 1.0), 0.0)
    a = u.abs()
    c = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
         + (a >= 3.5).int() + (a > 5.0).int())
    return torch.where((u < 0) & (c > 0), c + 8, c), e


def _e4m3(e):
    E, m = e // 8, (e % 8).float()
    return torch.where(E > 0, torch.ldexp(1.0 + m / 8, E - 7), m * 2.0 ** -9)


def _packed(x, g):
    c, e = _quantise(x, g)
    c = c.view(x.shape).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), e.squeeze(-1).to(torch.uint8)


def _unpacked(codes, scales, g):
    """fp32 values of packed codes [..., D / 2] and scales [..., D / 16]."""
    one = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    both = torch.stack([one.repeat(16), one.repeat_interleave(16)], dim=1)      # of a byte
    v = both[codes.long()].view(*codes.shape[:-1], scales.shape[-1], 16)
    s = _e4m3(torch.arange(128, dtype=torch.int32, device=codes.device))[scales.long()] * g
    return (v * s.unsqueeze(-1)).view(*codes.shape[:-1], codes.shape[-1] * 2)


def _sections(c):
    """Pairs of each axis: time first, then height and width, which are equal."""
    pairs = c["D"] // 2
    if c["axes"] == 3:
        return [pairs - 2 * (pairs // 3), pairs // 3, pairs // 3]
    return [pairs - pairs // 2, pairs // 2] if c["axes"] == 2 else [pairs]


THETA = 10000.0


def _inputs(case, seed):
    c = case
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)

    st = {"case": c}
    if c["op"] == "attention":
        B, Hkv, D, page, P = c["B"], c["Hkv"], c["D"], c["page"], _pages(c)
        n = B * P + 3                                  # some pages belong to nobody
        st["q"] = (randn(B, c["T"], c["Hq"], D) * 1.5).bfloat16()
        loud = torch.exp(0.4 * randn(Hkv, 1, D))       # channels of unequal energy
        for name, scale in (("k", K_SCALE), ("v", V_SCALE)):
            parts = []
            for n0 in range(0, n, 2048):
                x = randn(min(n, n0 + 2048) - n0, Hkv, page, D)
                parts.append(_packed(x * loud if name == "k" else x, scale))
            st[name + "_codes"] = torch.cat([p[0] for p in parts])
            st[name + "_scales"] = torch.cat([p[1] for p in parts])
        table = torch.randperm(n, generator=g, device=DEVICE)[:B * P].view(B, P).int()
        present = torch.tensor(_present(c), device=DEVICE)
        st["table"] = torch.where(present, table, -1).int()
        st["lens"] = torch.tensor(_lens(c), dtype=torch.int32, device=DEVICE)
    elif c["op"] == "cache":
        M, H, D, page = c["M"], c["H"], c["D"], c["page"]
        dt = _dtype(c["dtype"])
        loud = torch.exp(0.7 * randn(H, D))
        st["k"], st["v"] = (randn(M, H, D) * loud).to(dt), randn(M, H, D).to(dt)
        st["n_pages"] = -(-M // page) + 2
        st["slots"] = torch.randperm(st["n_pages"] * page, generator=g, device=DEVICE)[:M].int()
        if M > 64:                                     # tokens of a prompt fill pages in order
            st["slots"] = st["slots"].sort().values
    elif c["op"] == "rotary":
        M, dt = c["M"], _dtype(c["dtype"])
        st["q"], st["k"] = randn(M, c["Hq"], c["D"]).to(dt), randn(M, c["Hk"], c["D"]).to(dt)
        m = torch.arange(M, device=DEVICE) + int(torch.randint(0, 512, (1,), generator=g, device=DEVICE))
        if c["far"]:
            m = m + 1000000
        axes = [m] if c["axes"] == 1 else [m // 1560, m % 1560] if c["axes"] == 2 else [m // 1560, m // 52 % 30, m % 52]
        st["pos"] = torch.stack(axes, dim=1).int()
        st["freq"] = torch.tensor([THETA ** (-i / s) for s in _sections(c) for i in range(s)], dtype=torch.float64,
                                  device=DEVICE)
    else:
        M, C, R = c["M"], c["C"], c["rows"]
        st["x"] = (randn(M, C) * torch.exp(0.5 * randn(C)) + 0.5 * randn(C)).to(_dtype(c["x"]))
        st["h"] = (randn(M, C) * torch.exp(0.5 * randn(C))).to(_dtype(c["h"]))
        mod = randn(R, 3, C) * 0.3                     # shift, scale and gate of a timestep embedding
        st["shift"], st["scale"], st["gate"] = mod[:, 0], mod[:, 1], mod[:, 2] if c["gate"] else None
        st["post"] = 1.0 + 0.2 * randn(C) if c["post"] else None
        st["weight"] = 1.0 + 0.2 * randn(C) if c["kind"] == "rms" else None
        st["alpha"] = 1.0
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        from w4a4_post_quantized_channel_amd import ops
        c = case
        st["ops"] = ops
        if c["op"] == "attention":
            st["cache"] = ops.KVCache(st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"], K_SCALE, V_SCALE)
            st["out"] = torch.empty_like(st["q"])
            st["ws"] = ops.make_cache_attention_workspace(c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["L"], device=DEVICE)
        elif c["op"] == "cache":
            st["cache"] = ops.make_kv_cache(st["n_pages"], c["page"], c["H"], c["D"], K_SCALE, V_SCALE, device=DEVICE)
            st["k_out"], st["v_out"] = torch.empty_like(st["k"]), torch.empty_like(st["v"])
        elif c["op"] == "rotary":
            st["table"] = ops.make_rotary_table(_sections(c), THETA, device=DEVICE)
            st["q_out"], st["k_out"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])
        else:
            st["x_out"] = torch.empty_like(st["x"])
            st["y"] = torch.empty(st["x"].shape, dtype=_dtype(c["y"]), device=DEVICE)
    return st


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    c, ops = st["case"], st["ops"]
    if c["op"] == "attention":
        return ops.cache_attention(st["q"], st["cache"], st["table"], st["lens"], causal=c["causal"], max_len=c["L"],
                                   out=st["out"], workspace=st["ws"])
    if c["op"] == "cache":
        ops.cache_append(st["cache"], st["k"], st["v"], st["slots"])
        return ops.cache_read(st["cache"], st["slots"], k=st["k_out"], v=st["v_out"])
    if c["op"] == "rotary":
        return ops.rotary_axes(st["q"], st["k"], st["pos"], st["table"], interleaved=c["interleaved"], q_out=st["q_out"],
                               k_out=st["k_out"])
    return ops.gated_norm(st["x"], st["h"], gate=st["gate"], alpha=st["alpha"], post_weight=st["post"], kind=c["kind"],
                          weight=st["weight"], scale=st["scale"], shift=st["shift"], eps=EPS, x_out=st["x_out"], y=st["y"])


def _run_plain(st):
    return {"attention": _plain_attention, "cache": _plain_cache, "rotary": _plain_rotary,
            "gated_norm": _plain_gated_norm}[st["case"]["op"]](st)


def _plain_attention(st):
    c = st["case"]
    B, T, Hq, Hkv, D = (c[k] for k in ("B", "T", "Hq", "Hkv", "D"))
    G, P, page = Hq // Hkv, st["table"].shape[1], c["page"]
    at = st["table"].clamp(min=0).long()

    def keys(codes, scales, g):                        # [B, Hkv, P * page, D]
        x = _unpacked(codes[at], scales[at], g)
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, P * page, D)

    k, v = keys(st["k_codes"], st["k_scales"], K_SCALE), keys(st["v_codes"], st["v_scales"], V_SCALE)
    q = st["q"].float().view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    s = torch.matmul(q * (1.0 / math.sqrt(D)), k.transpose(2, 3).contiguous())
    pos = torch.arange(P * page, device=q.device)
    last = st["lens"].view(B, 1).expand(B, T)
    if c["causal"]:
        last = last - T + 1 + torch.arange(T, device=q.device)
    seen = (pos < last.unsqueeze(-1)) & (st["table"] >= 0).repeat_interleave(page, dim=1).view(B, 1, P * page)
    s = torch.where(seen.view(B, 1, T, 1, P * page), s.view(B, Hkv, T, G, P * page), -math.inf)
    s = s.view(B, Hkv, T * G, P * page)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m > -math.inf, m, 0.0))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v)
    out = torch.where(total > 0, out / total, 0.0)     # a query that sees nothing is zero
    return out.view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D).bfloat16()


def _plain_cache(st):
    out = []
    for x, g in ((st["k"], K_SCALE), (st["v"], V_SCALE)):
        codes, scales = _packed(x, g)
        out.append(_unpacked(codes, scales, g).to(x.dtype))
    return out


def _plain_rotary(st):
    c = st["case"]
    axis = torch.tensor([a for a, s in enumerate(_sections(c)) for _ in range(s)], device=st["pos"].device)
    angle = st["pos"].double()[:, axis] * st["freq"]
    cos, sin = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    out = []
    for x in (st["q"], st["k"]):
        if c["interleaved"]:
            a, b = x[..., 0::2].float(), x[..., 1::2].float()
            y = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).view(x.shape)
        else:
            a, b = x[..., :c["D"] // 2].float(), x[..., c["D"] // 2:].float()
            y = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
        out.append(y.to(x.dtype))
    return out


def _plain_gated_norm(st):
    c = st["case"]
    M, C, R = c["M"], c["C"], c["rows"]
    u = st["h"].float()
    if st["post"] is not None:
        u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + EPS) * st["post"]
    u = u.view(R, M // R, C)
    if st["gate"] is not None:
        u = u * st["gate"].unsqueeze(1)
    x = st["alpha"] * st["x"].float().view(R, M // R, C) + u
    d = x - x.mean(-1, keepdim=True) if c["kind"] == "layer" else x
    y = d / torch.sqrt((d * d).mean(-1, keepdim=True) + EPS)
    if st["weight"] is not None:
        y = y * st["weight"]
    y = y * (1.0 + st["scale"].unsqueeze(1)) + st["shift"].unsqueeze(1)
    return x.view(M, C).to(st["x"].dtype), y.view(M, C).to(_dtype(c["y"]))


# ----------------------------------------------------------------------------
# The definitions in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    st = _inputs(case, seed)
    return {"attention": _exact_attention, "cache": _exact_cache, "rotary": _exact_rotary,
            "gated_norm": _exact_gated_norm}[case["op"]](st)


def _nearest(v, grid):
    """Index of the entry of an ascending grid that is nearest to each v >= 0, ties to the even index."""
    hi = torch.bucketize(v, grid).clamp(1, len(grid) - 1)
    lo = hi - 1
    up, down = grid[hi] - v, v - grid[lo]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def _grids():
    small = [m * 2.0 ** -9 for m in range(8)]
    e4m3 = small + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    make = lambda v: torch.tensor(v, dtype=torch.float64, device=DEVICE)  # noqa: E731
    return make(E2M1), make(e4m3[:127])


def _exact_cache(st):
    e2m1, e4m3 = _grids()
    out = []
    for x, g in ((st["k"], K_SCALE), (st["v"], V_SCALE)):
        b = x.double().view(*x.shape[:-1], -1, 16)
        s = e4m3[_nearest(b.abs().amax(-1, keepdim=True) / (6.0 * g), e4m3)] * g
        u = torch.where(s > 0, b / torch.where(s > 0, s, 1.0), 0.0)
        out.append((e2m1[_nearest(u.abs(), e2m1)] * u.sign() * s).view(x.shape))
    return out


def _exact_attention(st):
    c = st["case"]
    B, T, Hq, Hkv, D = (c[k] for k in ("B", "T", "Hq", "Hkv", "D"))
    G, page = Hq // Hkv, c["page"]
    e2m1, e4m3 = _grids()
    signed = torch.cat([e2m1, -e2m1])
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device=DEVICE)

    def rows(codes, scales, g, pages, h):
        k = codes[pages, h].reshape(-1, D // 2)
        v = torch.stack([signed[(k & 15).long()], signed[(k >> 4).long()]], dim=-1).view(-1, D // 16, 16)
        return (v * (e4m3[scales[pages, h].reshape(-1, D // 16).long()] * g).unsqueeze(-1)).view(-1, D)

    present = _present(c)
    for b, n in enumerate(_lens(c)):                   # one sequence and KV head at a time, held keys only
        held = [p for p in range(-(-n // page)) if present[p]]
        if not held:
            continue
        pages = st["table"][b, held].long()
        pos = (torch.tensor(held, device=DEVICE).unsqueeze(1) * page + torch.arange(page, device=DEVICE)).reshape(-1)
        end = torch.full((T,), n, device=DEVICE)
        if c["causal"]:
            end = end - (T - 1 - torch.arange(T, device=DEVICE))
        blocked = pos.unsqueeze(0) >= end.unsqueeze(1)
        for h in range(Hkv):
            k = rows(st["k_codes"], st["k_scales"], K_SCALE, pages, h)
            v = rows(st["v_codes"], st["v_scales"], V_SCALE, pages, h)
            q = st["q"][b, :, h * G:(h + 1) * G].double().reshape(T * G, D)
            s = (q @ k.t().contiguous()).view(T, G, -1) / math.sqrt(D)
            p = torch.softmax(s.masked_fill(blocked.unsqueeze(1), -math.inf), dim=-1)
            p = torch.nan_to_num(p, nan=0.0)
            out[b, :, h * G:(h + 1) * G] = (p.view(T * G, -1) @ v).view(T, G, D)
    return out


def _exact_rotary(st):
    c = st["case"]
    out = []
    for x in (st["q"], st["k"]):
        y = x.double().clone()
        i = 0
        for a, s in enumerate(_sections(c)):
            for j in range(s):                         # a pair at a time, as a complex number
                turn = st["pos"][:, a].double() * THETA ** (-j / s)
                turn = torch.polar(torch.ones_like(turn), turn).unsqueeze(1)
                r, w = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + c["D"] // 2)
                z = torch.complex(x[:, :, r].double(), x[:, :, w].double()) * turn
                y[:, :, r], y[:, :, w] = z.real, z.imag
                i += 1
        out.append(y)
    return out


def _exact_gated_norm(st):
    c = st["case"]
    M, C, R = c["M"], c["C"], c["rows"]
    xs = torch.empty((M, C), dtype=torch.float64, device=DEVICE)
    ys = torch.empty_like(xs)
    n = M // R
    for r in range(R):                                 # the tokens of a modulation row
        part = slice(r * n, (r + 1) * n)
        u = st["h"][part].double()
        if st["post"] is not None:
            u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS) * st["post"].double()
        if st["gate"] is not None:
            u = u * st["gate"][r].double()
        x = u + st["alpha"] * st["x"][part].double()
        if c["kind"] == "layer":
            var, mean = torch.var_mean(x, dim=-1, unbiased=False, keepdim=True)
            y = (x - mean) * torch.rsqrt(var + EPS)
        else:
            y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        if st["weight"] is not None:
            y = y * st["weight"].double()
        xs[part] = x
        ys[part] = y * (1.0 + st["scale"][r].double()) + st["shift"][r].double()
    return xs, ys
