"""Cases of the 16-bit operators that stand beside the quantized linears.

Three operators of a world-action model step:

* ``attention``   queries of a batch over one observation prefix that the whole
  batch shares, joined with each sequence's own keys and values;
* ``linear``      a bf16 product with bias, activation and residual in its
  epilogue, for the layers that are kept out of quantization;
* ``group_norm``  group normalisation with an activation on channels-last
  features, as a video autoencoder applies it.

``run`` computes them either in plain torch operations in 32 bits (``own`` is
False) or through this package's operators (``own`` is True); ``exact`` gives
the same results from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda"


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------
def _attention(name, B, T, Hq, Hkv, D, P, S, ragged, keep, causal):
    return {"name": name, "op": "attention", "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "P": P, "S": S,
            "ragged": ragged, "keep": keep, "causal": causal}


def _linear(name, M, N, K, act, bias, residual, y):
    return {"name": name, "op": "linear", "M": M, "N": N, "K": K, "act": act, "bias": bias, "residual": residual,
            "y": y}


def _group_norm(name, N, S, C, G, dtype, act):
    return {"name": name, "op": "group_norm", "N": N, "S": S, "C": C, "G": G, "dtype": dtype, "act": act}


def listed():
    return [
        # one sequence, one new token, a short observation: the latency of a call
        _attention("attn_token", 1, 1, 8, 1, 64, 300, 17, False, False, True),
        # a serving batch that decodes one token each over a long common prefix
        _attention("attn_decode", 64, 1, 32, 8, 128, 8192, 256, True, False, True),
        # sampled action chunks, all tokens of a chunk see each other; absent
        # cameras are masked out of the observation
        _attention("attn_chunk", 8, 50, 16, 4, 128, 2040, 50, False, True, False),
        # one KV head of width 256, few rows: the long axis is all there is to split
        _attention("attn_wide_head", 2, 13, 8, 1, 256, 5001, 130, True, True, True),
        # the largest: many candidate rollouts over a long video context
        _attention("attn_rollouts", 16, 64, 32, 8, 128, 16384, 192, True, False, True),
        # a 2048-wide projection of one token, 32-bit residual stream
        _linear("linear_token", 1, 2048, 2048, "none", "f32", True, "f32"),
        # the batch-1 down projection (64 action tokens), 16-bit residual stream
        _linear("linear_step", 64, 2048, 8192, "none", "bf16", True, "bf16"),
        # prefill gate and up projections of 512 tokens with their SwiGLU
        _linear("linear_gated", 512, 8192, 2048, "swiglu", "none", False, "bf16"),
        # the video-latent projection, 4096 tokens, bias and GELU
        _linear("linear_video", 4096, 5120, 5120, "gelu_tanh", "f32", False, "bf16"),
        # low-resolution features of a video autoencoder
        _group_norm("norm_latent", 1, 1560, 384, 32, "bf16", "silu"),
        # odd widths (five channels a group), 32-bit features, no activation
        _group_norm("norm_odd", 3, 4095, 40, 8, "f32", "none"),
        # full-resolution features: four frames of 480 x 832, three channels a group
        _group_norm("norm_frames", 1, 1597440, 96, 32, "bf16", "silu"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["attention", "linear", "group_norm"])
    top = {"attention": "attn_rollouts", "linear": "linear_video", "group_norm": "norm_frames"}[op]
    limit = next(work(c) for c in listed() if c["name"] == top)   # no dearer than the largest of its kind
    while True:
        if op == "attention":
            Hkv = rng.choice([1, 2, 4, 5, 8])
            case = {"op": op, "B": _log_int(rng, 1, 64), "T": rng.choice([1, 1, _log_int(rng, 1, 64)]),
                    "Hq": Hkv * rng.choice([1, 2, 3, 4, 7, 8]), "Hkv": Hkv, "D": rng.choice([64, 128, 128, 256]),
                    "P": _log_int(rng, 1, 16384), "S": _log_int(rng, 1, 320), "ragged": rng.random() < 0.5,
                    "keep": rng.random() < 0.5, "causal": rng.random() < 0.5}
        elif op == "linear":
            case = {"op": op, "M": _log_int(rng, 1, 4096), "N": _log_int(rng, 64, 8192),
                    "K": 8 * _log_int(rng, 8, 1024),
                    "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"]),
                    "bias": rng.choice(["none", "f32", "bf16"]), "residual": rng.random() < 0.5,
                    "y": rng.choice(["bf16", "bf16", "f32"])}
        else:
            G = rng.choice([1, 4, 8, 16, 32])
            case = {"op": op, "N": rng.randint(1, 4), "S": _log_int(rng, 64, 400000),
                    "C": G * rng.choice([1, 2, 3, 5, 8, 12, 16, 20]), "G": G, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                    "act": rng.choice(["silu", "silu", "none"])}
            if case["C"] < 16:
                continue
        if all(work(case)[k] <= limit[k] for k in limit):
            return case


# ----------------------------------------------------------------------------
# What a pass cannot do without
# ----------------------------------------------------------------------------
def _own_lens(c):
    """Keys of its own that each sequence holds: all S, or between half and all."""
    if not c["ragged"]:
        return [c["S"]] * c["B"]
    return [c["S"] - (b * 37) % (c["S"] // 2 + 1) for b in range(c["B"])]


def _keep_mask(c):
    """Observation keys that are present: an absent camera's span and the
    padding at the end are not."""
    P = c["P"]
    keep = [True] * P
    if c["keep"]:
        for p in range(P * 3 // 8, P // 2):
            keep[p] = False
        for p in range(P - P // 50, P):
            keep[p] = False
    return keep


def work(case):
    c = case
    if c["op"] == "attention":
        rows = c["T"] * c["Hq"]
        kept = sum(_keep_mask(c))
        lens = _own_lens(c)
        seen = 0                                   # query-key pairs per query head
        for n in lens:
            seen += c["T"] * kept
            if c["causal"]:
                seen += sum(max(0, min(n, n - c["T"] + t + 1)) for t in range(c["T"]))
            else:
                seen += c["T"] * n
        kv = 2 * 2 * c["Hkv"] * c["D"] * (kept + sum(lens))
        return {"bytes": kv + 2 * 2 * c["B"] * rows * c["D"], "flops": 4 * c["Hq"] * c["D"] * seen}
    if c["op"] == "linear":
        nw = c["N"] * (2 if c["act"] == "swiglu" else 1)
        ysz = 4 if c["y"] == "f32" else 2
        byt = 2 * c["K"] * (c["M"] + nw) + c["M"] * c["N"] * ysz * (2 if c["residual"] else 1)
        byt += nw * {"none": 0, "f32": 4, "bf16": 2}[c["bias"]]
        return {"bytes": byt, "flops": 2 * c["M"] * nw * c["K"]}
    n = c["N"] * c["S"] * c["C"]
    return {"bytes": 2 * n * (4 if c["dtype"] == "f32" else 2) + 8 * c["C"], "flops": 10 * n}


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def _inputs(case, seed):
    c = case
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)

    st = {"case": c}
    if c["op"] == "attention":
        q = randn(c["B"], c["T"], c["Hq"], c["D"]) * 1.5
        kp, ko = randn(c["P"], c["Hkv"], c["D"]), randn(c["B"], c["S"], c["Hkv"], c["D"])
        kp[:4] += 0.5 * q[0, 0, :c["Hkv"]]         # a few observation keys that draw more weight
        st["q"] = q.bfloat16()
        st["kp"], st["vp"] = kp.bfloat16(), randn(c["P"], c["Hkv"], c["D"]).bfloat16()
        st["ko"], st["vo"] = ko.bfloat16(), randn(c["B"], c["S"], c["Hkv"], c["D"]).bfloat16()
        st["own_len"] = torch.tensor(_own_lens(c), dtype=torch.int32, device=DEVICE)
        st["keep"] = torch.tensor(_keep_mask(c), dtype=torch.bool, device=DEVICE) if c["keep"] else None
    elif c["op"] == "linear":
        nw = c["N"] * (2 if c["act"] == "swiglu" else 1)
        x = randn(c["M"], c["K"])
        loud = torch.randperm(c["K"], generator=g, device=DEVICE)[:max(1, c["K"] // 128)]
        x[:, loud] *= 15.0                         # persistent outlier channels
        st["x"], st["w"] = x.bfloat16(), (randn(nw, c["K"]) * 0.02).bfloat16()
        st["bias"] = None
        if c["bias"] != "none":
            st["bias"] = (randn(nw) * 0.1).to(torch.float32 if c["bias"] == "f32" else torch.bfloat16)
        ydt = torch.float32 if c["y"] == "f32" else torch.bfloat16
        st["residual"] = randn(c["M"], c["N"]).to(ydt) if c["residual"] else None
        st["y_dtype"] = ydt
    else:
        dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
        x = randn(c["N"], c["S"], c["C"])
        x *= torch.exp(0.5 * randn(c["C"]))        # channels of unequal energy, off centre
        x += 2.0 * randn(c["C"])
        st["x"] = x.to(dt)
        st["weight"], st["bias"] = 1.0 + 0.2 * randn(c["C"]), 0.2 * randn(c["C"])
    return st


EPS = 1e-5


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        from w4a4_post_quantized_channel_amd import ops
        c = case
        st["ops"] = ops
        if c["op"] == "attention":
            st["out"] = torch.empty_like(st["q"])
            st["ws"] = ops.make_prefix_attention_workspace(c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["P"], c["S"],
                                                           device=DEVICE)
        elif c["op"] == "linear":
            st["out"] = torch.empty((c["M"], c["N"]), dtype=st["y_dtype"], device=DEVICE)
            st["ws"] = ops.make_bf16_linear_workspace(c["M"], c["N"], c["K"], c["act"], device=DEVICE)
        else:
            st["out"] = torch.empty_like(st["x"])
            st["ws"] = ops.make_group_norm_workspace(c["N"], c["S"], c["C"], c["G"], device=DEVICE)
    return st


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    c, ops = st["case"], st["ops"]
    if c["op"] == "attention":
        return ops.prefix_attention(st["q"], st["kp"], st["vp"], st["ko"], st["vo"], own_len=st["own_len"],
                                    prefix_keep=st["keep"], causal=c["causal"], out=st["out"], workspace=st["ws"])
    if c["op"] == "linear":
        return ops.bf16_linear(st["x"], st["w"], bias=st["bias"], act=c["act"], residual=st["residual"], y=st["out"],
                               workspace=st["ws"])
    return ops.group_norm_act(st["x"], c["G"], st["weight"], st["bias"], eps=EPS, act=c["act"], out=st["out"],
                              workspace=st["ws"])


def _run_plain(st):
    op = st["case"]["op"]
    return {"attention": _plain_attention, "linear": _plain_linear, "group_norm": _plain_group_norm}[op](st)


def _plain_attention(st):
    c = st["case"]
    B, T, Hq, Hkv, D, P, S = (c[k] for k in ("B", "T", "Hq", "Hkv", "D", "P", "S"))
    G = Hq // Hkv
    # the rows of a KV head: every query of the batch that reads it
    q = st["q"].float().view(B, T, Hkv, G, D).permute(2, 0, 1, 3, 4).contiguous()
    q = q * (1.0 / math.sqrt(D))
    kp = st["kp"].float().permute(1, 2, 0).contiguous()
    vp = st["vp"].float().permute(1, 0, 2).contiguous()
    sp = torch.matmul(q.view(Hkv, B * T * G, D), kp)
    if st["keep"] is not None:
        sp = torch.where(st["keep"], sp, -math.inf)
    ko = st["ko"].float().permute(2, 0, 3, 1).contiguous()
    vo = st["vo"].float().permute(2, 0, 1, 3).contiguous()
    so = torch.matmul(q.view(Hkv, B, T * G, D), ko).view(Hkv, B, T, G, S)
    last = st["own_len"].view(B, 1).expand(B, T)
    if c["causal"]:
        last = last - T + 1 + torch.arange(T, device=q.device).view(1, T)
    seen = torch.arange(S, device=q.device) < last.unsqueeze(-1)
    so = torch.where(seen.view(1, B, T, 1, S), so, -math.inf).view(Hkv, B * T * G, S)
    m = torch.maximum(sp.amax(-1, keepdim=True), so.amax(-1, keepdim=True))
    m = torch.where(m > -math.inf, m, 0.0)
    pp, po = torch.exp(sp - m), torch.exp(so - m)
    total = pp.sum(-1, keepdim=True) + po.sum(-1, keepdim=True)
    out = torch.matmul(pp, vp)
    out += torch.matmul(po.view(Hkv, B, T * G, S), vo).view(Hkv, B * T * G, D)
    out = torch.where(total > 0, out / total, 0.0)
    return out.view(Hkv, B, T, G, D).permute(1, 2, 0, 3, 4).reshape(B, T, Hq, D).bfloat16()


def _plain_linear(st):
    c = st["case"]
    z = torch.matmul(st["x"].float(), st["w"].float().t())
    if st["bias"] is not None:
        z = z + st["bias"].float()
    act = c["act"]
    if act == "relu":
        z = torch.clamp(z, min=0.0)
    elif act == "gelu":
        z = 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        z = 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    elif act == "silu":
        z = z / (1.0 + torch.exp(-z))
    elif act == "swiglu":
        gate, up = z[:, :c["N"]], z[:, c["N"]:]
        z = gate / (1.0 + torch.exp(-gate)) * up
    if st["residual"] is not None:
        z = z + st["residual"].float()
    return z.to(st["y_dtype"])


def _plain_group_norm(st):
    c = st["case"]
    x = st["x"].float().view(c["N"], c["S"], c["G"], c["C"] // c["G"])
    mean = x.mean(dim=(1, 3), keepdim=True)
    d = x - mean
    y = d / torch.sqrt((d * d).mean(dim=(1, 3), keepdim=True) + EPS)
    y = y.view(c["N"], c["S"], c["C"]) * st["weight"] + st["bias"]
    if c["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    return y.to(st["x"].dtype)


# ----------------------------------------------------------------------------
# The definitions in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    st = _inputs(case, seed)
    c = case
    if c["op"] == "attention":
        return _exact_attention(st)
    if c["op"] == "linear":
        out = torch.empty((c["M"], c["N"]), dtype=torch.float64, device=DEVICE)
        x, w = st["x"].double(), st["w"].double()
        for n0 in range(0, c["N"], 2048):          # columns in slices
            n1 = min(c["N"], n0 + 2048)

            def product(lo, hi):
                z = x @ w[lo:hi].t().contiguous()
                return z if st["bias"] is None else z + st["bias"][lo:hi].double()

            z = product(n0, n1)
            if c["act"] == "relu":
                z = z.clamp(min=0)
            elif c["act"] == "gelu":
                z = z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
            elif c["act"] == "gelu_tanh":
                z = z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
            elif c["act"] == "silu":
                z = z * torch.sigmoid(z)
            elif c["act"] == "swiglu":
                z = z * torch.sigmoid(z) * product(c["N"] + n0, c["N"] + n1)
            if st["residual"] is not None:
                z = z + st["residual"][:, n0:n1].double()
            out[:, n0:n1] = z
        return out
    out = torch.empty((c["N"], c["S"], c["C"]), dtype=torch.float64, device=DEVICE)
    width = c["C"] // c["G"]
    for n in range(c["N"]):                        # one group of one sample at a time
        for k in range(c["G"]):
            ch = slice(k * width, (k + 1) * width)
            x = st["x"][n, :, ch].double()
            var, mean = torch.var_mean(x, unbiased=False)
            y = (x - mean) * torch.rsqrt(var + EPS) * st["weight"][ch].double() + st["bias"][ch].double()
            out[n, :, ch] = y * torch.sigmoid(y) if c["act"] == "silu" else y
    return out


def _exact_attention(st):
    c = st["case"]
    B, T, Hq, Hkv, D, P, S = (c[k] for k in ("B", "T", "Hq", "Hkv", "D", "P", "S"))
    G = Hq // Hkv
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device=DEVICE)
    lens = _own_lens(c)
    pos = torch.arange(S, device=DEVICE)
    for b in range(B):
        for h in range(Hkv):                       # one sequence and KV head at a time: keys side by side
            k = torch.cat([st["kp"][:, h], st["ko"][b, :, h]]).double()
            v = torch.cat([st["vp"][:, h], st["vo"][b, :, h]]).double()
            q = st["q"][b, :, h * G:(h + 1) * G].double().reshape(T * G, D)
            s = (q @ k.t().contiguous()).view(T, G, P + S) / math.sqrt(D)
            blocked = torch.zeros((T, P + S), dtype=torch.bool, device=DEVICE)
            if st["keep"] is not None:
                blocked[:, :P] = ~st["keep"]
            for t in range(T):
                end = lens[b] - (T - 1 - t) if c["causal"] else lens[b]
                blocked[t, P:] = pos >= end
            s = s.masked_fill(blocked.unsqueeze(1), -math.inf)
            p = torch.softmax(s, dim=-1)
            p = torch.nan_to_num(p, nan=0.0)       # a row that sees no key is zero
            out[b, :, h * G:(h + 1) * G] = (p.view(T * G, P + S) @ v).view(T, G, D)
    return out
