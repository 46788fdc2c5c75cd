"""Cases and plain forms of the layer operators around the attention: the
rotary embedding, the linear layer with its epilogue and differential
attention.

`prepare` draws a case's inputs on the GPU, `run` makes one pass: with `own`
the library's entry points, without it the same mathematics in elementary
torch operations (fp32, angles in fp64).  `exact` is the definition in fp64,
written apart from the plain form.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------- cases


def _rotary(name, **kw):
    c = dict(name=name, op="rotary", dtype="bf16", B=1, S=1, H=8, H_k=8, d=128, parts=1, rot=128, layout="interleaved",
             axial=False, scaling="none", factor=1.0, original=4096, theta=10000.0, first=0, inverse=False, fused=False)
    c.update(kw)
    return c


def _linear(name, **kw):
    c = dict(name=name, op="linear", dtype="bf16", out="bf16", M=1, N=128, K=128, bias=True, act="none",
             residual=False)
    c.update(kw)
    return c


def _diff(name, **kw):
    c = dict(name=name, op="diff", dtype="bf16", B=1, H=2, H_kv=2, S_q=1, S_kv=1, d=128, norm=True, len_min=-1,
             pad_from=0, pad_to=0)
    c.update(kw)
    return c


def listed():
    return [
        # one new token of 16 sequences far into a long context, queries and keys of shared heads
        _rotary("rotary_step", B=16, S=1, H=32, H_k=8, rot=128, layout="half", scaling="yarn", factor=32.0,
                first=100000),
        # the joint sequence of a 2048x2048 image: three axes, both maps of a head, read from the fused projection
        _rotary("rotary_joint", B=2, S=16896, H=24, H_k=24, parts=2, rot=64, axial=True, fused=True),
        # the gradient's way back through a partial rotation in fp32 at an odd length
        _rotary("rotary_grad", dtype="fp32", B=2, S=4133, H=12, H_k=4, d=96, rot=64, layout="half", scaling="ntk",
                factor=4.0, inverse=True),
        # a projection for four single tokens: the weight is all there is to read
        _linear("linear_step", M=4, N=4096, K=4096, residual=True),
        # the fused q, k, v projection of a 1024x1024 image's joint sequence, two guidance branches
        _linear("linear_qkv", M=9216, N=6144, K=2048),
        # the MLP's first product with its activation, a 2048x2048 image
        _linear("linear_up", M=16896, N=8192, K=2048, act="gelu_tanh"),
        # the MLP's second product with the residual stream
        _linear("linear_down", dtype="fp16", out="fp16", M=4608, N=2048, K=8192, residual=True),
        # an odd head of a model: no size is a multiple of anything
        _linear("linear_odd", out="fp32", M=1531, N=777, K=1003, act="silu"),
        # 32 text and 16x16 image tokens
        _diff("diff_tiny", dtype="fp16", H=2, H_kv=2, S_q=288, S_kv=288, d=64),
        # a 1024x1024 image, two guidance branches of which the short prompt's text is padded
        _diff("diff_1024", B=2, H=24, H_kv=24, S_q=4608, S_kv=4608, pad_from=40, pad_to=512),
        # a 2048x2048 image, one rank's heads of a four-way split
        _diff("diff_2048", H=6, H_kv=6, S_q=16896, S_kv=16896),
        # one new query for each of 8 sequences over their caches of unequal length, shared heads
        _diff("diff_step", B=8, H=32, H_kv=8, S_q=1, S_kv=16384, len_min=2000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotary", "linear", "diff"))
    if op == "rotary":
        d = rng.choice((32, 64, 80, 96, 128, 256))
        axial = d in (64, 128) and rng.random() < 0.3
        parts = rng.choice((1, 2)) if d % 32 == 0 else 1
        rot = d // parts if axial or rng.random() < 0.5 else 2 * rng.randint(1, d // parts // 2)
        H = rng.choice((2, 6, 12, 24, 32))
        B = rng.randint(1, 4)
        return dict(_rotary("", dtype=rng.choice(("bf16", "fp16", "fp32")), B=B, S=_log(rng, 1, 16896 // B), H=H,
                            H_k=rng.choice((1, 2, H)), d=d, parts=parts, rot=rot,
                            layout=rng.choice(("interleaved", "half")), axial=axial,
                            scaling="none" if axial else rng.choice(("none", "linear", "ntk", "yarn")),
                            factor=rng.choice((2.0, 8.0, 32.0)), first=0 if axial else _log(rng, 1, 1000000),
                            inverse=rng.random() < 0.3, fused=rng.random() < 0.5))
    if op == "linear":
        odd = rng.random() < 0.3
        up = lambda n: n if odd else -(-n // 8) * 8  # noqa: E731
        dt = rng.choice(("bf16", "fp16"))
        return dict(_linear("", dtype=dt, out=rng.choice((dt, dt, "fp32")), M=_log(rng, 1, 9000),
                            N=up(_log(rng, 64, 8000)), K=up(_log(rng, 64, 4000)), bias=rng.random() < 0.7,
                            act=rng.choice(("none", "gelu", "gelu_tanh", "silu", "relu")),
                            residual=rng.random() < 0.5))
    H_kv, G = rng.choice((1, 2, 4, 6)), rng.choice((1, 1, 2, 4))
    B = rng.randint(1, 4)
    S_kv = _log(rng, 1, 16384 // B)
    S_q = 1 if rng.random() < 0.3 else _log(rng, 1, 4096 // B)
    pad = rng.random() < 0.3
    a = rng.randint(0, S_kv)
    return dict(_diff("", dtype=rng.choice(("bf16", "fp16")), B=B, H=H_kv * G, H_kv=H_kv, S_q=S_q, S_kv=S_kv,
                      d=rng.choice((64, 128)), norm=rng.random() < 0.7,
                      len_min=rng.randint(0, S_kv) if rng.random() < 0.4 else -1, pad_from=a if pad else 0,
                      pad_to=rng.randint(a, S_kv) if pad else 0))


# ---------------------------------------------------------------- inputs


_LAMBDA_INIT = 0.35
_EPS = 1e-5


def _lengths(c):
    """Keys of every batch entry: all, or spread evenly from len_min up."""
    if c["len_min"] < 0:
        return [c["S_kv"]] * c["B"]
    return [c["len_min"] + (c["S_kv"] - c["len_min"]) * b // max(1, c["B"] - 1) for b in range(c["B"])]


def _split(c):
    n = c["d"] // c["parts"]
    return (n // 4, 3 * n // 8, 3 * n // 8)


def _frequencies(c):
    """(fp64 frequencies of the pairs, factor of their cos and sin)."""
    n, f = c["rot"], c["factor"]
    pairs = lambda m: torch.arange(m // 2, dtype=torch.float64, device="cuda") / m  # noqa: E731
    if c["axial"]:
        return torch.cat([c["theta"] ** (-2 * pairs(m)) for m in _split(c)]), 1.0
    if c["scaling"] == "ntk":
        return (c["theta"] * f ** (n / max(1, n - 2))) ** (-2 * pairs(n)), 1.0
    w = c["theta"] ** (-2 * pairs(n))
    if c["scaling"] == "linear":
        return w / f, 1.0
    if c["scaling"] == "yarn":
        turns = lambda r: n * math.log(c["original"] / (r * 2 * math.pi)) / (2 * math.log(c["theta"]))  # noqa: E731
        low, high = max(0, math.floor(turns(32.0))), min(n - 1, math.ceil(turns(1.0)))
        slow = ((n * pairs(n) - low) / max(high - low, 1e-3)).clamp(0, 1)
        return w / f * slow + w * (1 - slow), 0.1 * math.log(f) + 1.0
    return w, 1.0


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s, dt: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32).to(dt)  # noqa: E731
    s = {"case": c}
    if c["op"] == "rotary":
        dt, B, S, d = _DT[c["dtype"]], c["B"], c["S"], c["d"]
        if c["fused"]:
            # q and k as they lie in the fused projection, [B, S, H + 2 H_k, d]; outputs head-major
            qkv = randn(B, S, c["H"] + 2 * c["H_k"], d, dt=dt)
            s["q"], s["k"] = qkv[:, :, :c["H"]], qkv[:, :, c["H"]:c["H"] + c["H_k"]]
            s["out"] = tuple(torch.empty(B, h, S, d, dtype=dt, device="cuda").transpose(1, 2)
                             for h in (c["H"], c["H_k"]))
        else:
            s["q"], s["k"] = randn(B, S, c["H"], d, dt=dt), randn(B, S, c["H_k"], d, dt=dt)
            s["out"] = None
        if c["axial"]:
            side = max(1, math.isqrt(S))
            i = torch.arange(S, device="cuda")
            shift = torch.randint(0, 64, (3,), generator=g, device="cuda")
            s["pos"] = (torch.stack([i // (side * side), i // side % side, i % side], 1) + shift).int().contiguous()
        else:
            start = torch.randint(c["first"], 2 * c["first"] + 1, (B, 1), generator=g, device="cuda")
            s["pos"] = (start + torch.arange(S, device="cuda")).int().contiguous()
        s["freqs"], s["scale"] = _frequencies(c)
    elif c["op"] == "linear":
        dt, odt, M, N, K = _DT[c["dtype"]], _DT[c["out"]], c["M"], c["N"], c["K"]
        s["x"] = randn(M, K, dt=dt)
        s["w"] = (torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K)).to(dt)
        s["bias"] = randn(N, dt=dt) if c["bias"] else None
        s["residual"] = randn(M, N, dt=odt) if c["residual"] else None
    else:
        dt, B, d = _DT[c["dtype"]], c["B"], c["d"]
        s["q"] = randn(B, c["H"], c["S_q"], d, dt=dt)
        s["k"] = randn(B, c["H_kv"], c["S_kv"], d, dt=dt)
        s["v"] = randn(B, c["H_kv"], c["S_kv"], d, dt=dt)
        s["lam"] = 0.1 * randn(4, c["H"], d // 2, dt=torch.float32)
        s["norm_w"] = 1 + 0.1 * randn(d, dt=torch.float32) if c["norm"] else None
        s["kv_len"] = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda") if c["len_min"] >= 0 else None
        s["key_mask"] = None
        if c["pad_to"] > c["pad_from"]:
            s["key_mask"] = torch.ones(B, c["S_kv"], dtype=torch.bool, device="cuda")
            s["key_mask"][-1, c["pad_from"]:c["pad_to"]] = False
    return s


# ---------------------------------------------------------------- one pass


def _plain_rotary(s):
    c = s["case"]
    n, parts, rot = c["d"] // c["parts"], c["parts"], c["rot"]
    pos = s["pos"].double()
    if c["axial"]:
        axes = torch.cat([torch.full((m // 2,), a, device=pos.device) for a, m in enumerate(_split(c))])
        ang = (pos[:, axes] * s["freqs"])[None]
    else:
        ang = pos[:, :, None] * s["freqs"]
    ang = -ang if c["inverse"] else ang
    cos, sin = ((f(ang) * s["scale"]).float()[:, :, None, None] for f in (torch.cos, torch.sin))
    half = c["layout"] == "half"

    def turn(x):
        y = x.float().unflatten(-1, (parts, n))
        r, rest = y[..., :rot], y[..., rot:]
        a, b = (r[..., :rot // 2], r[..., rot // 2:]) if half else (r[..., ::2], r[..., 1::2])
        u, v = a * cos - b * sin, a * sin + b * cos
        r = torch.cat([u, v], -1) if half else torch.stack([u, v], -1).flatten(-2)
        return torch.cat([r, rest], -1).flatten(-2).to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def _act(y, name):
    if name == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if name == "silu":
        return y / (1 + torch.exp(-y))
    return y.clamp(min=0) if name == "relu" else y


def _plain_linear(s):
    y = torch.matmul(s["x"].float(), s["w"].float().t())
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _act(y, s["case"]["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(_DT[s["case"]["out"]])


def _allowed(s):
    """bool [B, S_kv]: the keys that take part."""
    c = s["case"]
    ok = torch.ones(c["B"], c["S_kv"], dtype=torch.bool, device=s["k"].device)
    if s["kv_len"] is not None:
        ok = torch.arange(c["S_kv"], device=ok.device) < s["kv_len"][:, None]
    return ok if s["key_mask"] is None else ok & s["key_mask"]


def _plain_diff(s):
    c = s["case"]
    B, H, Hk, d = c["B"], c["H"], c["H_kv"], c["d"]
    q = s["q"].float().view(B, Hk, H // Hk, c["S_q"], 2, d // 2).transpose(3, 4)
    k = s["k"].float().view(B, Hk, 1, c["S_kv"], 2, d // 2).transpose(3, 4)
    ok = _allowed(s)
    v = torch.where(ok[:, None, :, None], s["v"].float(), 0.0).view(B, Hk, 1, 1, c["S_kv"], d)
    x = torch.matmul(q, k.transpose(-1, -2))
    x *= (d // 2) ** -0.5
    x.masked_fill_(~ok[:, None, None, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x -= torch.where(m == -math.inf, 0.0, m)
    x.exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / torch.where(l == 0, 1.0, l)
    lq1, lk1, lq2, lk2 = s["lam"]
    lam = torch.exp((lq1 * lk1).sum(-1)) - torch.exp((lq2 * lk2).sum(-1)) + _LAMBDA_INIT
    o = o[:, :, :, 0] - lam.view(Hk, H // Hk, 1, 1) * o[:, :, :, 1]
    if s["norm_w"] is not None:
        o = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + _EPS) * s["norm_w"] * (1 - _LAMBDA_INIT)
    lse = (m + torch.log(l)).squeeze(-1)
    o = o.reshape(B, H, c["S_q"], d).transpose(1, 2).to(torch.bfloat16)
    return o.contiguous(), lse.reshape(B, H, 2, c["S_q"]).permute(2, 0, 1, 3).contiguous()


def run(state):
    s, c = state, state["case"]
    if own:
        from diffusion_transformer_joint_jattn_b200 import jattn
        if c["op"] == "rotary":
            return jattn.rotary(s["q"], s["k"], s["pos"], s["freqs"], split=_split(c) if c["axial"] else None,
                                layout=c["layout"], parts=c["parts"], scale=s["scale"], inverse=c["inverse"],
                                out=s["out"])
        if c["op"] == "linear":
            return jattn.linear(s["x"], s["w"], s["bias"], act=c["act"], residual=s["residual"],
                                out_dtype=_DT[c["out"]])
        return jattn.fwd_diff(s["q"], s["k"], s["v"], s["lam"], _LAMBDA_INIT, norm_w=s["norm_w"], eps=_EPS,
                              kv_len=s["kv_len"], key_mask=s["key_mask"], want_lse=True)
    return {"rotary": _plain_rotary, "linear": _plain_linear, "diff": _plain_diff}[c["op"]](s)


# ---------------------------------------------------------------- work and the definition


def work(case):
    c = case
    if c["op"] == "rotary":
        n = c["B"] * c["S"] * (c["H"] + c["H_k"]) * c["d"]
        pairs = c["B"] * c["S"] * (c["H"] + c["H_k"]) * c["parts"] * (c["rot"] // 2)
        tokens = c["S"] * 3 if c["axial"] else c["B"] * c["S"]
        return {"bytes": 2 * n * _SIZE[c["dtype"]] + 4 * tokens + 8 * (c["rot"] // 2), "flops": 6 * pairs}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        size = _SIZE[c["dtype"]]
        out = M * N * _SIZE[c["out"]]
        return {"bytes": (M * K + N * K + N * c["bias"]) * size + out * (1 + c["residual"]), "flops": 2 * M * N * K}
    lens, masked = _lengths(c), max(0, c["pad_to"] - c["pad_from"])
    keys = sum(lens) - max(0, min(c["pad_to"], lens[-1]) - c["pad_from"])
    rows = c["B"] * c["H"] * c["S_q"]
    size = _SIZE[c["dtype"]]
    return {"bytes": rows * c["d"] * (size + 2) + 8 * rows + 2 * c["H_kv"] * keys * c["d"] * size
            + (c["B"] * c["S_kv"] if masked else 0),
            "flops": 6 * c["H"] * c["S_q"] * keys * c["d"]}


def _exact_rotary(s):
    c = s["case"]
    n, rot = c["d"] // c["parts"], c["rot"]
    pos = s["pos"].double().cpu()
    pos = pos.view(1, c["S"], 3) if c["axial"] else pos.view(c["B"], c["S"], 1)
    scale = 1.0
    pairs = []                                     # (first channel, second channel, position axis, frequency)
    if c["axial"]:
        at = 0
        for axis, m in enumerate(_split(c)):
            pairs += [(at + i, axis, c["theta"] ** (-2.0 * i / m)) for i in range(m // 2)]
            at += m // 2
    else:
        base, f = c["theta"], c["factor"]
        if c["scaling"] == "ntk":
            base *= f ** (rot / max(1, rot - 2))
        low = high = 0.0
        if c["scaling"] == "yarn":
            scale = 1.0 + 0.1 * math.log(f)
            bound = [rot * math.log(c["original"] / (2 * math.pi * r)) / (2 * math.log(base)) for r in (32.0, 1.0)]
            low, high = max(math.floor(bound[0]), 0), min(math.ceil(bound[1]), rot - 1)
        for i in range(rot // 2):
            w = base ** (-2.0 * i / rot)
            if c["scaling"] == "linear":
                w /= f
            if c["scaling"] == "yarn":
                t = min(1.0, max(0.0, (i - low) / max(high - low, 1e-3)))
                w = t * w / f + (1 - t) * w
            pairs.append((i, 0, w))
    sign = -1.0 if c["inverse"] else 1.0
    res = []
    for x in (s["q"], s["k"]):
        y = x.double().clone()
        for part in range(c["parts"]):
            for p, axis, w in pairs:
                i, j = (p, p + rot // 2) if c["layout"] == "half" else (2 * p, 2 * p + 1)
                i, j = part * n + i, part * n + j
                z = torch.polar(torch.tensor(scale, dtype=torch.float64), sign * pos[..., axis] * w).to(x.device)
                r = torch.complex(x[..., i].double(), x[..., j].double()) * z[..., None]
                y[..., i], y[..., j] = r.real, r.imag
        res.append(y)
    return tuple(res)


def _exact_linear(s):
    c = s["case"]
    y = s["x"].double() @ s["w"].double().T
    if c["bias"]:
        y += s["bias"].double()
    if c["act"] == "gelu":
        y = y * (1 - 0.5 * torch.special.erfc(y / math.sqrt(2)))
    elif c["act"] == "gelu_tanh":
        y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
    elif c["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif c["act"] == "relu":
        y = torch.relu(y)
    return y + s["residual"].double() if c["residual"] else y


def _exact_diff(s):
    c = s["case"]
    B, H, d = c["B"], c["H"], c["d"]
    o = torch.zeros(B, c["S_q"], H, d, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((2, B, H, c["S_q"]), -math.inf, dtype=torch.float64, device=s["q"].device)
    lam = s["lam"].double()
    for b, n in enumerate(_lengths(c)):
        keep = torch.arange(n, device=o.device)
        if b == B - 1:
            keep = keep[(keep < c["pad_from"]) | (keep >= c["pad_to"])]
        if not len(keep):
            continue
        for h in range(H):
            kk, vv = (s[t][b, h // (H // c["H_kv"])][keep].double() for t in ("k", "v"))
            f = [1.0, -(torch.exp(lam[0, h] @ lam[1, h]) - torch.exp(lam[2, h] @ lam[3, h]) + _LAMBDA_INIT)]
            for m in range(2):
                ch = slice(m * d // 2, (m + 1) * d // 2)
                for at in range(0, c["S_q"], 4096):
                    t = s["q"][b, h, at:at + 4096, ch].double() @ kk[:, ch].T / math.sqrt(d // 2)
                    lse[m, b, h, at:at + 4096] = torch.logsumexp(t, -1)
                    o[b, at:at + 4096, h] += f[m] * (torch.softmax(t, -1) @ vv)
    if c["norm"]:
        r = (o.pow(2).mean(-1, keepdim=True) + _EPS).sqrt()
        o = o / r * s["norm_w"].double() * (1 - _LAMBDA_INIT)
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "linear": _exact_linear, "diff": _exact_diff}[case["op"]](s)
