"""The layer operators' entry points without a GPU: argument errors come back
before anything is launched, the workspace sizes and the rotary frequency
tables are host arithmetic."""
import math

import pytest
import torch

from diffusion_transformer_joint_jattn_b200 import jattn

A = 1 << 20          # a 256-byte aligned fake address: never dereferenced (validation fails first)
INV, UNS, ALI = jattn.ERR_INVALID_ARG, jattn.ERR_UNSUPPORTED, jattn.ERR_ALIGNMENT


def rotary(code, **kw):
    a = dict(dict(x=A, y=A, H=2, n=1, dtype=jattn.BF16, B=1, S=3, d=64, parts=1, rot=64, pos=A, split=None, freqs=A,
                  layout=0, scale=1.0), **kw)
    t = jattn._ROTARY_TENSOR.pack(a["x"] or 0, a["y"] or 0, a["H"], 384, 128, 64, 384, 128, 64)
    sp = None if a["split"] is None else (jattn.ctypes.c_int32 * 3)(*a["split"])
    got = jattn.load().jattn_rotary(t * max(a["n"], 1), a["n"], a["dtype"], a["B"], a["S"], a["d"], a["parts"], a["rot"],
                                    a["pos"], 0, sp, a["freqs"], a["layout"], a["scale"], 0, None)
    assert got == code, (kw, got)


def test_rotary_refusals():
    for kw in (dict(n=0), dict(n=3), dict(B=-1), dict(S=-1), dict(d=0), dict(parts=0), dict(parts=3), dict(d=6, parts=2, rot=2),
               dict(rot=0), dict(rot=3), dict(rot=66), dict(d=1032, rot=64), dict(layout=2), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(split=(16, 24, 22)), dict(split=(15, 25, 24)), dict(split=(-2, 42, 24)),
               dict(x=None), dict(y=None), dict(pos=None), dict(freqs=None), dict(H=-1),
               dict(H=(1 << 24) + 1), dict(H=(1 << 23) + 1, parts=2, rot=32)):
        rotary(INV, **kw)
    rotary(UNS, dtype=jattn.E4M3)
    rotary(UNS, dtype=9)
    for kw in (dict(x=A + 1), dict(y=A + 1), dict(pos=A + 2), dict(freqs=A + 4), dict(x=A + 2, dtype=jattn.FP32)):
        rotary(ALI, **kw)


def test_rotary_without_work_is_ok():
    for kw in (dict(B=0), dict(S=0), dict(H=0)):
        rotary(jattn.OK, x=None, y=None, pos=None, freqs=None, **kw)


def linear(code, **kw):
    a = dict(dict(M=4, N=8, K=16, ldx=16, ldw=16, ldy=8, ldr=8, i=jattn.BF16, o=jattn.BF16, b=jattn.BF16, act=0, x=A, w=A,
                  bias=None, res=None, y=2 * A, ws=None, n=0), **kw)
    sh = jattn._LINEAR_SHAPE.pack(a["M"], a["N"], a["K"], a["ldx"], a["ldw"], a["ldy"], a["ldr"], a["i"], a["o"], a["b"],
                                  a["act"])
    got = jattn.load().jattn_linear(sh, a["x"], a["w"], a["bias"], a["res"], a["y"], a["ws"], a["n"], None)
    assert got == code, (kw, got)


def test_linear_refusals():
    for kw in (dict(M=-1), dict(N=-1), dict(K=0), dict(ldx=15), dict(ldw=8), dict(ldy=7), dict(res=A, ldr=7), dict(x=None),
               dict(w=None), dict(y=None), dict(res=2 * A, ldy=16), dict(y=A), dict(ldx=1 << 38),
               dict(M=(1 << 30) + 1), dict(N=(1 << 30) + 1, ldy=1 << 31), dict(K=(1 << 30) + 1, ldx=1 << 31, ldw=1 << 31)):
        linear(INV, **kw)
    for kw in (dict(i=jattn.FP32), dict(i=jattn.E4M3), dict(o=jattn.E4M3), dict(bias=A, b=jattn.E4M3), dict(act=5), dict(act=-1)):
        linear(UNS, **kw)
    for kw in (dict(x=A + 1), dict(w=A + 1), dict(y=A + 1), dict(y=A + 2, o=jattn.FP32), dict(res=A + 1), dict(bias=A + 1)):
        linear(ALI, **kw)
    linear(jattn.OK, M=0, x=None, w=None, y=None)
    linear(jattn.OK, N=0, x=None, w=None, y=None)


def test_linear_workspace():
    lib = jattn.load()
    size = lambda M, N, K, ldx, ldw, x=A, w=A: lib.jattn_linear_workspace(  # noqa: E731
        jattn._LINEAR_SHAPE.pack(M, N, K, ldx, ldw, N, N, 0, 0, 0, 0), x, w)
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    assert size(4, 8, 16, 16, 16) == 0
    assert size(4, 8, 13, 16, 24) == 0                       # odd K in aligned rows
    assert size(4, 8, 13, 13, 16) == up(4 * 16 * 2)
    assert size(4, 8, 13, 13, 13) == up(4 * 16 * 2) + up(8 * 16 * 2)
    assert size(1, 8, 13, 13, 16) == 0                       # one row needs no stride
    assert size(1, 8, 13, 13, 16, x=A + 2) == up(16 * 2)
    assert size(4, 8, 0, 0, 0) == 0
    assert size(70000, 3, 40001, 40001, 40008) == up(70000 * 40008 * 2)      # past 2^32 bytes
    linear(INV, K=13, ldx=13, ldw=16, ws=None)
    linear(INV, K=13, ldx=13, ldw=16, ws=A, n=127)
    linear(ALI, K=13, ldx=13, ldw=16, ws=A + 16, n=256)


def diff(code, **kw):
    a = dict(dict(B=1, H=4, H_kv=2, S_q=3, S_kv=9, d=128, dt=jattn.BF16, q=A, k=A, v=A, lam=A, init=0.3, norm=None, eps=1e-5,
                  len=None, mask=None, ws=None, n=0, o=A, lse=None, scale=0.0, qs=None, ks=None), **kw)
    d = a["d"]
    qs = a["qs"] or (a["H"] * a["S_q"] * d, a["S_q"] * d, d)
    ks = a["ks"] or (a["H_kv"] * max(a["S_kv"], 1) * d, max(a["S_kv"], 1) * d, d)
    sh = jattn._DIFF_SHAPE.pack(a["B"], a["H"], a["H_kv"], a["S_q"], a["S_kv"], d, *qs, *ks, *ks)
    got = jattn.load().jattn_fwd_diff(sh, a["dt"], a["q"], a["k"], a["v"], a["lam"], a["init"], a["norm"], a["eps"], a["len"],
                                      a["mask"], a["ws"], a["n"], a["o"], a["lse"], a["scale"], None)
    assert got == code, (kw, got)


def test_diff_refusals():
    for kw in (dict(B=-1), dict(H=0), dict(H_kv=0), dict(H=3), dict(S_q=-1), dict(S_kv=-1), dict(S_kv=(1 << 24) + 1),
               dict(B=300, H=300, H_kv=300), dict(q=None), dict(k=None), dict(v=None), dict(lam=None), dict(o=None),
               dict(init=float("nan")), dict(scale=float("inf")), dict(norm=A, eps=0.0), dict(norm=A, eps=float("nan")),
               dict(qs=(1536, 384, 64)), dict(qs=(1540, 388, 132)), dict(ks=(2304, 0, 128)),
               dict(B=65535, H=1, H_kv=1, S_q=1 << 24)):
        diff(INV, **kw)
    for kw in (dict(d=96), dict(d=256), dict(dt=jattn.FP32), dict(dt=jattn.E4M3)):
        diff(UNS, **kw)
    for kw in (dict(q=A + 8), dict(k=A + 2), dict(v=A + 8), dict(o=A + 8), dict(lam=A + 4), dict(norm=A + 4), dict(len=A + 2),
               dict(lse=A + 2)):
        diff(ALI, **kw)
    diff(jattn.OK, B=0, q=None, k=None, v=None, o=None, lam=None)
    diff(jattn.OK, S_q=0, q=None, k=None, v=None, o=None, lam=None)


def test_diff_workspace():
    lib = jattn.load()

    def size(B, H, H_kv, S_q, S_kv, d=128, dt=jattn.BF16):
        return lib.jattn_fwd_diff_workspace(
            jattn._DIFF_SHAPE.pack(B, H, H_kv, S_q, S_kv, d, H * S_q * d, S_q * d, d,
                                   *(2 * (H_kv * S_kv * d, S_kv * d, d))), dt)
    assert size(1, 4, 2, 3, 9) == 0                                  # short: one walk, P in two parts
    assert size(1, 4, 2, 3, 9, d=96) == 0 and size(1, 3, 2, 3, 9) == 0
    assert size(1, 2, 2, 300, 300, dt=jattn.FP16) == 0
    # bf16, several row tiles and a long walk: V in fp16 too
    assert size(2, 24, 24, 1024, 1024) - size(2, 24, 24, 1024, 1024, dt=jattn.FP16) >= 48 * 1024 * 128 * 2
    # one query over a long cache: parts of up to 148 CTAs, and no copy of V
    n = size(1, 8, 8, 1, 16384)
    assert 0 < n <= 148 * 4 * 128 * 129 * 4 + 1024
    assert size(1, 8, 8, 1, 16384, dt=jattn.FP16) == n
    diff(INV, H=1, H_kv=1, S_q=1, S_kv=4096, ws=None)
    diff(INV, H=1, H_kv=1, S_q=1, S_kv=4096, ws=A, n=16)
    diff(ALI, H=1, H_kv=1, S_q=1, S_kv=4096, ws=A + 16, n=1 << 30)


def test_rotary_freqs():
    f, s = jattn.rotary_freqs(8, 10000.0, device="cpu")
    assert s == 1.0 and f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-15, atol=0)
    assert torch.equal(jattn.rotary_freqs(8, scaling="linear", factor=4.0, device="cpu")[0], f / 4)
    # ntk: the slowest pair is interpolated by the factor, the fastest untouched
    g, s = jattn.rotary_freqs(64, scaling="ntk", factor=4.0, device="cpu")
    p = jattn.rotary_freqs(64, device="cpu")[0]
    assert s == 1.0 and g[0] == p[0] and math.isclose(float(g[-1]), float(p[-1]) / 4, rel_tol=1e-12)
    # yarn: pairs of many turns untouched, of less than one interpolated, between the two a mean
    y, s = jattn.rotary_freqs(128, scaling="yarn", factor=8.0, original_length=4096, device="cpu")
    p = jattn.rotary_freqs(128, device="cpu")[0]
    turns = 4096 * p / (2 * math.pi)
    assert math.isclose(s, 0.1 * math.log(8.0) + 1.0)
    assert torch.equal(y[turns > 40], p[turns > 40]) and torch.equal(y[turns < 0.7], p[turns < 0.7] / 8)
    assert ((y <= p) & (y >= p / 8 * (1 - 1e-15))).all()
    # axes: three spans, the layout of the joint prologue
    a, _ = jattn.rotary_freqs(split=(16, 24, 24), device="cpu")
    assert torch.equal(a, torch.cat([jattn.rotary_freqs(n, device="cpu")[0] for n in (16, 24, 24)]))
    assert len(jattn.rotary_freqs(split=(0, 4, 4), device="cpu")[0]) == 4
    for kw in (dict(dim=7), dict(dim=0), dict(dim=None), dict(dim=8, theta=0.0), dict(dim=8, scaling="cubic"),
               dict(dim=8, scaling="ntk", factor=0.0), dict(split=(3, 5, 8)), dict(dim=8, split=(4, 4, 4)),
               dict(split=(4, 4, 4), scaling="linear"), dict(dim=8, theta=1.0, scaling="yarn")):
        with pytest.raises(ValueError):
            jattn.rotary_freqs(**dict(dict(device="cpu"), **kw))


def test_host_tensors_are_refused():
    x = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        jattn.rotary(x, None, torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        jattn.linear(x, torch.zeros(8, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        jattn.fwd_diff(x, x, x, torch.zeros(4, 2, 32), 0.2)
    qkv = torch.zeros(1, 4, 3, 2, 64, dtype=torch.bfloat16)
    pos = torch.zeros(4, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        jattn.joint_attention(qkv, None, None, pos, (16, 24, 24), proj_w=torch.zeros(8, 128, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        jattn.joint_attention(qkv, None, None, pos, (16, 24, 24), residual=torch.zeros(1, 4, 8, dtype=torch.bfloat16))


def test_yarn_scale_of_shorter_contexts():
    """The factor of cosine and sine makes up for a stretched context: there is
    none for a factor of 1 or less."""
    for factor in (0.25, 0.5, 1.0):
        assert jattn.rotary_freqs(64, scaling="yarn", factor=factor, device="cpu")[1] == 1.0
    assert jattn.rotary_freqs(64, scaling="yarn", factor=2.0, device="cpu")[1] == 0.1 * math.log(2.0) + 1.0


def test_outputs_over_inputs_are_refused():
    """Rotary: one tensor's output over the other tensor; differential
    attention: the output over q, k or v (valid calls otherwise)."""
    def two(code, x0, y0, x1, y1, H1=2):
        t = b"".join(jattn._ROTARY_TENSOR.pack(x, y, H, 384, 128, 64, 384, 128, 64) for x, y, H in ((x0, y0, 2), (x1, y1, H1)))
        got = jattn.load().jattn_rotary(t, 2, jattn.BF16, 1, 3, 64, 1, 64, A, 0, None, A, 0, 1.0, 0, None)
        assert got == code, got
    two(INV, A, 2 * A, 3 * A, 2 * A)
    two(INV, A, 2 * A, 3 * A, A)
    two(INV, A, 3 * A, 3 * A, 2 * A)
    two(INV, A, 3 * A, 3 * A, A)
    for kw in (dict(o=A, q=A, k=2 * A, v=3 * A), dict(o=A, q=2 * A, k=A, v=3 * A), dict(o=A, q=2 * A, k=3 * A, v=A)):
        diff(INV, **kw)


def test_diff_workspace_of_long_caches():
    """Past 2^15 keys every CTA has fp32 sums of its 256 rows in the workspace."""
    def size(S_kv, d):
        return jattn.load().jattn_fwd_diff_workspace(
            jattn._DIFF_SHAPE.pack(1, 1, 1, 128 * 160, S_kv, d, 128 * 160 * d, 128 * 160 * d, d,
                                   *(2 * (S_kv * d, S_kv * d, d))), jattn.FP16)
    for d in (64, 128):
        sums = 148 * 256 * (d + 1) * 4
        assert sums <= size(32769, d) - size(32768, d) <= sums + 512
