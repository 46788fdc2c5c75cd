"""Rotary embedding against the fp64 oracle.

Tolerance per element: half a step of the output type, plus the fp32
arithmetic's share of the pair's magnitude |a| + |b| times scale: the reduced
angle rounded to fp32 (2^-23 at pi), sincosf (2 ulp, 2^-23), two products and
a sum (2 * 2^-24), under 4 * 2^-23 together."""
import numpy as np
import pytest
import torch

import oracle.layer as ref
from diffusion_transformer_joint_jattn_b200 import jattn

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def check(got, x, pos, freqs, **kw):
    want = ref.rotary(x.double().cpu().numpy(), pos, freqs, **kw)
    plain = np.abs(x.double().cpu().numpy())
    R, n = 2 * len(freqs), x.shape[-1] // kw.get("parts", 1)
    size = plain.copy()
    for part in range(kw.get("parts", 1)):
        for p in range(R // 2):
            i, j = (p, p + R // 2) if kw.get("half") else (2 * p, 2 * p + 1)
            i, j = part * n + i, part * n + j
            size[..., i] = size[..., j] = plain[..., i] + plain[..., j]
    tol = torch.finfo(x.dtype).eps / 2 * np.abs(want) + 4 * 2.0 ** -23 * kw.get("scale", 1.0) * size
    tol += float(torch.finfo(x.dtype).smallest_normal) * torch.finfo(x.dtype).eps      # subnormal outputs
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err / tol).max())


def case(dev, dtype, B, S, H, H_k, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    mk = lambda h: torch.randn(B, S, h, d, generator=g).to(DT[dtype]).to(dev)  # noqa: E731
    return mk(H), mk(H_k)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("B,S,H,H_k,d,rot,parts", [
    (1, 1, 1, 1, 2, 2, 1), (2, 1, 8, 2, 128, 128, 1), (3, 37, 5, 1, 64, 32, 1), (1, 130, 24, 24, 128, 64, 2),
    (2, 7, 3, 3, 80, 36, 1), (1, 5, 2, 1, 96, 94, 1), (1, 9, 4, 2, 256, 126, 2), (2, 3, 33, 7, 10, 4, 1),
])
def test_against_the_definition(cuda_device, dtype, layout, B, S, H, H_k, d, rot, parts):
    q, k = case(cuda_device, dtype, B, S, H, H_k, d)
    pos = torch.randint(0, 5000, (B, S), generator=torch.Generator().manual_seed(1)).int()
    freqs, scale = jattn.rotary_freqs(rot, 10000.0, device=cuda_device)
    yq, yk = jattn.rotary(q, k, pos.to(cuda_device), freqs, layout=layout, parts=parts, scale=scale)
    for y, x in ((yq, q), (yk, k)):
        check(y, x, pos.numpy(), freqs.cpu().numpy(), half=layout == "half", parts=parts)


def test_axes_strides_head_major_and_in_place(cuda_device):
    """q and k as views of a fused projection into head-major outputs, with
    (t, row, col) positions; then in place, bit for bit the same."""
    B, S, H, d = 2, 50, 3, 128
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn(B, S, 3, H, d, generator=g).to(torch.bfloat16).to(cuda_device)
    q, k = qkv[:, :, 0], qkv[:, :, 1]
    pos = torch.randint(0, 128, (S, 3), generator=g).int()
    split = (16, 56, 56)
    freqs, _ = jattn.rotary_freqs(theta=10000.0, split=split, device=cuda_device)
    out = tuple(torch.zeros(B, H, S, d, dtype=torch.bfloat16, device=cuda_device).transpose(1, 2) for _ in range(2))
    before = qkv.clone()
    yq, yk = jattn.rotary(q, k, pos.to(cuda_device), freqs, split=split, out=out)
    assert yq is out[0] and torch.equal(qkv, before)
    axis = [0] * 8 + [1] * 28 + [2] * 28
    both = np.broadcast_to(pos.numpy(), (B, S, 3))
    check(yq, q, both, freqs.cpu().numpy(), axis=axis)
    check(yk, k, both, freqs.cpu().numpy(), axis=axis)
    jattn.rotary(q, k, pos.to(cuda_device), freqs, split=split, out=(q, k))
    assert torch.equal(q, yq) and torch.equal(k, yk) and torch.equal(qkv[:, :, 2], before[:, :, 2])


def test_matches_the_prologue(cuda_device):
    """The same rotation as rope_qkv's, bit for bit (bf16 outputs)."""
    from diffusion_transformer_joint_jattn_b200 import workloads as W
    from parity_util import to_device
    w = W.custom(B=2, H=3, d=128, S_txt=20, grid=6, n_ref=1)
    inp = to_device(W.make_inputs(w, 3), cuda_device)
    q, k, _, _ = jattn.rope_qkv(inp["qkv_txt"], inp["qkv_img"], inp["qkv_ref"], inp["pos"], w.split, w.theta, "bf16")
    joint = torch.cat([inp["qkv_txt"], inp["qkv_img"], inp["qkv_ref"]], 1)
    freqs, _ = jattn.rotary_freqs(theta=w.theta, split=w.split, device=cuda_device)
    yq, yk = jattn.rotary(joint[:, :, 0], joint[:, :, 1], inp["pos"], freqs, split=w.split)
    assert torch.equal(yq.transpose(1, 2), q) and torch.equal(yk.transpose(1, 2), k)


def test_far_positions_and_scalings(cuda_device):
    q, k = case(cuda_device, "fp32", 1, 64, 2, 1, 64, 4)
    pos = torch.arange(64).int() + (1 << 20) - 3
    for kw in (dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=8.0),
               dict(scaling="yarn", factor=32.0, original_length=4096)):
        freqs, scale = jattn.rotary_freqs(64, 10000.0, device=cuda_device, **kw)
        yq, yk = jattn.rotary(q, k, pos.to(cuda_device), freqs, layout="half", scale=scale)
        check(yq, q, pos.numpy()[None], freqs.cpu().numpy(), half=True, scale=scale)
        check(yk, k, pos.numpy()[None], freqs.cpu().numpy(), half=True, scale=scale)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_gradient(cuda_device, layout):
    """inverse is the gradient: against differences of sum(g * rotary(x)), which
    is linear in x, so that a difference of any step is exact up to fp32."""
    q, _ = case(cuda_device, "fp32", 2, 5, 2, 1, 24, 5)
    pos = torch.randint(0, 1000, (2, 5), generator=torch.Generator().manual_seed(6)).int().to(cuda_device)
    freqs, scale = jattn.rotary_freqs(16, 1000.0, scaling="yarn", factor=4.0, original_length=64, device=cuda_device)
    g = torch.randn(q.shape, generator=torch.Generator().manual_seed(7)).to(cuda_device)
    kw = dict(layout=layout, scale=scale)
    grad, _ = jattn.rotary(g, None, pos, freqs, inverse=True, **kw)
    check(grad, g, pos.cpu().numpy(), freqs.cpu().numpy(), half=layout == "half", scale=scale, inverse=True)
    f = lambda x: (jattn.rotary(x, None, pos, freqs, **kw)[0].double() * g.double()).sum().item()  # noqa: E731
    for at in ((0, 0, 0, 0), (1, 4, 1, 7), (0, 3, 1, 15), (1, 2, 0, 23)):
        hi, lo = q.clone(), q.clone()
        hi[at] += 1.0
        lo[at] -= 1.0
        # fp32 products of both evaluations: 2 * 24 channels of at most ~8
        assert abs((f(hi) - f(lo)) / 2 - grad[at].item()) <= 48 * 8 * 2.0 ** -23


def test_copied_channels_keep_infinities(cuda_device):
    q = torch.full((1, 3, 2, 16), float("inf"), dtype=torch.bfloat16, device=cuda_device)
    q[..., 4:8] = float("nan")
    freqs, _ = jattn.rotary_freqs(2, 10.0, device=cuda_device)
    y, none = jattn.rotary(q, None, torch.arange(3, device=cuda_device).int(), freqs)
    assert none is None and torch.isinf(y[..., 2:4]).all() and torch.isnan(y[..., 4:8]).all()
    assert torch.isinf(y[..., 8:]).all()


def test_nothing_to_do(cuda_device):
    freqs, _ = jattn.rotary_freqs(8, 10.0, device=cuda_device)
    for B, S, H in ((0, 3, 2), (2, 0, 2), (1, 3, 0)):
        q = torch.empty(B, S, H, 8, dtype=torch.float16, device=cuda_device)
        y, _ = jattn.rotary(q, None, torch.zeros(S, dtype=torch.int32, device=cuda_device), freqs)
        assert y.shape == q.shape


def test_refusals(cuda_device):
    q, k = case(cuda_device, "bf16", 2, 4, 2, 2, 16)
    pos = torch.zeros(4, dtype=torch.int32, device=cuda_device)
    freqs, _ = jattn.rotary_freqs(16, 10.0, device=cuda_device)
    for bad in (dict(q=q.cpu()), dict(q=q[0]), dict(q=q.double()), dict(k=k[:1]), dict(k=k.half()), dict(pos=pos[:3]),
                dict(pos=pos.long()), dict(freqs=freqs.float()), dict(freqs=freqs.cpu()), dict(layout="pairs"),
                dict(split=(4, 6, 6)), dict(out=(q[:1], k)), dict(out=(q,)), dict(q=q.transpose(2, 3))):
        a = dict(dict(q=q, k=k, pos=pos, freqs=freqs), **bad)
        with pytest.raises(ValueError):
            jattn.rotary(**a)
    for bad in (dict(parts=3), dict(freqs=torch.cat([freqs, freqs])), dict(scale=float("nan"))):
        with pytest.raises(jattn.JattnError):
            jattn.rotary(**dict(dict(q=q, k=k, pos=pos, freqs=freqs), **bad))


def test_other_stream_and_graph(cuda_device):
    q, k = case(cuda_device, "bf16", 1, 33, 4, 4, 64, 8)
    pos = torch.arange(33, device=cuda_device).int()
    freqs, _ = jattn.rotary_freqs(64, 10000.0, device=cuda_device)
    want = jattn.rotary(q, k, pos, freqs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = jattn.rotary(q, k, pos, freqs, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = jattn.rotary(q, k, pos, freqs)
    pos += 5
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(y, jattn.rotary(q, k, pos, freqs)))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("inverse", [False, True])
def test_odd_strides(cuda_device, dtype, layout, inverse):
    """Heads an odd number of elements apart, into heads at other odd strides and
    an odd offset: single channels at a time.  What lies between is left."""
    B, S, H, d, rot = 2, 9, 3, 20, 12
    g = torch.Generator().manual_seed(10)
    x = torch.randn(B, S, H, d + 1, generator=g).to(DT[dtype]).to(cuda_device)
    q, k = x[..., :d], x[:, :, 1:, 1:]
    pos = torch.randint(0, 3000, (B, S), generator=g).int().to(cuda_device)
    freqs, scale = jattn.rotary_freqs(rot, scaling="yarn", factor=8.0, device=cuda_device)
    bufs = [torch.full((B * S * h * (d + 3) + 1,), 7.0, dtype=DT[dtype], device=cuda_device) for h in (H, H - 1)]
    out = tuple(b[1:].view(B, S, h, d + 3)[..., :d] for b, h in zip(bufs, (H, H - 1)))
    jattn.rotary(q, k, pos, freqs, layout=layout, scale=scale, inverse=inverse, out=out)
    for y, x_ in zip(out, (q, k)):
        check(y, x_, pos.cpu().numpy(), freqs.cpu().numpy(), half=layout == "half", scale=scale, inverse=inverse)
        y.fill_(7.0)
    assert all((b == 7.0).all() for b in bufs)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_inverse_in_16_bits(cuda_device, dtype, layout):
    """The transposed map in every access width of the 16-bit kernels."""
    for d, rot, parts in ((128, 128, 1), (128, 64, 2), (64, 24, 1), (36, 12, 1), (10, 6, 1)):
        q, k = case(cuda_device, dtype, 2, 41, 3, 1, d, seed=d)
        pos = torch.randint(0, 9000, (2, 41), generator=torch.Generator().manual_seed(11)).int()
        freqs, scale = jattn.rotary_freqs(rot, scaling="yarn", factor=4.0, device=cuda_device)
        kw = dict(layout=layout, parts=parts, scale=scale)
        yq, yk = jattn.rotary(q, k, pos.to(cuda_device), freqs, inverse=True, **kw)
        for y, x in ((yq, q), (yk, k)):
            check(y, x, pos.numpy(), freqs.cpu().numpy(), half=layout == "half", parts=parts, scale=scale, inverse=True)
