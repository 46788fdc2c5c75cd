"""The linear layer with its epilogue against the fp64 oracle.

Tolerance per element: half a step of the output type of the result, plus the
fp32 sum: K products (exact in fp32) added with at most one unit of 2^-23 of
the sum of magnitudes each, scaled by the activation's slope (at most 1.13),
plus 2^-18 of the result for the epilogue's approximate exp and reciprocal."""
import numpy as np
import pytest
import torch

import oracle.layer as ref
from diffusion_transformer_joint_jattn_b200 import jattn

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def make(dev, dtype, M, N, K, seed=0, out=None, bias="same", residual=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g).to(DT[dtype]).to(dev)
    w = (torch.randn(N, K, generator=g) / K ** 0.5).to(DT[dtype]).to(dev)
    b = None if bias is None else torch.randn(N, generator=g).to(DT[dtype if bias == "same" else bias]).to(dev)
    r = torch.randn(M, N, generator=g).to(DT[out or dtype]).to(dev) if residual else None
    return x, w, b, r


def check(y, x, w, b, act, r):
    f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    want = ref.linear(f(x), f(w), f(b), act, f(r))
    sums = np.abs(f(x)) @ np.abs(f(w)).T + (0 if b is None else np.abs(f(b)))
    tol = (torch.finfo(y.dtype).eps / 2 + 2.0 ** -18) * np.abs(want) + 1.13 * (x.shape[1] + 2) * 2.0 ** -23 * sums
    if r is not None:
        tol += 2.0 ** -18 * np.abs(f(r))
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err / tol).max())


SIZES = [
    (1, 128, 64), (1, 1, 1), (3, 257, 512), (16, 1000, 2048), (17, 128, 96), (33, 300, 1000), (64, 64, 4096),
    (65, 65, 65), (127, 255, 63), (128, 128, 128), (129, 640, 72), (300, 777, 1003), (512, 2048, 512),
    (1000, 1500, 333), (2304, 2304, 192), (2500, 2700, 264),
]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp32")])
def test_sizes(cuda_device, M, N, K, dtype, out):
    x, w, b, r = make(cuda_device, dtype, M, N, K, out=out, residual=True)
    y = jattn.linear(x, w, b, residual=r, out_dtype=DT[out])
    assert y.shape == (M, N) and y.dtype == DT[out]
    check(y, x, w, b, "none", r)
    assert jattn.device_status()[0] == jattn.OK


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "silu", "relu"])
@pytest.mark.parametrize("M", [5, 200, 2304])
@pytest.mark.parametrize("dtype,out,bias", [("bf16", "fp32", "fp32"), ("fp16", "fp16", "same"), ("bf16", "fp16", None)])
def test_epilogues(cuda_device, act, M, dtype, out, bias):
    N, K = (2304, 128) if M > 1000 else (200, 128)
    x, w, b, _ = make(cuda_device, dtype, M, N, K, seed=M, out=out, bias=bias)
    y = jattn.linear(4 * x, w, b, act=act, out_dtype=DT[out])
    check(y, 4 * x, w, b, act, None)


@pytest.mark.parametrize("M,N,K", [(7, 129, 200), (150, 140, 130), (2304, 2310, 136)])
def test_strides(cuda_device, M, N, K):
    """Rows inside wider buffers, aligned for TMA or not, on both sides; what
    lies around the output is left as it was."""
    x0, w0, b, r0 = make(cuda_device, "bf16", M, N, K, residual=True)
    for pad, off in ((8, 8), (3, 1)):
        big = lambda t: torch.zeros(t.shape[0], t.shape[1] + pad + off, dtype=t.dtype, device=cuda_device)  # noqa: E731
        views = []
        for t in (x0, w0, r0):
            v = big(t)[:, off:off + t.shape[1]]
            v.copy_(t)
            views.append(v)
        x, w, r = views
        out = torch.full((M + 2, N + 40), 7.0, dtype=torch.bfloat16, device=cuda_device)
        y = jattn.linear(x, w, b, residual=r, out=out[1:-1, off:off + N])
        check(y, x0, w0, b, "none", r0)
        y.fill_(7.0)
        assert (out == 7.0).all()


def test_residual_in_place_and_leading_dimensions(cuda_device):
    x, w, b, _ = make(cuda_device, "bf16", 6 * 50, 320, 96)
    r = torch.randn(6, 50, 320, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(cuda_device)
    want = jattn.linear(x.view(6, 50, 96), w, b, "silu", residual=r)
    assert want.shape == (6, 50, 320)
    got = r.clone()
    assert jattn.linear(x.view(6, 50, 96), w, b, "silu", residual=got, out=got) is got
    assert torch.equal(got, want)
    check(want.view(300, 320), x, w, b, "silu", r.view(300, 320))


def test_infinities_stay_in_their_rows(cuda_device):
    for M, N, K in ((20, 300, 200), (300, 300, 200), (2304, 2304, 136)):
        x, w, b, _ = make(cuda_device, "bf16", M, N, K)
        clean = jattn.linear(x, w, b)
        x[M // 2, 3] = float("inf")
        w[7, 5] = float("nan")
        y = jattn.linear(x, w, b)
        assert torch.isnan(y[:, 7]).all() and not torch.isfinite(y[M // 2]).any()
        keep = torch.ones_like(y, dtype=torch.bool)
        keep[:, 7] = keep[M // 2] = False
        assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("out", ["fp16", "fp32"])
def test_activations_at_the_ends(cuda_device, out):
    """x = value * 1: the activation of values far out, where exp leaves the
    fp32 range.  Expected from fp64; what vanishes there is 0 here."""
    vals = torch.tensor([0.0, -0.5, 0.5, -20.0, 20.0, -86.0, -87.5, -90.0, -200.0, 200.0, -6e4, 6e4, -1e30, 1e30, -3e38, 3e38,
                         float("nan")])
    x = vals.bfloat16().view(-1, 1).to(cuda_device)
    w = torch.ones(40, 1, dtype=torch.bfloat16, device=cuda_device)
    ref64 = x.double().cpu()
    for act, f in (("gelu", torch.nn.functional.gelu), ("silu", torch.nn.functional.silu), ("relu", torch.relu),
                   ("gelu_tanh", lambda v: torch.nn.functional.gelu(v, approximate="tanh"))):
        want = f(ref64).to(DT[out]).double().expand(-1, 40)
        got = jattn.linear(x, w, act=act, out_dtype=DT[out]).double().cpu()
        assert torch.equal(got.isnan(), want.isnan()), act
        fine = want.isfinite()
        assert torch.equal(got[~fine & ~want.isnan()], want[~fine & ~want.isnan()]), act
        # half a step of the type, the epilogue's 2^-18, and what fp32 cannot hold
        tol = (torch.finfo(DT[out]).eps + 2.0 ** -18) * want[fine].abs() + max(torch.finfo(DT[out]).tiny, 2.0 ** -110)
        assert ((got[fine] - want[fine]).abs() <= tol).all(), (act, got[:, 0], want[:, 0])


@pytest.mark.parametrize("M,N,K", [(5, 300, 8192), (30, 130, 5000), (150, 300, 8192), (1000, 1300, 4100), (2304, 4480, 4096)])
def test_long_sums_in_fp32(cuda_device, M, N, K):
    """An fp32 output of a long sum: runs of 512 products, in which the tensor
    cores make 32 additions that each lose at most 2^-23 of the sum, half of
    it on average -- 32 * 2^-24 of the result -- and rounded sums of the runs."""
    x, w, _, _ = make(cuda_device, "bf16", M, N, K, seed=K)
    y = jattn.linear(x, w, out_dtype=torch.float32).double()
    want = x.double() @ w.double().t()
    assert (y - want).norm() <= 2.0 ** -19 * want.norm()


def test_same_bits_every_time(cuda_device):
    for M, N, K in ((4, 512, 4096), (100, 256, 2048), (2500, 2700, 264)):
        x, w, b, _ = make(cuda_device, "fp16", M, N, K)
        first = jattn.linear(x, w, b, "gelu")
        assert all(torch.equal(first, jattn.linear(x, w, b, "gelu")) for _ in range(3))


def test_nothing_to_do(cuda_device):
    w = torch.zeros(8, 16, dtype=torch.bfloat16, device=cuda_device)
    assert jattn.linear(torch.zeros(0, 16, dtype=torch.bfloat16, device=cuda_device), w).shape == (0, 8)
    assert jattn.linear(torch.zeros(3, 16, dtype=torch.bfloat16, device=cuda_device), w[:0]).shape == (3, 0)


def test_refusals(cuda_device):
    x, w, b, r = make(cuda_device, "bf16", 6, 8, 16, residual=True)
    for bad in (dict(x=x.cpu()), dict(x=x.float()), dict(w=w.half()), dict(w=w[:, :8]), dict(act="swish"),
                dict(bias=b[:4]), dict(bias=b.cpu()), dict(residual=r.float()), dict(residual=r[:3]),
                dict(out=torch.empty(6, 9, dtype=torch.bfloat16, device=cuda_device)), dict(out_dtype=torch.int32),
                dict(x=x.t().contiguous().t()), dict(x=torch.stack([x, x], 1)[:4:2].transpose(0, 1))):
        with pytest.raises(ValueError):
            jattn.linear(**dict(dict(x=x, w=w, bias=b, residual=r), **bad))
    with pytest.raises(jattn.JattnError):
        jattn.linear(x[:, :0], w[:, :0])


def test_other_stream_and_graph(cuda_device):
    for M, N, K in ((4, 256, 1024), (2304, 2304, 128)):
        x, w, b, _ = make(cuda_device, "bf16", M, N, K)
        want = jattn.linear(x, w, b)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = jattn.linear(x, w, b, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = jattn.linear(x, w, b)
        x.neg_()
        graph.replay()
        assert torch.equal(y, jattn.linear(x, w, b))


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M", [17, 200])
def test_gelu_of_negative_values(cuda_device, out, M):
    """x = value * 1 where x Phi(x) is small and has to keep its relative
    accuracy.  The exponent x^2 / 2 is off by at most 2^-23 relative (two
    roundings), which moves the exponential by x^2 / 2 times that; its own
    2^-22, the polynomial's 2^-22.5, the reciprocal and the products: under
    (x^2 + 8) 2^-23."""
    vals = torch.tensor([-0.25, -1.0, -2.0, -2.5, -3.0, -3.5, -4.0, -4.5, -5.0, -5.5, -6.0, -7.0, -8.0, -10.0, -12.0, 3.0, 6.0])
    x = vals.bfloat16().repeat(-(-M // len(vals)))[:M].view(-1, 1).to(cuda_device)
    w = torch.ones(40, 1, dtype=torch.bfloat16, device=cuda_device)
    v = x.double().cpu().numpy()
    want = torch.from_numpy(ref.activation(v, "gelu"))
    got = jattn.linear(x, w, act="gelu", out_dtype=DT[out]).double().cpu()
    t = torch.finfo(DT[out])
    tol = (t.eps / 2 + torch.from_numpy(v * v + 8) * 2.0 ** -23) * want.abs() + t.smallest_normal * t.eps / 2
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol)[:17, 0]


@pytest.mark.parametrize("M,N,K,out", [
    (4, 256, 1 << 18, "fp16"), (30, 130, 1 << 18, "fp16"), (300, 300, 1 << 18, "fp16"), (40, 70, 100001, "fp16"),
    (2304, 2304, 1 << 17, "fp16"), (2304, 2304, 1 << 19, "bf16"), (300, 300, 1 << 20, "bf16"),
])
def test_long_sums_of_one_sign(cuda_device, M, N, K, out):
    """Sums of so many products that the accumulator's losses would show in a
    16-bit output.  Runs of 512 products (32 additions of at most 2^-23 of the
    sum each), up to 2048 of them added with rounding in fp32 (2^-24 each, and
    no more than a quarter of them one way)."""
    g = torch.Generator(device=cuda_device).manual_seed(K)
    x, w = (torch.empty(n, K, dtype=torch.bfloat16, device=cuda_device) for n in (M, N))
    for t in (x, w):
        for i in range(0, len(t), 256):
            t[i:i + 256] = torch.rand(t[i:i + 256].shape, generator=g, device=cuda_device) / (K if t is w else 1)
    y = jattn.linear(x, w, out_dtype=DT[out])
    rows = torch.arange(0, M, max(1, M // 16), device=cuda_device)
    want = sum(x[rows, i:i + 65536].double() @ w[:, i:i + 65536].double().t() for i in range(0, K, 65536))
    tol = torch.finfo(DT[out]).eps / 2 + 2.0 ** -18 + K // 512 / 4 * 2.0 ** -24
    assert ((y[rows].double() / want - 1).abs() <= tol).all()
    assert jattn.device_status()[0] == jattn.OK
