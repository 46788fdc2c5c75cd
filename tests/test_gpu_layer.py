"""The layer operators as a model uses them together: a differential attention
layer (fused projection -> rotary -> differential attention -> output
projection with the residual stream) for a prompt and then token by token over
a cache, and the output projection of joint_attention."""
import numpy as np
import pytest
import torch

import oracle.layer as ref
from diffusion_transformer_joint_jattn_b200 import jattn
from diffusion_transformer_joint_jattn_b200 import workloads as W
from parity_util import to_device

pytestmark = pytest.mark.gpu

INIT, EPS = 0.2, 1e-5


def rel(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


def f64(t):
    return t.double().cpu().numpy()


class Layer:
    def __init__(self, dev, width, H, H_kv, d, seed=0):
        g = torch.Generator().manual_seed(seed)
        mk = lambda *s: (torch.randn(*s, generator=g) / s[-1] ** 0.5).to(torch.bfloat16).to(dev)  # noqa: E731
        self.H, self.H_kv, self.d = H, H_kv, d
        self.w_in, self.b_in = mk((H + 2 * H_kv) * d, width), mk((H + 2 * H_kv) * d)
        self.w_out = mk(width, H * d)
        self.lam = (0.1 * torch.randn(4, H, d // 2, generator=g)).to(dev)
        self.norm = (1 + 0.1 * torch.randn(d, generator=g)).to(dev)
        self.freqs, self.scale = jattn.rotary_freqs(d // 2, 10000.0, device=dev)

    def __call__(self, x, pos, k_cache, v_cache, at, lens):
        """x [B, S, width] at positions `at` .. on; writes the cache [B, H_kv,
        capacity, d] and attends to its first `lens` keys."""
        B, S, _ = x.shape
        H, n, d = self.H, self.H_kv, self.d
        qkv = jattn.linear(x, self.w_in, self.b_in).view(B, S, H + 2 * n, d)
        q = torch.empty(B, H, S, d, dtype=x.dtype, device=x.device)
        jattn.rotary(qkv[:, :, :H], qkv[:, :, H:H + n], pos, self.freqs, layout="half", parts=2, scale=self.scale,
                     out=(q.transpose(1, 2), k_cache[:, :, at:at + S].transpose(1, 2)))
        v_cache[:, :, at:at + S] = qkv[:, :, H + n:].transpose(1, 2)
        o, _ = jattn.fwd_diff(q, k_cache, v_cache, self.lam, INIT, norm_w=self.norm, eps=EPS, kv_len=lens)
        return jattn.linear(o.flatten(2), self.w_out, residual=x), qkv, o

    def exact(self, x, pos, qkv, o, k_past, v_past):
        """Every step's definition on the inputs that the step had."""
        H, n, d = self.H, self.H_kv, self.d
        B, S, _ = x.shape
        want_qkv = ref.linear(f64(x).reshape(B * S, -1), f64(self.w_in), f64(self.b_in))
        t = f64(qkv)
        turn = lambda a: ref.rotary(a, f64(pos), f64(self.freqs), half=True, parts=2, scale=self.scale)  # noqa: E731
        head = lambda a: a.transpose(0, 2, 1, 3)  # noqa: E731
        k = np.concatenate([k_past, head(turn(t[:, :, H:H + n]))], 2)
        v = np.concatenate([v_past, head(t[:, :, H + n:])], 2)
        want_o, _, _ = ref.diff_attention(head(turn(t[:, :, :H])), k, v, f64(self.lam), INIT, f64(self.norm), EPS)
        want_y = ref.linear(f64(o).reshape(B * S, -1), f64(self.w_out), residual=f64(x).reshape(B * S, -1))
        return want_qkv, want_o, want_y, k, v


def test_prompt_then_tokens(cuda_device):
    """Each step is held to its own inputs, so nothing accumulates: a
    projection is off by its output's rounding (2^-8 at most), the attention
    also by q's, k's and P's.  Rounded q and k move logits of size ~1 by
    2^-8 * sqrt(2) relative, P by as much: 4 * 2^-8 covers them with the
    cancellation of the two maps."""
    B, S, steps, cap, width = 2, 150, 3, 400, 256
    layer = Layer(cuda_device, width, 4, 2, 64)
    g = torch.Generator().manual_seed(9)
    x = torch.randn(B, S + steps, width, generator=g).to(torch.bfloat16).to(cuda_device)
    kc = torch.full((B, 2, cap, 64), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    vc = torch.full((B, 2, cap, 64), float("inf"), dtype=torch.bfloat16, device=cuda_device)
    kp = vp = np.zeros((B, 2, 0, 64))
    for at, n in [(0, S)] + [(S + i, 1) for i in range(steps)]:
        pos = (at + torch.arange(n, device=cuda_device)).int().expand(B, n).contiguous()
        lens = torch.full((B,), at + n, dtype=torch.int32, device=cuda_device)
        xs = x[:, at:at + n].contiguous()
        y, qkv, o = layer(xs, pos, kc, vc, at, lens)
        want_qkv, want_o, want_y, kp, vp = layer.exact(xs, pos, qkv, o, kp, vp)
        assert rel(f64(qkv).reshape(want_qkv.shape), want_qkv) <= 2.0 ** -8
        assert rel(f64(o), want_o) <= 4 * 2.0 ** -8
        assert rel(f64(y).reshape(want_y.shape), want_y) <= 2.0 ** -8
    assert torch.isnan(kc[:, :, S + steps:]).all() and torch.isinf(vc[:, :, S + steps:]).all()
    assert jattn.device_status()[0] == jattn.OK


def test_captured_step_follows_its_lengths(cuda_device):
    """One captured single-token step, replayed with other inputs, positions
    and lengths, equals the eager step bit for bit."""
    B, cap, width = 3, 5000, 256
    layer = Layer(cuda_device, width, 8, 2, 128, seed=1)
    g = torch.Generator().manual_seed(2)
    mk = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(cuda_device)  # noqa: E731
    kc, vc, x = mk(B, 2, cap, 128), mk(B, 2, cap, 128), mk(B, 1, width)
    pos = torch.tensor([[5], [6], [7]], dtype=torch.int32, device=cuda_device)
    lens = torch.tensor([100, 4000, 1], dtype=torch.int32, device=cuda_device)
    run = lambda: layer(x, pos, kc, vc, 0, lens)[0]  # noqa: E731
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run()
    x.copy_(mk(B, 1, width))
    pos += 1000
    lens.copy_(torch.tensor([5000, 0, 129], dtype=torch.int32))
    graph.replay()
    got = y.clone()
    assert torch.equal(got, run())
    assert jattn.device_status()[0] == jattn.OK


@pytest.mark.parametrize("path", ["bf16", "fp8"])
def test_joint_attention_output_projection(cuda_device, path):
    w = W.custom(B=2, H=2, d=128, S_txt=20, grid=8, n_ref=0)
    inp = to_device(W.make_inputs(w, 3), cuda_device)
    g = torch.Generator().manual_seed(4)
    wo = (torch.randn(192, w.H * w.d, generator=g) / 16).to(torch.bfloat16).to(cuda_device)
    bo = torch.randn(192, generator=g).to(torch.bfloat16).to(cuda_device)
    x = torch.randn(w.B, w.S, 192, generator=g).to(torch.bfloat16).to(cuda_device)
    args = (inp["qkv_txt"], inp["qkv_img"], inp["qkv_ref"], inp["pos"], w.split, w.theta, path)
    o, lse = jattn.joint_attention(*args, want_lse=True)
    y, lse2 = jattn.joint_attention(*args, want_lse=True, proj_w=wo, proj_b=bo, residual=x)
    assert torch.equal(lse, lse2) and y.shape == x.shape
    want = ref.linear(f64(o).reshape(w.B * w.S, -1), f64(wo), f64(bo), residual=f64(x).reshape(w.B * w.S, -1))
    assert rel(f64(y).reshape(want.shape), want) <= 2.0 ** -8
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y3 = jattn.joint_attention(*args, proj_w=wo, proj_b=bo, residual=x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y3, y)


def test_offsets_past_32_bits(cuda_device):
    """Elements more than 2^32 from their tensor's start: the last sequence of a
    cache of 5.4e9 elements (what is not its keys is never read), a rotary
    view and the rows of a linear layer with strides of 2^31 elements."""
    B, n, cap, d, L = 5, 8, 1 << 20, 128, 300
    g = torch.Generator().manual_seed(5)
    mk = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(cuda_device)  # noqa: E731
    k, v = (torch.empty(B, n, cap, d, dtype=torch.bfloat16, device=cuda_device) for _ in range(2))
    assert k.numel() > 1 << 32
    q, ks, vs, lam = mk(B, n, 1, d), mk(1, n, L, d), mk(1, n, L, d), 0.1 * torch.randn(4, n, d // 2, generator=g)
    k[-1:, :, :L], v[-1:, :, :L] = ks, vs
    lens = torch.tensor([0, 0, 0, 0, L], dtype=torch.int32, device=cuda_device)
    o, _ = jattn.fwd_diff(q, k, v, lam.to(cuda_device), INIT, kv_len=lens)
    want, _ = jattn.fwd_diff(q[-1:], ks, vs, lam.to(cuda_device), INIT)
    # the same keys in other shares of the walk: both forms' rounding
    assert torch.allclose(o[-1:].float(), want.float(), rtol=2 * 2.0 ** -8, atol=2.0 ** -9) and (o[:-1] == 0).all()
    freqs, _ = jattn.rotary_freqs(d, device=cuda_device)
    pos = torch.arange(2, device=cuda_device).int()
    far = k[:, 3:5, 77].view(B, 1, 2, d)[-2:].expand(2, 1, 2, d)          # strides of n * cap * d elements
    far.copy_(mk(2, 1, 2, d))
    near = far.contiguous()
    pos1 = pos[1:].contiguous()
    assert torch.equal(jattn.rotary(far, None, pos1, freqs)[0], jattn.rotary(near, None, pos1, freqs)[0])
    jattn.rotary(far, None, pos1, freqs, out=(far,))
    assert torch.equal(far, jattn.rotary(near, None, pos1, freqs)[0])
    flat = k.view(-1)
    K, N, step = 64, 96, 1 << 31
    w = mk(N, K)
    for off in (0, 1):                                                    # addressed by TMA, and copied first
        x = flat[off:].as_strided((3, K), (step, 1), storage_offset=off)
        x.copy_(mk(3, K))
        y = v.view(-1).as_strided((3, N), (step, 1), storage_offset=off)
        assert torch.equal(jattn.linear(x, w, out=y), jattn.linear(x.contiguous(), w))
    assert jattn.device_status()[0] == jattn.OK


def test_two_streams_at_once(cuda_device):
    """Calls on two streams share nothing: the results are those of one."""
    g = torch.Generator().manual_seed(6)
    mk = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(cuda_device)  # noqa: E731
    q, k, v = mk(1, 8, 1, 128), mk(1, 2, 6000, 128), mk(1, 2, 6000, 128)
    lam = (0.1 * torch.randn(4, 8, 64, generator=g)).to(cuda_device)
    x, w = mk(40, 1003), mk(777, 1003)
    want_o, want_y = jattn.fwd_diff(q, k, v, lam, INIT)[0], jattn.linear(x, w)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[] for _ in streams]
    for _ in range(20):
        for s, out in zip(streams, got):
            out.append((jattn.fwd_diff(q, k, v, lam, INIT, stream=s)[0], jattn.linear(x, w, stream=s)))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want_o) and torch.equal(y, want_y) for out in got for o, y in out)


def test_workspaces_of_the_caller(cuda_device):
    """A workspace given is used (and big enough at the size asked for)."""
    g = torch.Generator().manual_seed(7)
    mk = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(cuda_device)  # noqa: E731
    q, k, v = mk(1, 4, 1, 64), mk(1, 4, 3000, 64), mk(1, 4, 3000, 64)
    lam = (0.1 * torch.randn(4, 4, 32, generator=g)).to(cuda_device)
    x, w = mk(10, 33), mk(20, 33)
    lib = jattn.load()
    need = lib.jattn_fwd_diff_workspace(jattn._DIFF_SHAPE.pack(1, 4, 4, 1, 3000, 64, *q.stride()[:3], *k.stride()[:3],
                                                               *v.stride()[:3]), jattn.BF16)
    need_y = lib.jattn_linear_workspace(jattn._LINEAR_SHAPE.pack(10, 20, 33, 33, 33, 20, 20, 0, 0, 0, 0), x.data_ptr(),
                                        w.data_ptr())
    assert need > 0 and need_y == 1024 + 1792
    for n, f in ((need, lambda ws: jattn.fwd_diff(q, k, v, lam, INIT, workspace=ws)[0]),
                 (need_y, lambda ws: jattn.linear(x, w, workspace=ws))):
        ws = torch.full((n + 512,), 77, dtype=torch.uint8, device=cuda_device)
        assert torch.equal(f(ws[:n]), f(None)) and (ws[n:] == 77).all() and not (ws[:n] == 77).all()
        with pytest.raises(ValueError):
            f(ws[:n - 1])
