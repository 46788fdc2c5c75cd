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
