"""The layer oracle's own pins: closed forms, invariants and library routines
that do not share its formulas."""
import math

import numpy as np
import torch

import oracle
import oracle.layer as layer

R = np.random.default_rng(0)


def test_rotary_is_a_rotation():
    x = R.standard_normal((2, 5, 3, 16))
    pos = R.integers(0, 100, (2, 5))
    w = 100.0 ** (-np.arange(4) / 4)
    for half in (False, True):
        y = layer.rotary(x, pos, w, half=half, parts=2)
        assert np.allclose(layer.rotary(y, pos, w, half=half, parts=2, inverse=True), x, atol=1e-14)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        # relative positions: q.k depends on the difference of positions alone
        k = layer.rotary(x[:, :, :1], pos + 7, w, half=half, parts=2)
        q = layer.rotary(x[:, :, 1:2], pos + 7, w, half=half, parts=2)
        k0, q0 = (layer.rotary(x[:, :, i:i + 1], pos, w, half=half, parts=2) for i in (0, 1))
        assert np.allclose((q * k).sum(-1), (q0 * k0).sum(-1))
    assert np.array_equal(layer.rotary(x, pos * 0, w), x)
    assert np.array_equal(layer.rotary(x, pos, w[:2])[..., 4:], x[..., 4:])


def test_rotary_quarter_turn_and_layouts():
    x = np.arange(1.0, 5.0).reshape(1, 1, 1, 4)
    w = np.array([math.pi / 2, 0.0])
    assert np.allclose(layer.rotary(x, np.ones((1, 1)), w)[0, 0, 0], [-2, 1, 3, 4])
    assert np.allclose(layer.rotary(x, np.ones((1, 1)), w, half=True)[0, 0, 0], [-3, 2, 1, 4])
    assert np.allclose(layer.rotary(x, np.ones((1, 1)), w, scale=2.0)[0, 0, 0], [-4, 2, 6, 8])


def test_rotary_axes_match_the_joint_oracle():
    S, split = 6, (4, 6, 6)
    x = R.standard_normal((1, S, 2, 16))
    pos = R.integers(0, 9, (S, 3))
    w = np.concatenate([10000.0 ** (-np.arange(n // 2) / (n / 2)) for n in split])
    axis = [0] * 2 + [1] * 3 + [2] * 3
    got = layer.rotary(x, np.broadcast_to(pos, (1, S, 3)), w, axis=axis)
    want = oracle.rope_rotate(x.transpose(0, 2, 1, 3), pos, split, 10000.0).transpose(0, 2, 1, 3)
    assert np.allclose(got, want, atol=1e-12)


def test_linear_and_activations_against_torch():
    x, w, b, r = (R.standard_normal(s) for s in ((7, 5), (3, 5), (3,), (7, 3)))
    t = lambda a: torch.from_numpy(a)  # noqa: E731
    y = torch.nn.functional.linear(t(x), t(w), t(b))
    F = torch.nn.functional
    for name, f in (("none", lambda v: v), ("gelu", F.gelu), ("gelu_tanh", lambda v: F.gelu(v, approximate="tanh")),
                    ("silu", F.silu), ("relu", F.relu)):
        assert np.allclose(layer.linear(x, w, b, name, r), (f(y) + t(r)).numpy(), atol=1e-13), name


def _diff(S_q=4, S_kv=9, H=4, H_kv=2, d=16):
    return (R.standard_normal((2, H, S_q, d)), R.standard_normal((2, H_kv, S_kv, d)),
            R.standard_normal((2, H_kv, S_kv, d)), 0.3 * R.standard_normal((4, H, d // 2)))


def test_diff_attention_is_two_attentions():
    q, k, v, lam = _diff()
    o, lse, _ = layer.diff_attention(q, k, v, lam, 0.25)
    t = lambda a: torch.from_numpy(a)  # noqa: E731
    kk, vv = (t(a).repeat_interleave(2, 1) for a in (k, v))
    sd = torch.nn.functional.scaled_dot_product_attention
    one, two = (sd(t(q)[..., c], kk[..., c], vv) for c in (slice(0, 8), slice(8, 16)))
    lh = np.exp((lam[0] * lam[1]).sum(-1)) - np.exp((lam[2] * lam[3]).sum(-1)) + 0.25
    want = one - t(lh)[None, :, None, None] * two
    assert np.allclose(o, want.transpose(1, 2).numpy(), atol=1e-13)
    s = torch.matmul(t(q)[..., 8:], kk[..., 8:].transpose(-1, -2)) / math.sqrt(8)
    assert np.allclose(lse[1], torch.logsumexp(s, -1).numpy(), atol=1e-13)


def test_diff_attention_invariants():
    q, k, v, lam = _diff()
    lh = np.exp((lam[0] * lam[1]).sum(-1)) - np.exp((lam[2] * lam[3]).sum(-1)) + 0.25
    o, _, _ = layer.diff_attention(q, k, np.ones_like(v), lam, 0.25)
    assert np.allclose(o, np.broadcast_to((1 - lh)[None, None, :, None], o.shape))      # constant V
    perm = R.permutation(9)
    a, la, _ = layer.diff_attention(q, k, v, lam, 0.25)
    b, lb, _ = layer.diff_attention(q, k[:, :, perm], v[:, :, perm], lam, 0.25)
    assert np.allclose(a, b) and np.allclose(la, lb)
    # masked keys are as if they were not there, whatever they hold
    allowed = np.ones((2, 9), bool)
    allowed[:, 5:] = False
    k2, v2 = k.copy(), v.copy()
    k2[:, :, 5:], v2[:, :, 5:] = np.nan, np.inf
    m, lm, _ = layer.diff_attention(q, k2, v2, lam, 0.25, allowed=allowed)
    c, lc, _ = layer.diff_attention(q, k[:, :, :5], v[:, :, :5], lam, 0.25)
    assert np.allclose(m, c) and np.allclose(lm, lc)
    z, lz, _ = layer.diff_attention(q, k, v, lam, 0.25, allowed=np.zeros((2, 9), bool), norm_w=np.ones(16))
    assert (z == 0).all() and np.isneginf(lz).all()


def test_diff_attention_norm_and_bound():
    q, k, v, lam = _diff()
    w = R.standard_normal(16)
    o, _, _ = layer.diff_attention(q, k, v, lam, 0.25)
    n, _, bound = layer.diff_attention(q, k, v, lam, 0.25, norm_w=w, eps=1e-12, u=1e-3)
    rms = np.sqrt(((n / (w * 0.75)) ** 2).mean(-1))
    assert np.allclose(rms, 1.0) and np.allclose(n / np.abs(n), o * w / np.abs(o * w))
    assert (bound > 0).all() and bound.max() < 0.1
