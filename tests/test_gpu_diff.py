"""Differential attention against the fp64 oracle.

Tolerance per element: half a step of the bf16 output, plus the oracle's
first-order bound for probabilities that are off by u = half a step of the
operand type (P is rounded to it) + 2^-13 (the fp32 logits: d / 2 products of
up to 2^-23 of sum |q k| each, 64 * 2^-23 * 64 * scale at most, and exp2's
2^-22), twice for the terms of second order.  The log-sum-exp moves by 2^-13."""
import numpy as np
import pytest
import torch

import oracle.layer as ref
from diffusion_transformer_joint_jattn_b200 import jattn

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
INIT, EPS = 0.35, 1e-5


def make(dev, dtype, B, H, H_kv, S_q, S_kv, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    mk = lambda h, s: torch.randn(B, h, s, d, generator=g).to(DT[dtype]).to(dev)  # noqa: E731
    lam = (0.2 * torch.randn(4, H, d // 2, generator=g)).to(dev)
    return mk(H, S_q), mk(H_kv, S_kv), mk(H_kv, S_kv), lam, (1 + 0.1 * torch.randn(d, generator=g)).to(dev)


def check(o, lse, q, k, v, lam, w, allowed=None, scale=None):
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    u = torch.finfo(q.dtype).eps / 2 + 2.0 ** -13
    want, lref, bound = ref.diff_attention(f(q), f(k), f(v), f(lam), INIT, None if w is None else f(w), EPS, allowed,
                                           scale, u)
    err = np.abs(f(o) - want)
    tol = 2.0 ** -8 * np.abs(want) + 2 * bound + 1e-6
    assert (err <= tol).all(), float((err / tol).max())
    if lse is not None:
        l = f(lse)
        assert (np.isneginf(l) == np.isneginf(lref)).all()
        live = np.isfinite(lref)
        assert np.abs(l[live] - lref[live]).max(initial=0.0) <= 2.0 ** -13
    assert jattn.device_status()[0] == jattn.OK


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,H_kv,S_q,S_kv", [
    (1, 1, 1, 1, 1), (1, 2, 2, 288, 288), (2, 4, 2, 1, 700), (3, 6, 2, 5, 129), (1, 3, 1, 130, 127), (2, 2, 1, 257, 385),
    (1, 4, 4, 1, 5000), (1, 8, 1, 16, 4100), (1, 2, 2, 64, 1),
])
def test_sizes(cuda_device, dtype, d, B, H, H_kv, S_q, S_kv):
    q, k, v, lam, w = make(cuda_device, dtype, B, H, H_kv, S_q, S_kv, d)
    for norm in (w, None):
        o, lse = jattn.fwd_diff(q, k, v, lam, INIT, norm_w=norm, eps=EPS, want_lse=True)
        check(o, lse, q, k, v, lam, norm)


@pytest.mark.parametrize("S_q,S_kv", [(1, 3000), (40, 3000), (150, 300)])
def test_lengths(cuda_device, S_q, S_kv):
    """Lengths of 0, 1, inside a tile, at its end, all, and past the cache; the
    rest of the cache holds NaN and infinities."""
    lens = [0, 1, 100, 128, 129, S_kv - 1, S_kv, S_kv + 50]
    q, k, v, lam, w = make(cuda_device, "bf16", len(lens), 4, 2, S_q, S_kv, 128)
    allowed = np.arange(S_kv)[None] < np.array(lens)[:, None]
    for b, n in enumerate(lens):
        k[b, :, n:] = float("nan")
        v[b, :, n:] = float("inf")
    n = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    o, lse = jattn.fwd_diff(q, k, v, lam, INIT, norm_w=w, eps=EPS, kv_len=n, want_lse=True)
    clean = lambda t: torch.where(torch.from_numpy(allowed).to(t.device)[:, None, :, None], t, 0)  # noqa: E731
    check(o, lse, q, clean(k), clean(v), lam, w, allowed)
    assert (o[0] == 0).all() and torch.isneginf(lse[:, 0]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S_q", [1, 9, 16, 17])
def test_many_sequences(cuda_device, dtype, d, S_q):
    """More ranges than SMs over caches of unequal length, empty ones among
    them: a CTA walks whole ranges and parts of others in one go.  16 queries
    of two heads are the 32 rows of the few-row kernel, 17 are past it."""
    B, S_kv = 80, 1100
    q, k, v, lam, w = make(cuda_device, dtype, B, 4, 2, S_q, S_kv, d, seed=S_q)
    lens = np.random.default_rng(S_q).integers(0, S_kv + 1, B)
    lens[[3, 4, 41, 79]] = 0, 0, S_kv, 0
    allowed = np.arange(S_kv)[None] < lens[:, None]
    n = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    for norm in (w, None):
        o, lse = jattn.fwd_diff(q, k, v, lam, INIT, norm_w=norm, eps=EPS, kv_len=n, want_lse=True)
        check(o, lse, q, k, v, lam, norm, allowed)


@pytest.mark.parametrize("S_q", [1, 200])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3.0e38])
def test_key_mask(cuda_device, S_q, bad):
    """Padded text inside the joint sequence, whole masked tiles, scattered
    keys, a single key, none; masked rows of k and v hold what they like."""
    S = 900
    q, k, v, lam, w = make(cuda_device, "bf16", 5, 2, 2, S_q, S, 128, seed=1)
    allowed = np.ones((5, S), bool)
    allowed[0, 40:512] = False
    allowed[1] = np.random.default_rng(0).random(S) < 0.5
    allowed[2] = False
    allowed[2, 700] = True
    allowed[3] = False
    m = torch.from_numpy(allowed).to(cuda_device)
    kk, vv = (torch.where(m[:, None, :, None], t, torch.full_like(t, bad)) for t in (k, v))
    n = torch.tensor([900, 830, 900, 900, 384], dtype=torch.int32, device=cuda_device)
    both = allowed & (np.arange(S)[None] < n.cpu().numpy()[:, None])
    zero = lambda t: torch.where(torch.from_numpy(both).to(t.device)[:, None, :, None], t, 0)  # noqa: E731
    for mask in (m, m.to(torch.uint8) * 255):
        o, lse = jattn.fwd_diff(q, kk, vv, lam, INIT, norm_w=w, eps=EPS, kv_len=n, key_mask=mask, want_lse=True)
        check(o, lse, q, zero(k), zero(v), lam, w, both)
        assert (o[3] == 0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_long_walk(cuda_device, d):
    """Whole waves of items and a shared tail, bf16 V copied to fp16 with a power
    of two per head (here 2^-40 to 2^40, and a head of zeros), lengths and mask
    together; against the oracle on some of the heads."""
    B, H, S = 2, 24, 1050
    q, k, v, lam, w = make(cuda_device, "bf16", B, H, H, S, S, d, seed=11)
    e = torch.arange(B * H, device=cuda_device).view(B, H, 1, 1)
    v.mul_(torch.pow(2.0, (e % 9 - 4) * 10.0))
    v[1, 3] = 0
    lens = np.array([S, 700])
    allowed = np.random.default_rng(1).random((B, S)) < 0.9
    m = torch.from_numpy(allowed).to(cuda_device)
    v[0].masked_fill_(~m[0][None, :, None], float("nan"))
    allowed &= np.arange(S)[None] < lens[:, None]
    n = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    for norm in (None, w):
        o, lse = jattn.fwd_diff(q, k, v, lam, INIT, norm_w=norm, eps=EPS, kv_len=n, key_mask=m, want_lse=True)
        for h in (0, 3, 4, 8, 13, 23):
            vh = torch.nan_to_num(v[:, h:h + 1])
            if norm is None:
                # a power of two out of V is one out of O: held in the units of N(0, 1) values
                f = torch.pow(2.0, -(e[:, h:h + 1] % 9 - 4) * 10.0)
                check(o[:, :, h:h + 1].double() * f.transpose(1, 2), lse[:, :, h:h + 1], q[:, h:h + 1], k[:, h:h + 1],
                      vh.double() * f, lam[:, h:h + 1], norm, allowed)
            else:
                big = (e[:, h] % 9 - 4 >= 0).view(B)     # eps hides what is far below 1
                for b in range(B):
                    if big[b] or (b == 1 and h == 3):
                        s = slice(b, b + 1)
                        check(o[s, :, h:h + 1], lse[:, s, h:h + 1], q[s, h:h + 1], k[s, h:h + 1], vh[s], lam[:, h:h + 1],
                              norm, allowed[s])


def test_split_and_whole_walk_agree(cuda_device):
    """The same queries alone (keys split over CTAs) and among enough others to
    fill the GPU (one walk): within both forms' rounding of the output."""
    q, k, v, lam, w = make(cuda_device, "fp16", 1, 2, 2, 128 * 80, 2048, 128)
    a, la = jattn.fwd_diff(q, k, v, lam, INIT, norm_w=w, eps=EPS, want_lse=True)
    b, lb = jattn.fwd_diff(q[:, :, :100], k, v, lam, INIT, norm_w=w, eps=EPS, want_lse=True)
    assert torch.allclose(a[:, :100].float(), b.float(), rtol=2 * 2.0 ** -8, atol=4 * 2.0 ** -11)
    assert torch.allclose(la[..., :100], lb, rtol=0, atol=2.0 ** -13)


def test_strided_operands(cuda_device):
    """q, k and v as views of a fused [B, S, 3, H, d] projection, and a query
    tensor whose shared heads' rows are not equally spaced."""
    B, S, H, d = 2, 150, 4, 128
    qkv = torch.randn(B, S, 3, H, d, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).to(cuda_device)
    q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    _, _, _, lam, w = make(cuda_device, "bf16", B, H, H, 1, 1, d)
    o, lse = jattn.fwd_diff(q, k, v, lam, INIT, norm_w=w, eps=EPS, want_lse=True)
    same, _ = jattn.fwd_diff(q.contiguous(), k.contiguous(), v.contiguous(), lam, INIT, norm_w=w, eps=EPS)
    assert torch.equal(o, same)
    check(o, lse, q, k, v, lam, w)
    shared, _ = jattn.fwd_diff(q, k[:, :2], v[:, :2], lam, INIT, norm_w=w, eps=EPS)
    check(shared, None, q, k[:, :2], v[:, :2], lam, w)
    packed, _ = jattn.fwd_diff(q.contiguous(), k[:, :2], v[:, :2], lam, INIT, norm_w=w, eps=EPS)
    assert torch.equal(shared, packed)


def test_large_logits_and_scale(cuda_device):
    """Logits of hundreds: the running maximum moves far between tiles, and the
    softmax picks single keys.  fp32 logits of size L are off by 64 * 2^-23 of
    their magnitudes; at scale 1 and |q k| sums of up to 4000 that is 2^-5."""
    q, k, v, lam, _ = make(cuda_device, "fp16", 1, 2, 2, 130, 600, 128, seed=5)
    for t in (q, k):
        t.mul_(2)
    o, lse = jattn.fwd_diff(q, k, v, lam, INIT, want_lse=True, softmax_scale=1.0)
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    want, lref, _ = ref.diff_attention(f(q), f(k), f(v), f(lam), INIT, scale=1.0)
    assert np.abs(f(lse) - lref).max() <= 2.0 ** -5
    assert np.linalg.norm(f(o) - want) <= (2.0 ** -8 + 2.0 ** -5) * np.linalg.norm(want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S_q", [1, 4, 5, 16])
def test_few_rows_by_key_columns(cuda_device, dtype, d, S_q):
    """2 S_q rows, whose keys are spread over warps by their place in a half of
    64: masks that leave one warp keys, all but one, a last half of few keys,
    and one key alone; masked rows of k and v hold NaN."""
    S = 1000
    q, k, v, lam, w = make(cuda_device, dtype, 12, 2, 1, S_q, S, d, seed=S_q)
    place = np.arange(S) % 64
    allowed = np.stack([place // 16 == i for i in range(4)] + [place // 16 != i for i in range(4)] +
                       [place < 32, place >= 32, place == 47, np.arange(S) == 990])
    m = torch.from_numpy(allowed).to(cuda_device)
    kk, vv = (torch.where(m[:, None, :, None], t, torch.full_like(t, float("nan"))) for t in (k, v))
    zero = lambda t: torch.where(m[:, None, :, None], t, 0)  # noqa: E731
    o, lse = jattn.fwd_diff(q, kk, vv, lam, INIT, norm_w=w, eps=EPS, key_mask=m, want_lse=True)
    check(o, lse, q, zero(k), zero(v), lam, w, allowed)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("S_q", [1, 4, 16])
def test_few_rows_large_logits(cuda_device, dtype, S_q):
    """As test_large_logits_and_scale: the maxima of a row's key columns move by
    themselves, in one CTA and across several."""
    for S in (600, 2300):
        q, k, v, lam, _ = make(cuda_device, dtype, 2, 4, 2, S_q, S, 128, seed=5)
        for t in (q, k):
            t.mul_(2)
        o, lse = jattn.fwd_diff(q, k, v, lam, INIT, want_lse=True, softmax_scale=1.0)
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        want, lref, _ = ref.diff_attention(f(q), f(k), f(v), f(lam), INIT, scale=1.0)
        assert np.abs(f(lse) - lref).max() <= 2.0 ** -5
        assert np.linalg.norm(f(o) - want) <= (2.0 ** -8 + 2.0 ** -5) * np.linalg.norm(want)


@pytest.mark.parametrize("d", [64, 128])
def test_few_rows_repeat(cuda_device, d):
    """CTAs that go from range to range reuse the memory of the queries: the
    same call gives the same bits every time."""
    q, k, v, lam, w = make(cuda_device, "bf16", 96, 4, 2, 9, 300, d)
    n = torch.arange(96, dtype=torch.int32, device=cuda_device) * 3 + 1
    first, l0 = jattn.fwd_diff(q, k, v, lam, INIT, norm_w=w, kv_len=n, want_lse=True)
    check(first, l0, q, k, v, lam, w, np.arange(300)[None] < n.cpu().numpy()[:, None])
    for _ in range(50):
        o, lse = jattn.fwd_diff(q, k, v, lam, INIT, norm_w=w, kv_len=n, want_lse=True)
        assert torch.equal(o, first) and torch.equal(lse, l0)


def test_nan_and_infinite_logits_stay_in_their_rows(cuda_device):
    """A query of NaN, one whose logit with some key is +inf, in every column of a
    key half (some exponentials are computed another way): NaN in that row's
    output and log-sum-exp, the other rows as they were."""
    for S_q in (3, 70):
        q, k, v, lam, w = make(cuda_device, "fp16", 1, 1, 1, S_q, 64, 128)
        clean, lse = jattn.fwd_diff(q, k, v, lam, INIT, norm_w=w, want_lse=True)
        for col in range(64):
            q2, k2 = q.clone(), k.clone()
            q2[0, 0, 0, 5] = float("nan")
            k2[0, 0, col, 70] = float("inf")              # map 2: +inf where q's channel is positive
            q2[0, 0, 1, 70], q2[0, 0, 2:, 70] = 1.0, 0.0
            k3 = k2.clone()
            k3[0, 0, col, 70] = 0.0
            o, l = jattn.fwd_diff(q2, k2, v, lam, INIT, norm_w=w, want_lse=True)
            assert torch.isnan(o[0, 0]).all() and torch.isnan(o[0, 1]).all() and torch.isnan(l[0, 0, 0, 0])
            assert torch.isnan(l[1, 0, 0, 1])
            o3, _ = jattn.fwd_diff(q2, k3, v, lam, INIT, norm_w=w)
            assert torch.isfinite(o3[0, 1:]).all()
        assert torch.isfinite(clean).all()


def test_no_keys_and_no_queries(cuda_device):
    q, k, v, lam, w = make(cuda_device, "bf16", 2, 2, 1, 3, 4, 64)
    o, lse = jattn.fwd_diff(q, k[:, :, :0], v[:, :, :0], lam, INIT, norm_w=w, want_lse=True)
    assert (o == 0).all() and torch.isneginf(lse).all()
    o, lse = jattn.fwd_diff(q[:, :, :0], k, v, lam, INIT, want_lse=True)
    assert o.shape == (2, 0, 2, 64) and lse.shape == (2, 2, 2, 0)
    assert jattn.fwd_diff(q[:0], k[:0], v[:0], lam, INIT)[0].shape == (0, 3, 2, 64)


def test_outputs_in_place_and_what_surrounds_them(cuda_device):
    q, k, v, lam, w = make(cuda_device, "bf16", 1, 3, 1, 70, 200, 64)
    buf = torch.full((70 * 3 * 64 + 64,), 7.0, dtype=torch.bfloat16, device=cuda_device)
    o = buf[8:8 + 70 * 192].view(1, 70, 3, 64)                 # 16-byte, not 32-byte aligned
    lse = torch.full((2, 1, 3, 70), 7.0, device=cuda_device)
    got, l = jattn.fwd_diff(q, k, v, lam, INIT, norm_w=w, eps=EPS, o=o, lse=lse)
    assert got is o and l is lse
    check(o, lse, q, k, v, lam, w)
    assert (buf[:8] == 7).all() and (buf[8 + 70 * 192:] == 7).all()


def test_refusals(cuda_device):
    q, k, v, lam, w = make(cuda_device, "bf16", 2, 4, 2, 3, 9, 128)
    ok = dict(q=q, k=k, v=v, lam=lam, lambda_init=INIT, norm_w=w)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=cuda_device)  # noqa: E731
    for bad in (dict(q=q.cpu()), dict(q=q.float()), dict(k=k.half()), dict(v=v[:, :, :4]), dict(q=q[0]),
                dict(lam=lam[:3]), dict(lam=lam.cpu()), dict(norm_w=w[:64]), dict(kv_len=i32(3)),
                dict(kv_len=i32(2).long()), dict(key_mask=i32(2, 9)), dict(key_mask=i32(2, 8).bool()),
                dict(o=torch.empty(2, 3, 4, 128, device=cuda_device)), dict(lse=torch.empty(2, 4, 3, device=cuda_device)),
                dict(q=q.transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises(ValueError):
            jattn.fwd_diff(**dict(ok, **bad))
    for bad in (dict(eps=0.0), dict(lambda_init=float("inf")), dict(softmax_scale=float("nan")),
                dict(q=q[:, :3], lam=lam[:, :3].contiguous()), dict(k=k[:, :1].expand(2, 2, 9, 128), v=v)):
        with pytest.raises(jattn.JattnError):
            jattn.fwd_diff(**dict(ok, **bad))
    q1, k1, v1, lam1, _ = make(cuda_device, "bf16", 1, 1, 1, 1, 4096, 128)
    with pytest.raises(ValueError):
        jattn.fwd_diff(q1, k1, v1, lam1, INIT, workspace=torch.empty(16, dtype=torch.uint8, device=cuda_device))


def test_other_stream_and_graph(cuda_device):
    for S_q in (1, 300):
        q, k, v, lam, w = make(cuda_device, "bf16", 1, 4, 2, S_q, 3000, 128)
        want, _ = jattn.fwd_diff(q, k, v, lam, INIT, norm_w=w)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got, _ = jattn.fwd_diff(q, k, v, lam, INIT, norm_w=w, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)
        graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
        outs = []
        for g in graphs:
            with torch.cuda.graph(g):
                outs.append(jattn.fwd_diff(q, k, v, lam, INIT, norm_w=w)[0])
        q.neg_()
        for g in graphs:
            g.replay()
        want, _ = jattn.fwd_diff(q, k, v, lam, INIT, norm_w=w)
        assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("S_q", [1, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_full_and_short_caches_in_turn(cuda_device, dtype, d, S_q):
    """CTAs that go from caches without a masked key to short or masked ones and
    back: the V tiles of both kinds share one ring, and the rows that take no
    part hold NaN.  The same bits every time."""
    B, S = 90, 1500
    q, k, v, lam, w = make(cuda_device, dtype, B, 4, 2, S_q, S, d, seed=d)
    lens = np.where(np.arange(B) % 3 == 1, S, np.arange(B) * 97 % (S - 1))
    lens[20:30] = S
    allowed = np.arange(S)[None] < lens[:, None]
    n = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    keep = torch.from_numpy(allowed).to(cuda_device)[:, None, :, None]
    bad = torch.full_like(v, float("nan"))
    vv, kk = torch.where(keep, v, bad), torch.where(keep, k, bad)
    zero = torch.zeros_like(v)
    o, lse = jattn.fwd_diff(q, kk, vv, lam, INIT, norm_w=w, eps=EPS, kv_len=n, want_lse=True)
    check(o, lse, q, torch.where(keep, k, zero), torch.where(keep, v, zero), lam, w, allowed)
    for _ in range(20):
        again, _ = jattn.fwd_diff(q, kk, vv, lam, INIT, norm_w=w, eps=EPS, kv_len=n)
        assert torch.equal(again, o)


def of_rows(q, k, v, lam, b, h, rows, allowed=None):
    """The definition in fp64 on the GPU, without the norm, of some rows of one
    head: (o [rows, d], lse [2, rows])."""
    n, d = h // (q.shape[1] // k.shape[1]), q.shape[3]
    keep = slice(None) if allowed is None else allowed[b]
    kk, vv = k[b, n][keep], v[b, n][keep].double()
    f = [1.0, -(torch.exp(lam[0, h].double() @ lam[1, h].double()) - torch.exp(lam[2, h].double() @ lam[3, h].double())
                + INIT)]
    o, lse = 0.0, []
    for m in range(2):
        ch = slice(m * d // 2, (m + 1) * d // 2)
        t = q[b, h, rows][:, ch].double() @ kk[:, ch].double().t() / (d // 2) ** 0.5
        lse.append(torch.logsumexp(t, -1))
        o = o + f[m] * (torch.softmax(t, -1) @ vv)
    return o, torch.stack(lse)


# Forms of the walk over 2^18 to 2^20 keys: (dtype, H, H_kv, S_q, S_kv).  One range of 148 row tiles, walked whole
# (bf16: V copied to fp16); 50 ranges of three row tiles, some whole and the others shared (bf16: P in two parts); one
# query per head, each CTA with more than 2^15 keys of a cache.
LONG = [("fp16", 1, 1, 148 * 128, 1 << 20), ("bf16", 1, 1, 148 * 128, 1 << 20), ("bf16", 50, 1, 300, 1 << 18),
        ("fp16", 50, 1, 300, 1 << 18), ("bf16", 16, 8, 1, 1 << 20), ("fp16", 16, 8, 1, 1 << 20)]


def make_long(dev, dtype, H, H_kv, S_q, S_kv):
    g = torch.Generator(device=dev).manual_seed(S_kv + H)
    mk = lambda *s: torch.randn(*s, generator=g, device=dev, dtype=DT[dtype])  # noqa: E731
    q = mk(1, S_q, H, 128).transpose(1, 2)                     # shared heads' rows not equally spaced: a range per head
    lam = 0.2 * torch.randn(4, H, 64, generator=g, device=dev)
    return q, mk(1, H_kv, S_kv, 128), mk(1, H_kv, S_kv, 128), lam


@pytest.mark.parametrize("dtype,H,H_kv,S_q,S_kv", LONG)
def test_long_walks_keep_their_sums(cuda_device, dtype, H, H_kv, S_q, S_kv):
    """V the same at every key: every row's output is (1 - lambda) V, up to its
    rounding and what the accumulator loses in runs of 2^15 keys -- for each 16
    keys at most two units of 2^-23 of a sum that grows evenly, 2^-12."""
    q, k, v, _ = make_long(cuda_device, dtype, H, H_kv, S_q, S_kv)
    c = (1 + torch.arange(128, device=cuda_device) / 128).to(DT[dtype])
    v.copy_(c)
    o, lse = jattn.fwd_diff(q, k, v, torch.zeros(4, H, 64, device=cuda_device), INIT, want_lse=True)
    err = (o.double() / ((1 - INIT) * c.double()) - 1).abs()
    assert err.max() <= 2.0 ** -8 + 2.0 ** -11
    assert torch.isfinite(lse).all() and jattn.device_status()[0] == jattn.OK


@pytest.mark.parametrize("dtype,H,H_kv,S_q,S_kv", LONG)
@pytest.mark.parametrize("how", ["growing", "masked"])
def test_long_walks_against_the_definition(cuda_device, dtype, H, H_kv, S_q, S_kv, how):
    """Maxima that move from run to run (keys that grow along the cache), and a
    cache whose first runs, and most of the others, are masked.  The output's
    rounding is spread evenly over a step, 2^-7 of a value with mantissa 1: at
    most 2^-7 / sqrt(12) = 2.26e-3 in the L2 norm (outputs near 0.0713, mantissa
    1.14, have 1.98e-3 of it); P's in fp16 adds 2e-4: 2.5e-3 together."""
    q, k, v, lam = make_long(cuda_device, dtype, H, H_kv, S_q, S_kv)
    v += 0.5
    kw, allowed = {}, None
    if how == "growing":
        k *= torch.linspace(0.2, 2.0, S_kv, device=cuda_device).to(k.dtype)[:, None]    # linspace in fp16 is NaN
    else:
        m = torch.rand(1, S_kv, generator=torch.Generator(device=cuda_device).manual_seed(1), device=cuda_device) < 0.1
        m[:, :S_kv // 3] = False
        n = S_kv - 1000
        kw = dict(key_mask=m, kv_len=torch.tensor([n], dtype=torch.int32, device=cuda_device))
        allowed = m & (torch.arange(S_kv, device=cuda_device) < n)
        v.masked_fill_(~allowed[:, None, :, None], float("nan"))
    o, lse = jattn.fwd_diff(q, k, v, lam, INIT, want_lse=True, **kw)
    for h in {0, H // 2, H - 1}:
        rows = torch.tensor(sorted({0, S_q // 3, S_q - 1}), device=cuda_device)
        want, lref = of_rows(q, k, v, lam, 0, h, rows, allowed)
        assert (o[0, rows, h].double() - want).norm() <= 2.5e-3 * want.norm()
        assert (lse[:, 0, h][:, rows].double() - lref).abs().max() <= 2.0 ** -13
    assert jattn.device_status()[0] == jattn.OK


def near(o, want):
    """As near to `want` in the L2 norm as its own rounding to bf16, plus 2^-12:
    P in fp16 is off by 2^-11 / sqrt(3) = 2.8e-4 at most (evenly spread over a
    step), which adds to the rounding's 1.5e-3 or more as squares do, 3e-5; P as
    the sum of two bf16 by 2^-18, logits by 2^-16.  P in bf16 alone would add
    0.7e-3 (1.7e-3 as squares), a key of 64 left out 0.1."""
    own = (want.to(torch.bfloat16).double() - want).norm() / want.norm()
    return ((o.double() - want).norm() / want.norm() <= own + 2.0 ** -12).item()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,H_kv,S_q,S_kv", [(1, 2, 2, 1, 5000), (1, 4, 1, 8, 3001), (2, 2, 2, 40, 5000),
                                               (1, 2, 1, 300, 4100), (1, 40, 40, 512, 2400), (60, 4, 2, 9, 700)])
def test_precision_of_the_probabilities(cuda_device, dtype, d, B, H, H_kv, S_q, S_kv):
    """Long rows, V random, and V zero but for one 64-key half at a time (the
    first ones, both of a tile in the middle, the last): every half's keys meet
    their own V rows, with all the precision that P is held in."""
    q, k, v, lam, _ = make(cuda_device, dtype, B, H, H_kv, S_q, S_kv, d, seed=S_kv)
    rows = torch.arange(S_q, device=cuda_device)
    last = (S_kv - 1) // 64
    for half in (None, 0, 1, last // 2, last // 2 + 1, last):
        vv = v
        if half is not None:
            vv = torch.zeros_like(v)
            vv[:, :, 64 * half:64 * half + 64] = v[:, :, 64 * half:64 * half + 64]
        o, _ = jattn.fwd_diff(q, k, vv, lam, INIT)
        for b, h in {(0, 0), (B // 2, H // 2), (B - 1, H - 1)}:
            assert near(o[b, :, h], of_rows(q, k, vv, lam, b, h, rows)[0]), (half, b, h)


@pytest.mark.parametrize("dtype,G,H_kv", [("bf16", 2, 19), ("bf16", 2, 23), ("bf16", 1, 38), ("bf16", 1, 45), ("fp16", 2, 23),
                                          ("fp16", 1, 45)])
@pytest.mark.parametrize("d", [64, 128])
def test_whole_items_and_a_shared_tail(cuda_device, dtype, d, G, H_kv):
    """Ranges of several row tiles, most walked whole and the last wave shared by
    all CTAs; with two heads per K/V head (four row tiles) a bf16 V is copied to
    fp16 by powers of two, else P is in two parts.  Lengths and a mask, NaN in
    masked rows; the tail's rows against the definition."""
    B, S_q, S_kv = 2, 250, 2300
    n_rt, tiles = -(-G * S_q // 128), -(-S_kv // 128)
    items, sms = B * H_kv * n_rt, torch.cuda.get_device_properties(0).multi_processor_count
    rest = items % sms
    assert items > sms and rest > 0 and (sms - rest) * tiles > 8 * sms             # a tail that is shared
    q, k, v, lam, _ = make(cuda_device, dtype, B, G * H_kv, H_kv, S_q, S_kv, d, seed=H_kv)
    need = jattn.load().jattn_fwd_diff_workspace(
        jattn._DIFF_SHAPE.pack(B, G * H_kv, H_kv, S_q, S_kv, d, *q.stride()[:3], *k.stride()[:3], *v.stride()[:3]),
        jattn.BF16 if dtype == "bf16" else jattn.FP16)
    copy = 2 * v.numel() if dtype == "bf16" and n_rt >= 4 and items * tiles >= 18 * sms else 0
    assert (copy > 0) == (dtype == "bf16" and G == 2)
    assert 0 <= need - copy - sms * 4 * 128 * (d + 1) * 4 < 4096
    v *= 2.0 ** (5.0 * (torch.arange(B * H_kv, device=cuda_device).view(B, H_kv, 1, 1) % 5 - 2))
    n = torch.tensor([S_kv, 2100], dtype=torch.int32, device=cuda_device)
    m = torch.rand(B, S_kv, generator=torch.Generator().manual_seed(1)).to(cuda_device) < 0.9
    allowed = m & (torch.arange(S_kv, device=cuda_device) < n[:, None])
    v.masked_fill_(~allowed[:, None, :, None], float("nan"))
    o, lse = jattn.fwd_diff(q, k, v, lam, INIT, kv_len=n, key_mask=m, want_lse=True)
    rows = torch.arange(S_q, device=cuda_device)
    whole = (items - rest) // n_rt // H_kv, (items - rest) // n_rt % H_kv * G      # where the tail begins
    for b, h in [(0, 0), whole] + [(B - 1, G * H_kv - i) for i in (1, 2, 3, 8)]:
        want, lref = of_rows(q, k, v, lam, b, h, rows, allowed)
        assert near(o[b, :, h], want), (b, h)
        assert (lse[:, b, h].double() - lref).abs().max() <= 2.0 ** -13
    again, _ = jattn.fwd_diff(q, k, v, lam, INIT, kv_len=n, key_mask=m)
    assert torch.equal(again, o) and jattn.device_status()[0] == jattn.OK


def test_long_walks_at_once_and_captured(cuda_device):
    """Calls whose accumulators are emptied on the way have sums of their own: two
    captured graphs replayed at the same time, with new queries, and eager calls
    on two streams, give the bits of one call alone."""
    for H, H_kv, S_q, S_kv in ((1, 1, 148 * 128, 70000), (8, 8, 1, 1 << 20)):
        q, k, v, lam = make_long(cuda_device, "bf16", H, H_kv, S_q, S_kv)
        streams = [torch.cuda.Stream() for _ in range(2)]
        graphs, outs = [torch.cuda.CUDAGraph() for _ in streams], []
        jattn.fwd_diff(q, k, v, lam, INIT)
        torch.cuda.synchronize()
        for g in graphs:
            with torch.cuda.graph(g):
                outs.append(jattn.fwd_diff(q, k, v, lam, INIT, want_lse=True))
        q.neg_()
        torch.cuda.synchronize()
        for _ in range(3):
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
        eager = [jattn.fwd_diff(q, k, v, lam, INIT, want_lse=True, stream=s) for s in streams]
        torch.cuda.synchronize()
        want = jattn.fwd_diff(q, k, v, lam, INIT, want_lse=True)
        assert all(torch.equal(a, b) for got in outs + eager for a, b in zip(got, want))
    assert jattn.device_status()[0] == jattn.OK
