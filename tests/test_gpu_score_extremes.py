"""Caps, slopes and distances at the ends of their ranges."""
import math

import pytest
import torch

from image_dits_b200 import rf2
from layer_ref import HALF, Shape, attention, attention_tolerance, backward_tolerance, csr_of, scores

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _inputs(sh, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = [torch.randn((sh.batch, sh.heads, sh.n, sh.dim), generator=g, device=DEV) for _ in range(4)]
    return [(t * scale if i < 2 else t).bfloat16() for i, t in enumerate(x)]


def _run(sh, q, k, v, do, mod):
    kept = torch.ones((sh.batch * sh.heads, sh.blocks, sh.blocks), dtype=torch.bool, device=DEV)
    mask = csr_of(sh, kept)
    lse = torch.empty((sh.batch, sh.heads, sh.n), device=DEV)
    o = rf2.block_sparse_attn_mod(sh.geometry(), q, k, v, mask, mod, lse=lse)
    grads = rf2.block_sparse_attn_backward(sh.geometry(), q, k, v, o, lse, do, mask, mod)
    assert rf2.device_status() == rf2.RF2_OK
    return o, lse, grads


@pytest.mark.parametrize("slope", [-300.0, -1000.0, 1000.0, 3e7])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("n", [67, 129, 131, 257, 1027])
@pytest.mark.parametrize("dim", [64, 128])
def test_slopes_of_any_size(dim, n, masked, slope):
    """A bias that leaves each row the token(s) furthest from it (or itself alone), one grid row, so that
    the sequence ends inside a group of neighbours; scores too large for anything but a one-hot softmax."""
    sh = Shape(1, 2, dim, 1, 1, n, (1, 1, n))
    q, k, v, do = _inputs(sh, n)
    doc = torch.zeros((1, n), dtype=torch.int32, device=DEV) if masked else None
    o, lse, grads = _run(sh, q, k, v, do, rf2.ScoreMod(slopes=torch.full((2,), slope, device=DEV), document=doc))
    i = torch.arange(n, device=DEV)
    if slope > 0:
        src = i
    else:
        # the furthest token is an end of the row; the middle one of an odd row has two
        src = torch.where(2 * i < n - 1, n - 1, 0)
    one = torch.ones(n, dtype=torch.bool, device=DEV)
    if slope < 0 and n % 2:
        one[n // 2] = False
    assert torch.equal(o[:, :, one], v[:, :, src[one]])
    for x in (o, lse, *grads):
        assert torch.isfinite(x.float()).all()
    # dV: one-hot rows add their dO (the middle row's is dealt out over both ends)
    want = torch.zeros(v.shape, dtype=torch.float64, device=DEV)
    want.index_add_(2, src[one], do.double()[:, :, one])
    rest = torch.zeros_like(want)
    rest.index_add_(2, torch.tensor([0, n - 1], device=DEV), do.double().abs()[:, :, ~one].sum(2, keepdim=True).expand(-1, -1, 2, -1))
    mag = torch.zeros_like(want).index_add_(2, src, do.double().abs())
    # the log-sum-exp of a score s is good to 2^-24 s, and so are the probabilities' logarithms
    p = 2 ** (abs(slope) * n * 1.5 * 2.0 ** -23) - 1 if slope < 0 else 1e-3
    if p < 0.1:
        assert ((grads[2].double() - want).abs() <= rest * (1 + p) + (p + HALF) * mag + HALF * want.abs() + 1e-6).all()


@pytest.mark.parametrize("cap", [0.05, 1.0, 999.0, 1e4, 1.001e4, 1e6])
@pytest.mark.parametrize("dim", [64, 128])
def test_caps_of_any_size(dim, cap):
    sh = Shape(1, 2, dim, 3, 5, 9, (2, 4, 4))
    q, k, v, do = _inputs(sh, dim, 1.5)
    o, lse, grads = _run(sh, q, k, v, do, rf2.ScoreMod(softcap=cap))
    perm = sh.perm(DEV)
    vis = torch.ones((1, 2, sh.n, sh.n), dtype=torch.bool, device=DEV)
    ref, rlse, p = attention(sh, q.double(), k.double(), v.double(), vis, perm, softcap=cap)
    assert ((o.double() - ref).abs() <= attention_tolerance(p, v.double(), ref)).all()
    assert ((lse.double() - rlse).abs() <= 1e-3).all()
    qd, kd, vd = (x.double().requires_grad_() for x in (q, k, v))
    p = torch.softmax(scores(sh, qd, kd, perm, softcap=cap), -1)
    ref = p @ vd
    ref.backward(do.double())
    with torch.no_grad():
        raw = qd @ kd.transpose(-1, -2) / math.sqrt(dim)
        slope = 1 / torch.cosh(raw / cap) ** 2
        # the slope's relative error is 2 |x| that of x where tanh is saturated, or 2 (error of raw) / cap:
        # raw is off by at most d 2^-24 sum |q k| / sqrt(d)
        off = 2 * dim * 2.0 ** -24 * (qd.abs() @ kd.abs().transpose(-1, -2)) / math.sqrt(dim) / cap
        dp = do.double() @ vd.transpose(-1, -2)
        extra = p * slope * off * (dp - (do.double() * ref).sum(-1, keepdim=True)).abs() / math.sqrt(dim)
        tols = backward_tolerance(sh, qd, kd, vd, ref, do.double(), p, slope)
        more = (extra @ kd.abs(), extra.transpose(-1, -2) @ qd.abs(), 0.0)
        for name, a, b, tol, m in zip("qkv", grads, (qd.grad, kd.grad, vd.grad), tols, more):
            assert ((a.double() - b).abs() <= tol + m + HALF * b.abs() + 1e-6).all(), name


def test_smallest_cap():
    """1e-3: every score is the cap or minus it, so rows are near their mean over V, and nearly flat."""
    sh = Shape(1, 2, 64, 3, 5, 9, (2, 4, 4))
    q, k, v, do = _inputs(sh, 3, 2.0)
    o, lse, grads = _run(sh, q, k, v, do, rf2.ScoreMod(softcap=1e-3))
    # P is within e^(+-2e-3) of 1/n
    mean = v.double().mean(2, keepdim=True)
    tol = (2.1e-3 + 2.0 ** -8) * v.double().abs().mean(2, keepdim=True) + HALF * mean.abs() + 1e-6
    assert ((o.double() - mean).abs() <= tol).all()
    assert ((lse - math.log(sh.n)).abs() <= 1.1e-3).all()
    assert all(torch.isfinite(x.float()).all() for x in grads)
