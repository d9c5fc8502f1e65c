"""Gradient of norm + rotation: eps = 0, and rows without a gradient."""
import pytest
import torch

from image_dits_b200 import rf2
from layer_ref import HALF, Shape, angles, norm_rope

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _inputs(sh, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    xs = [torch.randn((sh.batch, sh.heads, sh.n, sh.dim), generator=g, device=DEV).bfloat16() for _ in range(5)]
    return xs, [1 + 0.4 * torch.randn(sh.dim, generator=g, device=DEV) for _ in range(2)]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("shape", [(1, 1, 1, 0), (1, 7, 9, 0), (5, 1, 13, 0), (3, 7, 9, 11), (1, 8, 8, 0)], ids=str)
def test_backward_with_eps_zero(shape, interleaved, dim):
    f, h, w, text = shape
    sh = Shape(2, 3, dim, f, h, w, (1, 4, 4), f > 1, text)
    g, perm, ang = sh.geometry(), sh.perm(DEV), angles(sh, DEV)
    (q, k, dqp, dkp, dvp), ws = _inputs(sh, 1)
    rope = rf2.rope_table(g, sh.split(), device=DEV)
    dq, dk, dv, dwq, dwk = rf2.norm_rope_permute_backward(g, q, k, dqp, dkp, dvp, q_weight=ws[0], k_weight=ws[1], rope=rope,
                                                          eps=0.0, interleaved=interleaved)
    for x, ww, dy, dx, dw in ((q, ws[0], dqp, dq, dwq), (k, ws[1], dkp, dk, dwk)):
        xr, wr = x.double().requires_grad_(), ww.double().requires_grad_()
        norm_rope(sh, xr, wr, ang, 0.0, interleaved)[:, :, perm].backward(dy.double())
        r = 1 / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True))
        # dx: one bf16 rounding; fp32 arithmetic on r |dy| |w| (the subtraction can cancel)
        back = torch.empty_like(r)
        back[:, :, perm] = (dy.double().abs().amax(-1)[..., None] * ww.double().abs().amax() * 2)
        assert ((dx.double() - xr.grad).abs() <= HALF * xr.grad.abs() + 2.0 ** -17 * r * back * 4).all()
        # dw: an fp32 sum of terms dz h; its error is below rows 2^-24 of their absolute sum
        zb = torch.zeros_like(x, dtype=torch.float64)
        zb[:, :, perm] = dy.double()
        mag = (norm_rope(sh, zb, None, -ang, 0.0, interleaved, False) * x.double() * r).abs().sum((0, 1, 2))
        assert ((dw.double() - wr.grad).abs() <= 2.0 ** -17 * mag + 1e-6).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38, 0.0])
def test_rows_without_a_gradient_add_nothing(value, dim):
    """Rows whose gradient is 0 (of either sign) throughout may hold anything; a row with one
    gradient that is not 0 counts."""
    sh = Shape(2, 3, dim, 3, 7, 9, (2, 4, 4), True, 11)
    g, perm = sh.geometry(), sh.perm(DEV)
    (q, k, dqp, dkp, dvp), ws = _inputs(sh, 2)
    rope = rf2.rope_table(g, sh.split(), device=DEV)
    dead = torch.zeros((sh.batch, 1, sh.n, 1), dtype=torch.bool, device=DEV)
    dead[:, :, -5:] = True
    dead[1, :, 40:90:3] = True
    dead[0, :, 64:128] = True
    dqp, dkp = (torch.where(dead[:, :, perm], -0.0, d).bfloat16() for d in (dqp, dkp))
    dqp[0, 1, 3] = 0
    dqp[0, 1, 3, 7] = 1.0                                  # one channel of a permuted row whose token is live or not:
    q2 = torch.where(dead, value, q).bfloat16()
    k2 = torch.where(dead, value, k).bfloat16()
    src = int(perm[3])
    q2[0, 1, src] = q[0, 1, src]                           # its x counts, so it is the same in both
    kw = dict(q_weight=ws[0], k_weight=ws[1], rope=rope, eps=0.0)
    want = rf2.norm_rope_permute_backward(g, q, k, dqp, dkp, dvp, **kw)
    got = rf2.norm_rope_permute_backward(g, q2, k2, dqp, dkp, dvp, **kw)
    for a, b in zip(got, want):
        assert torch.equal(a, b) and torch.isfinite(a.float()).all()
    assert (got[0][0, 1, src] != 0).any()
    rows = dead.expand(q.shape).clone()
    rows[0, 1, src] = False
    assert (got[0][rows] == 0).all() and (got[1][dead.expand(q.shape)] == 0).all()
    zero = torch.zeros_like(dqp)
    none = rf2.norm_rope_permute_backward(g, q2, k2, zero, zero, zero, **kw)
    assert all((x == 0).all() for x in none)


@pytest.mark.parametrize("dim", [64, 128])
def test_layer_gradient_with_anything_in_the_padding(dim):
    """All blocks kept (the ranking is over block means, padding included): a layer whose padding holds
    NaN has the gradients, those of the norm weights included, of one whose padding holds zeros."""
    sh = Shape(2, 2, dim, 3, 8, 9, (2, 4, 4), True, 20)
    g = sh.geometry()
    (q, k, v, do, _), ws = _inputs(sh, 3)
    i = torch.arange(sh.n, device=DEV)
    doc = torch.stack([torch.where(i >= sh.n - 4 - 3 * b, -1, 0) for b in range(sh.batch)]).int()
    pad = (doc < 0)[:, None, :, None]
    rope = rf2.rope_table(g, sh.split(), device=DEV)
    outs = []
    for value in (0.0, float("nan")):
        a, b, c, d = (torch.where(pad, value, x).bfloat16() for x in (q, k, v, do))
        o, st = rf2.layer_attention(g, a, b, c, 1.0, q_weight=ws[0], k_weight=ws[1], rope=rope, mod=rf2.ScoreMod(document=doc))
        outs.append((o, *rf2.layer_attention_backward(st, d)))
        assert rf2.device_status() == rf2.RF2_OK
    for a, b in zip(*outs):
        assert torch.isfinite(b.float()).all() and torch.equal(a, b)
    for x in outs[1][:4]:
        assert (x[pad.expand(x.shape)] == 0).all()
