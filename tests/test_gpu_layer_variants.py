"""Compiled variants and ways through the kernels that the other files do not reach: every set of score
modifications at both head sizes, mask prediction in several groups of heads, and norm kernels with more
units to a CTA than it has warps."""
import math

import pytest
import torch

from image_dits_b200 import rf2
from layer_ref import (HALF, Shape, angles, attention, attention_tolerance, backward_tolerance, csr_of, norm_rope,
                       random_kept, scores, visible)

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("cap", [0.0, 12.0])
@pytest.mark.parametrize("dim", [64, 128])
def test_every_set_of_modifications(dim, cap, bias, masked):
    """5 blocks, the last of 4 tokens, text and a moved first frame, one row without kept blocks; raw
    scores on both sides of half the cap and of the cap."""
    sh = Shape(2, 2, dim, 4, 7, 8, (2, 4, 4), True, 36)
    assert sh.n % 64 == 4
    g = torch.Generator(device=DEV).manual_seed(dim)
    q, k, v, do = (torch.randn((sh.batch, sh.heads, sh.n, dim), generator=g, device=DEV) for _ in range(4))
    q, k = q * 2, k * 2
    q[0, 1] *= 2.5                                   # one head beyond the cap
    q, k, v, do = (x.bfloat16() for x in (q, k, v, do))
    i = torch.arange(sh.n, device=DEV)
    doc = order = None
    if masked:
        doc = torch.stack([((i + 5 * b) // 37) % 4 - 1 for b in range(sh.batch)]).int()
        order = (i - sh.n // 5).clamp(min=0).int()[None].repeat(sh.batch, 1)
    mod = rf2.ScoreMod(softcap=cap, slopes=0.7 * 0.5 ** torch.arange(sh.heads, device=DEV, dtype=torch.float32) if bias else None,
                       distance=(1.5, 0.5, 0.25), document=doc, order=order)
    kw = dict(softcap=cap, slopes=mod.slopes, distance=mod.distance)
    perm = sh.perm(DEV)
    kept = random_kept(sh, 0.6, 3, DEV, empty_rows=(1,))
    vis = visible(sh, kept, doc, order, perm)
    mask = csr_of(sh, kept)
    lse = torch.empty((sh.batch, sh.heads, sh.n), device=DEV)
    o = rf2.block_sparse_attn_mod(sh.geometry(), q, k, v, mask, mod, lse=lse)
    got = rf2.block_sparse_attn_backward(sh.geometry(), q, k, v, o, lse, do, mask, mod)
    assert rf2.device_status() == rf2.RF2_OK

    ref, rlse, p = attention(sh, q.double(), k.double(), v.double(), vis, perm, **kw)
    assert ((o.double() - ref).abs() <= attention_tolerance(p, v.double(), ref)).all()
    dead = rlse == -math.inf
    assert torch.equal(lse == -math.inf, dead) and (o[dead] == 0).all()
    assert ((lse.double() - rlse)[~dead].abs() <= 1e-3).all()
    qd, kd, vd = (x.double().requires_grad_() for x in (q, k, v))
    x = scores(sh, qd, kd, perm, **kw).masked_fill(~vis, -1e300)
    p = torch.softmax(x, -1) * vis
    ref = p @ vd
    ref.backward(do.double())
    with torch.no_grad():
        raw = qd @ kd.transpose(-1, -2) / math.sqrt(dim)
        if cap:
            assert float(raw[0, 1].abs().max()) > cap > 0.5 * cap > float(raw.abs().median())
        slope = 1 / torch.cosh(raw / cap) ** 2 if cap else torch.ones_like(raw)
        tols = backward_tolerance(sh, qd, kd, vd, ref, do.double(), p, slope)
        for name, a, b, tol in zip("qkv", got, (qd.grad, kd.grad, vd.grad), tols):
            err, bound = (a.double() - b).abs(), tol + HALF * b.abs() + 1e-6
            assert torch.isfinite(a.float()).all()
            assert (err <= bound).all(), (name, float((err - bound).max()))


def test_visible_prediction_over_groups_of_heads():
    """4,096 blocks: a head's scores fill a group of their own, so each head's visibility is looked up at
    an offset; three batch elements with documents and orders of their own."""
    sh = Shape(3, 1, 64, 16, 128, 128, (1, 8, 8))
    g, keep = sh.geometry(), 0.02
    assert sh.blocks == 4096
    gen = torch.Generator(device=DEV).manual_seed(1)
    q, k = (torch.randn((3, 1, sh.n, 64), generator=gen, device=DEV).bfloat16() for _ in range(2))
    frame = torch.arange(sh.n, device=DEV) // (128 * 128)
    doc = torch.stack([frame // 8, frame // 4, frame // 2]).int().contiguous()
    order = torch.stack([frame, -frame, frame % 2]).int().contiguous()
    mod = rf2.ScoreMod(document=doc, order=order)
    mask, ws = rf2.alloc_mask(g, keep, DEV)
    qp, kp = rf2.permute_qk_pool(g, q, k, ws)
    rf2.predict_mask_visible(g, keep, mask, ws, mod)
    assert rf2.device_status() == rf2.RF2_OK
    n = mask.sizes.n_keep
    assert (mask.row_count == n).all()
    cols = mask.col_idx.long()[mask.row_start.long()[:, None] + torch.arange(n, device=DEV)].view(sh.batch, sh.blocks, n)
    # a block is 64 tokens of one frame here: of one document and one order
    first = torch.from_numpy(rf2.permutation_index(g).astype("int64")).to(DEV)[::64]
    d, o = doc[:, first], order[:, first]
    mean = lambda x: x.double().view(sh.batch, sh.blocks, 64, 64).mean(2)
    qm, km = mean(qp[:, 0]), mean(kp[:, 0])
    for b in range(sh.batch):
        may = (d[b][:, None] == d[b][None]) & (o[b][None] <= o[b][:, None])
        assert int(may.sum(1).min()) >= n
        assert may.gather(1, cols[b]).all()
        s = (qm[b] @ km[b].T).masked_fill(~may, -math.inf)
        # the kept ones are the n best, but for ties of the 2^-20 that the scores are good to
        worst = s.gather(1, cols[b]).amin(1)
        best_left = s.scatter(1, cols[b], -math.inf).amax(1)
        assert (worst >= best_left - 2.0 ** -18 * qm[b].norm(dim=1) * km[b].norm(dim=1).max()).all()


@pytest.mark.parametrize("heads,frames,interleaved", [(12, 8, False), (24, 8, True), (24, 13, False), (17, 21, True)])
def test_norm_rope_with_several_units_a_warp(heads, frames, interleaved):
    """Long calls give a CTA 16 or 24 (tensor, head) units for its 8 warps: forward and gradient of every
    head, and the weight gradients over all of them."""
    sh = Shape(1, heads, 64, frames, 61, 65, (4, 4, 4), True, 9)
    g, perm, ang = sh.geometry(), sh.perm(DEV), angles(sh, DEV)
    gen = torch.Generator(device=DEV).manual_seed(heads)
    q, k, v, dqp, dkp, dvp = (torch.randn((1, heads, sh.n, 64), generator=gen, device=DEV).bfloat16() for _ in range(6))
    ws = [1 + 0.4 * torch.randn(64, generator=gen, device=DEV) for _ in range(2)]
    rope = rf2.rope_table(g, sh.split(), device=DEV)
    kw = dict(q_weight=ws[0], k_weight=ws[1], rope=rope, interleaved=interleaved)
    qp, kp, vp = rf2.norm_rope_permute(g, q, k, v, **kw)
    dq, dk, dv, dwq, dwk = rf2.norm_rope_permute_backward(g, q, k, dqp, dkp, dvp, **kw)
    assert rf2.device_status() == rf2.RF2_OK
    assert torch.equal(vp, v[:, :, perm])
    back = torch.empty_like(dvp)
    back[:, :, perm] = dvp
    assert torch.equal(dv, back)
    for x, w, y, dy, dx, dw in ((q, ws[0], qp, dqp, dq, dwq), (k, ws[1], kp, dkp, dk, dwk)):
        wr, mag = w.double().requires_grad_(), 0.0
        for h in range(heads):
            xr = x[:, h:h + 1].double().requires_grad_()
            ref = norm_rope(sh, xr, wr, ang, 1e-6, interleaved)[:, :, perm]
            tol = HALF * ref.abs() + 2.0 ** -19 * ref.abs().amax(-1, keepdim=True)
            assert ((y[:, h:h + 1].double() - ref).abs() <= tol).all()
            ref.backward(dy[:, h:h + 1].double())
            with torch.no_grad():
                r = 1 / torch.sqrt((xr ** 2).mean(-1, keepdim=True) + 1e-6)
                size = torch.empty_like(r)
                size[:, :, perm] = dy[:, h:h + 1].double().abs().amax(-1, keepdim=True) * w.double().abs().amax() * 2
                assert ((dx[:, h:h + 1].double() - xr.grad).abs() <= HALF * xr.grad.abs() + 2.0 ** -17 * r * size * 4).all()
                zb = torch.zeros_like(xr)
                zb[:, :, perm] = dy[:, h:h + 1].double()
                mag = mag + (norm_rope(sh, zb, None, -ang, 1e-6, interleaved, False) * xr * r).abs().sum((0, 1, 2))
        # an fp32 sum in stages (a lane's rows, the warp's units, the CTAs): at most 2^13 terms in a row
        assert ((dw.double() - wr.grad).abs() <= 2.0 ** -11 * mag).all()
