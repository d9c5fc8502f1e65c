"""The gradient under a cap whose scores are saturated: 1 - tanh^2 keeps its relative accuracy."""
import math

import pytest
import torch

from image_dits_b200 import rf2
from layer_ref import HALF, Shape, attention, backward_tolerance, csr_of

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("lo,hi", [(2.0, 4.0), (6.0, 8.0), (8.0, 10.0), (10.0, 14.0)])
@pytest.mark.parametrize("shape", [(1, 8, 8), (1, 9, 15)], ids=str)
@pytest.mark.parametrize("dim", [64, 128])
def test_backward(dim, shape, lo, hi):
    """Raw scores lo to hi times the cap, of both signs: the whole gradient by Q and K goes through
    slopes of 4 e^(-2 lo) to 4 e^(-2 hi)."""
    sh = Shape(1, 2, dim, *shape, (1, 8, 8))
    cap, n = 2.0, sh.n
    g = torch.Generator(device=DEV).manual_seed(int(10 * hi) + dim)
    rand = lambda *s: torch.rand(s, generator=g, device=DEV, dtype=torch.float64)
    axis = torch.where(rand(dim) < 0.5, -1.0, 1.0).double()
    # q = a axis, k = +-b axis with a b sqrt(d) between lo and hi caps, and some noise across
    a = math.sqrt(lo * cap) + rand(1, 2, n, 1) * (math.sqrt(hi * cap) - math.sqrt(lo * cap))
    b = math.sqrt(lo * cap) + rand(1, 2, n, 1) * (math.sqrt(hi * cap) - math.sqrt(lo * cap))
    sign = torch.where(rand(1, 2, n, 1) < 0.3, -1.0, 1.0)
    f = dim ** -0.25
    q, k = (f * (a * axis) + 0.01 * (rand(1, 2, n, dim) - 0.5)).bfloat16(), (f * (sign * b * axis) + 0.01 * (rand(1, 2, n, dim) - 0.5)).bfloat16()
    v, do = (rand(1, 2, n, dim) * 2 - 1).bfloat16(), (rand(1, 2, n, dim) * 2 - 1).bfloat16()
    kept = torch.ones((2, sh.blocks, sh.blocks), dtype=torch.bool, device=DEV)
    mask, mod = csr_of(sh, kept), rf2.ScoreMod(softcap=cap)
    lse = torch.empty((1, 2, n), device=DEV)
    o = rf2.block_sparse_attn_mod(sh.geometry(), q, k, v, mask, mod, lse=lse)
    got = rf2.block_sparse_attn_backward(sh.geometry(), q, k, v, o, lse, do, mask, mod)
    assert rf2.device_status() == rf2.RF2_OK

    qd, kd, vd, dd = (x.double() for x in (q, k, v, do))
    vis = torch.ones((1, 2, n, n), dtype=torch.bool, device=DEV)
    ref, _, p = attention(sh, qd, kd, vd, vis, torch.arange(n, device=DEV), softcap=cap)
    raw = qd @ kd.transpose(-1, -2) / math.sqrt(dim)
    assert 0.9 * lo <= float(raw.abs().min()) / cap and float(raw.abs().max()) / cap <= 1.1 * hi
    slope = 1 / torch.cosh(raw / cap) ** 2
    ds = p * (dd @ vd.transpose(-1, -2) - (dd * ref).sum(-1, keepdim=True)) * slope / math.sqrt(dim)
    want = (ds @ kd, ds.transpose(-1, -2) @ qd, p.transpose(-1, -2) @ dd)
    # slope: 2 |x| times the score's relative error (products exact, summed in fp32: d 2^-24 at most, as all
    # terms have one sign) below 2 * 14 * 128 * 2^-24 < 3e-4, its own arithmetic below 1e-5: inside the
    # tolerance's 2 P_REL.  No absolute part: the gradients are as small as 1e-12.
    tols = backward_tolerance(sh, qd, kd, vd, ref, dd, p, slope)
    for name, x, y, tol in zip("qkv", got, want, tols):
        err = (x.double() - y).abs()
        assert (err <= tol + HALF * y.abs()).all(), (name, float((err / (tol + HALF * y.abs())).max()))
