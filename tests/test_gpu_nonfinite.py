"""Non-finite values in tokens that are not padding: they stay in the rows they
belong to, and the calls come back."""
import pytest
import torch

from image_dits_b200 import rf2
from layer_ref import Shape, csr_of, random_kept

pytestmark = pytest.mark.gpu
DEV = "cuda"

# 5 and 6 blocks, the last one ragged
SHAPES = [Shape(1, 2, 64, 5, 8, 7, (1, 8, 8)), Shape(1, 2, 128, 6, 7, 8, (4, 4, 4))]
# (cap, bias, document mask); None: the unmodified calls
VARIANTS = [None, (0.0, False, False), (20.0, False, False), (0.0, True, False), (20.0, True, False), (0.0, False, True),
            (20.0, True, True)]


def _mod(sh, variant):
    if variant is None:
        return None
    cap, bias, masked = variant
    # the last three tokens are padding, the others one document
    doc = torch.where(torch.arange(sh.n, device=DEV) < sh.n - 3, 4, -1).int()[None].repeat(sh.batch, 1) if masked else None
    return rf2.ScoreMod(softcap=cap, slopes=torch.full((sh.heads,), 0.2, device=DEV) if bias else None, document=doc)


def _qkv(sh, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn((sh.batch, sh.heads, sh.n, sh.dim), generator=g, device=DEV).bfloat16() for _ in range(3)]


def _run(sh, q, k, v, mask, mod):
    lse = torch.empty((sh.batch, sh.heads, sh.n), device=DEV)
    g = sh.geometry()
    o = (rf2.block_sparse_attn(g, q, k, v, mask, lse=lse) if mod is None else
         rf2.block_sparse_attn_mod(g, q, k, v, mask, mod, lse=lse))
    assert rf2.device_status() == rf2.RF2_OK
    return o, lse


@pytest.mark.parametrize("value", ["nan", "inf", "all -inf"])
@pytest.mark.parametrize("variant", VARIANTS, ids=str)
@pytest.mark.parametrize("sh", SHAPES, ids=str)
def test_forward_of_one_query_row(sh, variant, value):
    """One row of Q holds a NaN, or an infinity that leaves its first block no finite score: every
    other row is what it is without, and the row itself is NaN (unless the cap makes an infinite
    product finite)."""
    q, k, v = _qkv(sh)
    mask, mod = csr_of(sh, random_kept(sh, 1.0, 1, DEV)), _mod(sh, variant)
    k[..., 5] = k[..., 5].abs() + 0.1                     # no zero: an infinity times it is no NaN
    row = 70
    bad = q.clone()
    if value == "nan":
        bad[0, 1, row, 5] = float("nan")
    else:
        bad[0, 1, row, 5] = float("-inf" if value == "all -inf" else "inf")
        if value == "inf":
            k[..., :64, 5] *= -1                          # -inf in the first block, +inf behind it
    want, want_lse = _run(sh, q, k, v, mask, mod)
    got, got_lse = _run(sh, bad, k, v, mask, mod)
    others = torch.ones(q.shape[:3], dtype=torch.bool, device=DEV)
    others[0, 1, row] = False
    masked, capped = bool(variant and variant[2]), bool(variant and variant[0])
    if masked or (capped and value != "nan"):
        # Under a mask such a row may send its warp's rows to their maxima; under the cap an infinite
        # product moves its warp from one form of tanh to another, each good to 2^-21, so scores of at
        # most 20 move by 2 * 20 * 2^-21 < 2e-5 and so does the log-sum-exp (less than 10: rounded to
        # 2^-21 in either run).  The same probabilities to 2e-5, rounded against another maximum (P is
        # off by 2^-8 of itself each time, O once more).
        tol = (2 * 2.0 ** -8 + 2e-5) * v.float().abs().max() + 2.0 ** -8 * want.float().abs()
        assert ((got.float() - want.float()).abs() <= tol)[others].all()
        if not masked:
            assert ((got_lse - want_lse).abs() <= 2e-5 + 2.0 ** -20)[others].all()
    else:
        assert torch.equal(got[others], want[others]) and torch.equal(got_lse[others], want_lse[others])
    if value == "nan" or (value == "inf" and not capped):
        assert torch.isnan(got[0, 1, row]).all()


# three pairs of blocks, each keeping itself and nothing else
PAIRS = [Shape(1, 2, 64, 6, 8, 8, (1, 8, 8)), Shape(1, 1, 128, 6, 8, 8, (1, 8, 8))]


def _pair_mask(sh):
    kept = torch.zeros((sh.batch * sh.heads, 6, 6), dtype=torch.bool, device=DEV)
    for p in range(0, 6, 2):
        kept[:, p:p + 2, p:p + 2] = True
    return csr_of(sh, kept)


@pytest.mark.parametrize("sh", PAIRS, ids=str)
def test_gradient_keeps_a_query_rows_nan(sh):
    """A NaN in one row of Q makes its probabilities NaN: all of dV in its pair of blocks, whichever
    column of the product the row comes to stand in; nothing elsewhere."""
    q, k, v = _qkv(sh)
    g, mask = sh.geometry(), _pair_mask(sh)
    do = torch.randn_like(q)
    clean = rf2.block_sparse_attn_backward(g, q, k, v, *_run(sh, q, k, v, mask, None), do, mask)
    for row in range(128, 144):
        bad = q.clone()
        bad[:, :, row, 3] = float("nan")
        got = rf2.block_sparse_attn_backward(g, bad, k, v, *_run(sh, bad, k, v, mask, None), do, mask)
        assert rf2.device_status() == rf2.RF2_OK
        assert torch.isnan(got[2][:, :, 128:256]).all(), row
        for a, b in zip(got, clean):
            assert torch.equal(a[:, :, :128], b[:, :, :128]) and torch.equal(a[:, :, 256:], b[:, :, 256:])


def _pair_reference(sh, q, k, v, do, softcap):
    """(O, lse, dQ, dK, dV) in fp64, pair by pair, from the formulas."""
    outs = []
    for p in range(3):
        a, b, c, d = (x[:, :, 128 * p:128 * p + 128].double() for x in (q, k, v, do))
        s = a @ b.transpose(-1, -2) * sh.dim ** -0.5
        t = torch.tanh(s / softcap) if softcap else None
        s = softcap * t if softcap else s
        m = s.amax(-1, keepdim=True)
        e = torch.exp(s - m)
        l = e.sum(-1, keepdim=True)
        w = e / l
        o = w @ c
        ds = w * (d @ c.transpose(-1, -2) - (d * o).sum(-1, keepdim=True)) * (1 - t * t if softcap else 1.0)
        ds = ds * sh.dim ** -0.5
        outs.append((o, (m + torch.log(l))[..., 0], ds @ b, ds.transpose(-1, -2) @ a, w.transpose(-1, -2) @ d))
    return [torch.cat(x, 2) for x in zip(*outs)]


@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("where", ["q", "k", "v", "do"])
@pytest.mark.parametrize("sh", PAIRS, ids=str)
def test_nan_reaches_what_it_has_to(sh, where, softcap):
    """One NaN in a token that sees and is seen: wherever the formulas give NaN the calls do, the
    log-sum-exp included, and the other pairs of blocks keep their bits."""
    mask = _pair_mask(sh)
    mod = rf2.ScoreMod(softcap=softcap) if softcap else None
    names = ("q", "k", "v", "do")
    clean = dict(zip(names, (*_qkv(sh), torch.randn((sh.batch, sh.heads, sh.n, sh.dim), device=DEV).bfloat16())))
    bad = dict(clean)
    bad[where] = clean[where].clone()
    bad[where][:, :, 150, 9] = float("nan")
    outs = []
    for x in (clean, bad):
        o, lse = _run(sh, x["q"], x["k"], x["v"], mask, mod)
        outs.append((o, lse, *rf2.block_sparse_attn_backward(sh.geometry(), x["q"], x["k"], x["v"], o, lse, x["do"], mask, mod)))
        assert rf2.device_status() == rf2.RF2_OK
    for name, want, a, b in zip(("o", "lse", "dq", "dk", "dv"), _pair_reference(sh, *(bad[n] for n in names), softcap), *outs):
        assert torch.isfinite(a.float()).all()
        assert torch.isnan(b[torch.isnan(want)]).all(), name
        assert torch.equal(a[:, :, :128], b[:, :, :128]) and torch.equal(a[:, :, 256:], b[:, :, 256:]), name
