"""What the binding of the layer operators refuses before any launch, without a GPU."""
import ctypes

import pytest
import torch

from image_dits_b200 import build as rf2_build
from image_dits_b200 import rf2


@pytest.fixture(scope="module", autouse=True)
def built():
    rf2_build.build()


def geo(**kw):
    a = dict(batch=2, heads=3, head_dim=128, frames=3, height=7, width=9, win_t=2, win_h=4, win_w=4, sink=True, text=11)
    a.update(kw)
    return rf2.make_geometry(**a)


@pytest.mark.parametrize("made,used", [(0.2, 0.5), (0.2, 1.0), (0.5, 0.9)])
def test_visible_prediction_refuses_a_mask_made_for_a_lower_keep(made, used):
    # host tensors: the refusal comes before anything is looked up on a device
    g = geo(frames=6, height=16, width=16)
    mask, ws = rf2.alloc_mask(g, made, "cpu")
    mod = rf2.ScoreMod(document=torch.zeros((2, rf2.num_tokens(g)), dtype=torch.int32))
    with pytest.raises(ValueError, match="col_idx"):
        rf2.predict_mask_visible(g, used, mask, ws, mod)
    # one made for as much or more gets past it, to the refusal of host tensors
    for keep in (made, made / 2):
        with pytest.raises(ValueError, match="CUDA"):
            rf2.predict_mask_visible(g, keep, mask, ws, mod)


def _bf16(g, n):
    return [torch.zeros((g.batch, g.heads, rf2.num_tokens(g), g.head_dim), dtype=torch.bfloat16) for _ in range(n)]


@pytest.mark.parametrize("n", [0, 1, 2, 4])
def test_outputs_come_in_threes(n):
    """Another number of outputs would shift the pointers behind them."""
    g = geo()
    x = _bf16(g, 5)
    out = tuple(_bf16(g, n))
    mask = rf2.BlockMask(*(torch.zeros(24, dtype=torch.int32) for _ in range(3)), rf2.query(g, 1.0))
    lse = torch.zeros(2, 3, 200)
    for call in (lambda: rf2.norm_rope_permute(g, *x[:3], out=out),
                 lambda: rf2.norm_rope_permute(g, *x[:2], out=out),
                 lambda: rf2.norm_rope_permute_backward(g, *x, out=out),
                 lambda: rf2.norm_rope_permute_backward(g, *x[:4], out=out),
                 lambda: rf2.block_sparse_attn_backward(g, *x[:4], lse, x[4], mask, out=out)):
        with pytest.raises(ValueError, match="three"):
            call()


def test_visible_prediction_refuses_one_workspace_for_both():
    g, a = geo(), 1 << 20
    m = rf2.ScoreModStruct(0.0, 1.0, 1.0, 1.0, None, None, None)
    need = rf2.query(g, 0.5).mask_workspace_bytes

    def call(w, mw):
        # one byte short, so that a call that gets past the pointers stops at the workspace's size
        return rf2.lib().rf2_predict_mask_visible(ctypes.byref(g), 0.5, ctypes.byref(m), 20 * a, 21 * a, 22 * a, w, need - 1, mw,
                                                  1 << 30, None)
    assert call(23 * a, 23 * a) == rf2.RF2_ERR_INVALID_ARGUMENT
    assert call(23 * a, 24 * a) == rf2.RF2_ERR_INSUFFICIENT_WORKSPACE
