"""What the checkpointed grouped MLP asks of the buffers it is given, on the host
(no GPU needed): the sizes of the saved tensors."""
import os

import pytest
import torch

import mxfp8_block_scaled_top_amd as moe

ALL, IDS = [moe.MOE_BF16, moe.MOE_MXFP8, moe.MOE_FP8], ["bf16", "mxfp8", "fp8"]
ROWS, H, I, E = 48, 256, 384, 3
CPU = torch.device("cpu")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not os.path.exists(moe.LIB_PATH):
        from mxfp8_block_scaled_top_amd import build
        build.build()
    moe.lib()


def _check(saved, precision):
    moe._saved_members(saved, precision, ROWS, H, I, E, CPU)


@pytest.mark.parametrize("precision", ALL, ids=IDS)
def test_saved_of_these_sizes_or_larger(precision):
    _check(moe.alloc_saved(ROWS, H, I, E, precision, "cpu", checkpoint=True), precision)
    _check(moe.alloc_saved(ROWS, H, I, E, precision, "cpu", weight_cols=False, checkpoint=True), precision)
    _check(moe.alloc_saved(2 * ROWS, 2 * H, I, 2 * E, precision, "cpu", checkpoint=True), precision)


@pytest.mark.parametrize("precision", ALL[1:], ids=IDS[1:])
@pytest.mark.parametrize("h,e", [(H - 128, E), (H, 1)], ids=["narrower", "fewer_experts"])
def test_saved_of_smaller_sizes(precision, h, e):
    """The same rows and I: A1's own tensors have the right shapes."""
    saved = moe.alloc_saved(ROWS, h, I, e, precision, "cpu", checkpoint=True)
    assert saved["a1_codes"].shape == (ROWS, 2 * I)
    with pytest.raises(moe.MoEError, match="bytes"):
        _check(saved, precision)


@pytest.mark.parametrize("precision", ALL, ids=IDS)
def test_every_member_is_checked(precision):
    """One member too small, another device's, of a strided view or no tensor."""
    saved = moe.alloc_saved(ROWS, H, I, E, precision, "cpu", checkpoint=True)
    for name in saved:
        if name.startswith("a1_"):
            continue
        t = saved[name]
        for bad in (t.flatten()[:-1].clone(), t.to("meta"), torch.cat([t, t], -1)[..., ::2], t.numpy
                    if t.dtype == torch.uint8 else t.float()):
            with pytest.raises(moe.MoEError):
                _check(saved | {name: bad}, precision)
        if name != "a2":          # exactly what is needed passes
            need = dict(moe._saved_needs(precision, ROWS, H, I, E))[name]
            _check(saved | {name: t[:need].clone()}, precision)
