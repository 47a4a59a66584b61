"""What the checkpointed grouped MLP asks of the buffers it is given, on the host
(no GPU needed): the sizes of the saved tensors and of the workspaces,
and their alignment."""
import ctypes
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


def _edges(E, I):
    """Counts of rows around those where the rule for few rows changes."""
    near = [64 * E, 256 * E, (1 << 21) // I]
    return sorted({max(0, n + d) for n in near for d in (-40, -1, 0, 1, 4, 44, 300)} | {0, 1, 100000})


@pytest.mark.parametrize("precision", ALL, ids=IDS)
@pytest.mark.parametrize("e,h,i", [(8, 4096, 14336), (64, 2048, 1408), (8, 2048, 1408), (1, 128, 128),
                                   (16, 65536, 128), (2, 65664, 128), (3, 128, 65664)])
def test_workspace_of_a_batch_serves_smaller_ones(precision, e, h, i):
    for op in (moe.MOE_OP_MLP_FWD, moe.MOE_OP_MLP_BWD):
        rows = _edges(e, i)
        need = [moe.moe_workspace_bytes(op, n, h, i, e, 1, precision) for n in rows]
        assert all(need) and need == sorted(need), (op, [r for r, a, b in zip(rows, need, need[1:]) if a > b])


@pytest.mark.parametrize("bwd", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("precision", ALL, ids=IDS)
@pytest.mark.parametrize("what", ["workspace", "a2", "a2_col_codes", "a2_col_scales", "xp_col_codes",
                                  "xp_col_scales"])
def test_misaligned_buffers(bwd, precision, what):
    """4104 is 8 bytes past a 16-byte address; no address here is read."""
    p = ctypes.c_void_p(4096)
    ws = ctypes.c_void_p(4104 if what == "workspace" else 4096)
    saved = moe._Saved(None, *[4104 if n == what else 4096 for n, _ in moe._Saved._fields_[1:6]])
    tab = (ctypes.c_void_p * 2)(4096, 4096)
    f, n = moe.lib(), 1 << 40
    if bwd:
        st = f.grouped_mlp_bwd_ckpt(precision, 2, 128, 256, 8, p, None, p, p, tab, tab, p, ctypes.byref(saved),
                                    p, p, p, tab, tab, p, ws, n, None)
    else:
        st = f.grouped_mlp_fwd_ckpt(precision, 2, 128, 256, 8, p, None, p, tab, tab, p, p, ctypes.byref(saved),
                                    p, p, ws, n, None)
    assert st == 3
