"""The copies that fwd / bwd write record their scale layout, and the products refuse compact scales, which for whole
tiles have the same size as the tiled ones.  No GPU needed: the helpers' checks run on CPU buffers."""
import pytest
import torch

from nvfp4_quantization_grouped_gb300 import gsa

COMPACT, TILED = gsa.SCALES_COMPACT, gsa.SCALES_TILED
CPU = torch.device("cpu")


def operand(q, side, recipe):
    gsa._torch or gsa._setup()
    return gsa._operand(q, side, recipe, 2, "operand", CPU)


@pytest.mark.parametrize("recipe", [gsa.MXFP8, gsa.NVFP4])
@pytest.mark.parametrize("bound", [False, True])
@pytest.mark.parametrize("side", ["row", "col"])
def test_compact_scales_are_refused(recipe, bound, side):
    def alloc(*layout):
        if bound:
            return gsa.alloc_qtensor_bound(2, 512, 512, recipe, True, True, "cpu", *layout)
        return gsa.alloc_qtensor([256, 256], 512, recipe, True, True, "cpu", None, *layout)

    tiled = alloc(TILED)
    operand(tiled, side, recipe)
    for q in (alloc(COMPACT), alloc()):
        if not bound:
            assert q["row_scale"].numel() == tiled["row_scale"].numel()   # what the byte counts cannot tell
        with pytest.raises(gsa.GsaError, match="compact"):
            operand(q, side, recipe)
    own = alloc(COMPACT)
    own[side + "_scale"] = own[side + "_scale"].clone()   # a buffer of the caller's own is taken as tiled
    operand(own, side, recipe)


def test_the_last_writer_counts():
    """Buffers allocated for one layout and written in the other, and copies taken out of their dict."""
    q = gsa.alloc_qtensor([128], 512, gsa.MXFP8, True, True, "cpu", scale_layout=TILED)
    gsa._record_layout(q, COMPACT, ("col_scale",))
    operand(q, "row", gsa.MXFP8)
    with pytest.raises(gsa.GsaError, match="compact"):
        operand({k: q[k] for k in ("col_data", "col_scale")}, "col", gsa.MXFP8)
    gsa._record_layout(q, TILED)
    operand(q, "col", gsa.MXFP8)
