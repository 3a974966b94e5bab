"""Every kernel of the weight gradient that a size selects, on the GPU, against float64."""
import pytest

import act_reference as R
from test_act_plans import TILES, WGRAD_SHAPES, wgrad_plan

pytestmark = pytest.mark.gpu
DT = {"f32": "float32", "bf16": "bfloat16", "f16": "float16"}
CASES = [(dtype, tile, i) for dtype in WGRAD_SHAPES for tile in WGRAD_SHAPES[dtype] for i in (0, 1)]


@pytest.mark.parametrize("dtype,tile,sliced", CASES)
def test_tile(dtype, tile, sliced):
    """dY contiguous, in rows of even pitch (16-bit rows start on words) and of odd pitch at an odd
    offset (they start inside them), NaN around it: the same bits, near the float64 product; added to
    a gradient of ones, one more rounding.  A sum of m terms has m / 16 additions of matrix steps at
    most (16 products each, up to 16 roundings inside one) and the joins of slices."""
    import torch
    from layer_wise_top_amd import lags
    m, o, c = WGRAD_SHAPES[dtype][tile][sliced]
    p = wgrad_plan(m, o, c, dtype)
    assert TILES[p.tile] == tile and (p.split > 1) == bool(sliced)
    print("tile", tile, dtype, (m, o, c), "slices", p.split, flush=True)
    g = torch.Generator(device="cuda").manual_seed(m + o + c)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    x = torch.relu(normal(m, c) * torch.exp(normal(c)))
    dy = (normal(m, o) * torch.exp(2 * normal(m, 1))).to(getattr(torch, DT[dtype]))
    ck, val = lags.checkpoint(m, c), torch.empty_like(x)
    lags.lags_ckpt_pack(x, ck)
    lags.lags_ckpt_unpack(ck, val)
    ws = lags.wgrad_workspace(m, o, c, dy.dtype)
    ws.fill_(0xFF)

    def run(t, dw=None):
        out = torch.full((o, c), 7.0, device="cuda") if dw is None else dw
        lags.lags_ckpt_wgrad(t, ck, out, ws, add=dw is not None)
        return out

    got = run(dy)
    d, v = dy.double().t().contiguous(), val.double()
    want, bound = d @ v, (m / 16 + 64) * R.U * (d.abs() @ v.abs())
    off = (got.double() - want).abs()
    assert (off <= bound).all(), (float((off - bound).max()), int((off > bound).sum()))
    even, odd = o + o % 2 + 6, o + 1 - o % 2 + 6
    for pitch, at in ((even, 2), (even, 1), (odd, 0), (odd, 3)):
        wide = torch.full((m, pitch), float("nan"), dtype=dy.dtype, device="cuda")
        wide[:, at:at + o] = dy
        assert torch.equal(run(wide[:, at:at + o]), got), (pitch, at)
    assert torch.equal(run(dy, torch.ones(o, c, device="cuda")), 1 + got)
