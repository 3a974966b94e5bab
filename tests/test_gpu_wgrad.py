"""Weight gradient from an 8-bit checkpoint on the GPU, against float64."""
import numpy as np
import pytest

import act_reference as R

pytestmark = pytest.mark.gpu
DT = {"f32": "float32", "bf16": "bfloat16", "f16": "float16"}


def _inputs(m, o, c, dtype, seed):
    import torch
    from layer_wise_top_amd import lags
    rng = np.random.default_rng(seed)
    x = np.maximum(rng.standard_normal((m, c)), -0.3) * np.exp(rng.standard_normal(c))
    dy = torch.from_numpy(rng.standard_normal((m, o)) * np.exp(2 * rng.standard_normal((m, 1)))).to(
        getattr(torch, DT[dtype])).cuda()
    xd = torch.from_numpy(x).float().cuda()
    ck = lags.checkpoint(m, c)
    lags.lags_ckpt_pack(xd, ck)
    val = torch.empty_like(xd)
    lags.lags_ckpt_unpack(ck, val)
    return dy, ck, val.double().cpu().numpy()


def _run(dy, ck, o, c, dw=None, add=False):
    import torch
    from layer_wise_top_amd import lags
    ws = lags.wgrad_workspace(dy.shape[0], o, c, dy.dtype)
    ws.fill_(0xFF)
    dw = torch.full((o, c), 7.0, device="cuda") if dw is None else dw
    print("wgrad", tuple(dy.shape), c, dy.dtype, dy.stride(), flush=True)
    lags.lags_ckpt_wgrad(dy, ck, dw, ws, add=add)
    torch.cuda.synchronize()
    return dw


def _check(tag, dw, dy, val):
    """Products are exact; a sum of m terms in the kernel's order has at most m / 16 additions of
    matrix steps (16 products each, up to 16 roundings inside one) and the joins of slices."""
    d = dy.double().cpu().numpy()
    want, mag = d.T @ val, np.abs(d).T @ np.abs(val)
    bound = (d.shape[0] / 16 + 64) * R.U * mag
    R.check(tag, dw.double().cpu().numpy(), want, bound)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("m,o,c", [(1, 1, 1), (1, 64, 64), (3, 5, 17), (31, 64, 64), (32, 65, 63), (33, 128, 128),
                                   (64, 1, 300), (100, 300, 1), (257, 129, 200), (1000, 70, 33), (513, 256, 256),
                                   (2048, 64, 32), (5000, 256, 64), (700, 1000, 500), (300, 513, 777),
                                   (900, 190, 250), (130, 383, 700), (64, 6000, 31), (2000, 63, 1000)])
def test_shapes(m, o, c, dtype):
    dy, ck, val = _inputs(m, o, c, dtype, m + o + c)
    _check(f"{m}x{o}x{c} {dtype}", _run(dy, ck, o, c), dy, val)


@pytest.mark.parametrize("m,o,c", [(96, 2600, 2500), (4096, 2048, 2304)])
def test_large_tiles(m, o, c):
    """Enough output for the widest tiles, with ragged edges: compared on the GPU in float64."""
    import torch
    dy, ck, val = _inputs(m, o, c, "bf16", m)
    dw = _run(dy, ck, o, c)
    d, v = dy.double(), torch.from_numpy(val).cuda()
    want, mag = d.t().contiguous() @ v, d.abs().t().contiguous() @ v.abs()
    assert ((dw.double() - want).abs() <= (m / 16 + 64) * R.U * mag).all()


@pytest.mark.parametrize("dtype", list(DT))
def test_slice_add_and_flat_gradient(dtype):
    """dY as a slice at an odd offset; dW into a layer's slice of a flat gradient at an odd offset,
    whose neighbours stay; added to."""
    import torch
    m, o, c = 300, 70, 45
    dy, ck, val = _inputs(m, o, c, dtype, 4)
    wide = torch.full((m, 201), 3.0, dtype=dy.dtype, device="cuda")
    wide[:, 13:83] = dy
    base = _run(dy, ck, o, c)
    flat = torch.full((o * c + 10,), 2.0, device="cuda")
    _run(wide[:, 13:83], ck, o, c, flat[3:3 + o * c].view(o, c))
    assert torch.equal(flat[3:3 + o * c].view(o, c), base)
    assert (flat[:3] == 2).all() and (flat[3 + o * c:] == 2).all()
    _run(wide[:, 13:83], ck, o, c, flat[3:3 + o * c].view(o, c), add=True)
    assert torch.equal(flat[3:3 + o * c].view(o, c), base + base)
    assert (flat[:3] == 2).all() and (flat[3 + o * c:] == 2).all()


def test_no_rows():
    import torch
    from layer_wise_top_amd import lags
    dy = torch.empty(0, 20, device="cuda")
    ck = lags.checkpoint(0, 30)
    dw = _run(dy, ck, 20, 30)
    assert not dw.any()
    dw.fill_(3)
    _run(dy, ck, 20, 30, dw, add=True)
    assert (dw == 3).all()


@pytest.mark.parametrize("dtype", list(DT))
def test_non_finite(dtype):
    """An infinity or NaN in dY reaches its output's row alone; a marked run of X its 32 columns."""
    import torch
    from layer_wise_top_amd import lags
    m, o, c = 70, 66, 96
    dy, ck, val = _inputs(m, o, c, dtype, 8)
    x = torch.from_numpy(val).float().cuda()
    x = torch.where(x == 0, torch.ones_like(x), x)
    x[5, 40] = float("inf")
    ck = lags.checkpoint(m, c)
    lags.lags_ckpt_pack(x, ck)
    dy[7, 3], dy[9, 60], dy[11, 64] = float("inf"), float("nan"), float("-inf")
    dw = _run(dy, ck, o, c).cpu().numpy()
    assert np.isnan(dw[:, 32:64]).all()
    rest = np.concatenate([dw[:, :32], dw[:, 64:]], axis=1)
    assert np.isnan(rest[60]).all()
    xs = np.concatenate([x.cpu().numpy()[:, :32], x.cpu().numpy()[:, 64:]], axis=1)
    held = R.held(xs.astype(np.float64))
    for row, src, sign in ((3, 7, 1.0), (64, 11, -1.0)):
        with np.errstate(invalid="ignore"):
            want = sign * np.inf * held[src]                  # NaN where the held value is zero
        assert np.array_equal(rest[row], want, equal_nan=True)
    keep = [i for i in range(o) if i not in (3, 60, 64)]
    assert np.isfinite(rest[keep]).all()


@pytest.mark.parametrize("dtype", list(DT))
def test_odd_rows_past_the_slice(dtype):
    """Rows of odd length start inside a word; what follows the matrix there, and the first value of
    the next slice of the rows, stay out of the sums, infinities and NaN too."""
    import torch
    m, o, c = 5000, 67, 64
    dy, ck, val = _inputs(m, o, c, dtype, 12)
    base = _run(dy, ck, o, c)
    big = torch.full((m * o + 70,), float("nan"), dtype=dy.dtype, device="cuda")
    for off in (0, 1, 3):
        big[off:off + m * o] = dy.reshape(-1)
        view = torch.as_strided(big, (m, o), (o, 1), off)
        assert torch.equal(_run(view, ck, o, c), base), off
        big.fill_(float("nan"))
    dy[::64, 0] = float("inf")
    with np.errstate(invalid="ignore"):
        want = (np.inf * val[::64]).sum(axis=0)
    got = _run(dy, ck, o, c).cpu().numpy()
    assert np.array_equal(np.isnan(got[0]), np.isnan(want)) and np.isfinite(got[1:]).all()
    one = np.sign(val[::64])
    same = (one == one[0]).all(axis=0) & (one[0] != 0)        # infinities of one sign: no NaN
    assert np.array_equal(got[0][same], np.inf * one[0][same])


def test_fp32_keeps_its_digits():
    """One row: each product of a 24-bit dY and a 7-bit X, correctly rounded to within two roundings."""
    import torch
    from layer_wise_top_amd import lags
    rng = np.random.default_rng(0)
    dy = torch.from_numpy(rng.standard_normal((1, 64)).astype(np.float32)).cuda()
    x = torch.from_numpy(rng.integers(-127, 128, (1, 64)).astype(np.float32)).cuda()
    x[0, 0] = 127
    x[0, 32] = 127
    ck = lags.checkpoint(1, 64)
    lags.lags_ckpt_pack(x, ck)
    dw = _run(dy, ck, 64, 64).double()
    want = dy.double().t() @ x.double()
    assert ((dw - want).abs() <= 2 * R.U * want.abs()).all()


def test_large_magnitudes_fp32():
    """The leading term of the largest fp32 values does not overflow."""
    import torch
    from layer_wise_top_amd import lags
    dy = torch.full((1, 64), 3.4028234e38, device="cuda")
    x = torch.ones(1, 64, device="cuda")
    ck = lags.checkpoint(1, 64)
    lags.lags_ckpt_pack(x, ck)
    dw = _run(dy, ck, 64, 64)
    assert torch.isfinite(dw).all() and ((dw.double() - 3.4028234e38).abs() <= 1e31 * 10).all()


def test_repeats_bit_for_bit_and_in_graphs():
    import torch
    from layer_wise_top_amd import lags
    m, o, c = 6000, 128, 96
    dy, ck, _ = _inputs(m, o, c, "bf16", 1)
    ws = lags.wgrad_workspace(m, o, c, dy.dtype)
    dw = torch.empty(o, c, device="cuda")
    base = _run(dy, ck, o, c)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lags.lags_ckpt_wgrad(dy, ck, dw, ws)
    for i in range(4):
        dw.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dw, base), i
        dw.zero_()
        lags.lags_ckpt_wgrad(dy, ck, dw, ws, stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert torch.equal(dw, base), i
