"""8-bit activation checkpoints on the GPU: the buffer bit for bit, and the
values it holds."""
import numpy as np
import pytest

import act_reference as R

pytestmark = pytest.mark.gpu
DT = {"f32": "float32", "bf16": "bfloat16", "f16": "float16"}


def _x(rows, cols, dtype, seed):
    import torch
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal(cols))
    return torch.from_numpy(x).to(getattr(torch, DT[dtype])).cuda()


def _pack(x, fill=0xAB):
    import torch
    from layer_wise_top_amd import lags
    rows = x.numel() // x.shape[-1]
    ck = lags.checkpoint(rows, x.shape[-1])
    ck.fill_(fill)
    lags.lags_ckpt_pack(x, ck)
    torch.cuda.synchronize()
    return ck


def _check(x, tag):
    import torch
    from layer_wise_top_amd import lags
    print("case", tag, tuple(x.shape), x.dtype, x.stride(), flush=True)
    x64 = x.double().cpu().numpy().reshape(-1, x.shape[-1])
    want, n = R.codes(x64)
    ck = _pack(x)
    got = ck.cpu().numpy()[:n]
    diff = np.flatnonzero(got != want[:n])
    assert diff.size == 0, f"{tag}: {diff.size} bytes differ, first at {diff[0]} of {n}"
    vals = R.held(x64)
    for dt in DT.values():
        out = torch.full_like(x, 7.0, dtype=getattr(torch, dt), memory_format=torch.contiguous_format)
        lags.lags_ckpt_unpack(ck, out)
        ref = torch.from_numpy(vals).to(getattr(torch, dt)).reshape(out.shape)
        o = out.cpu()
        assert torch.equal(torch.isnan(o), torch.isnan(ref)), (tag, dt)
        assert torch.equal(torch.nan_to_num(o), torch.nan_to_num(ref)), (tag, dt)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 15), (1, 16), (4, 17), (2, 31), (7, 32), (3, 33),
                                       (64, 64), (129, 100), (33, 250), (2, 2049), (1025, 8)])
def test_shapes(rows, cols, dtype):
    _check(_x(rows, cols, dtype, rows * 1000 + cols), f"{rows}x{cols}")


@pytest.mark.parametrize("dtype", list(DT))
def test_every_exponent(dtype):
    """Runs whose largest magnitude is every power of two of the type, on both sides of the value
    that rounds past 127, ties included; zeros and negative zeros."""
    import torch
    dt = getattr(torch, DT[dtype])
    lo, hi = (-24, 15) if dtype == "f16" else (-133, 127)
    rows = []
    for e in range(lo, hi + 1):
        for m in (1.0, 1.5, 127 / 64, 1.98828125, 1.9921875, 1.99609375):
            top = np.ldexp(m, e)
            r = np.linspace(-1, 1, 32) * top
            r[5], r[6], r[7] = top, 0.0, -0.0
            r[8:16] = top / 256 * np.arange(1, 9)             # halves of the step
            rows.append(r)
    x = torch.from_numpy(np.array(rows)).to(dt)
    x = x[torch.isfinite(x).all(dim=1)]
    _check(torch.cat([x, torch.zeros(2, 32, dtype=dt)]).cuda(), f"exponents {dtype}")


@pytest.mark.parametrize("dtype", list(DT))
def test_non_finite_runs(dtype):
    x = _x(6, 70, dtype, 5)
    x[0, 0], x[1, 33], x[2, 69], x[3, 40] = float("inf"), float("-inf"), float("nan"), float("nan")
    _check(x, "non-finite")


@pytest.mark.parametrize("dtype", list(DT))
def test_slices_and_leading_dimensions(dtype):
    """A slice of the channels (any offset), rows of odd pitch, and the values written into a slice
    leave everything around them as it was."""
    import torch
    from layer_wise_top_amd import lags
    whole = _x(50, 77, dtype, 9)
    _check(whole[:, 3:44], "slice")
    _check(_x(30, 40, dtype, 4).view(5, 6, 40), "3-D")
    ck = _pack(whole[:, 3:44])
    out = torch.full((50, 77), 5.0, dtype=whole.dtype, device="cuda")
    lags.lags_ckpt_unpack(ck, out[:, 21:62])
    ref = torch.from_numpy(R.held(whole[:, 3:44].double().cpu().numpy())).to(whole.dtype)
    assert torch.equal(out[:, 21:62].cpu(), ref)
    assert (out[:, :21] == 5).all() and (out[:, 62:] == 5).all()


def test_buffer_end_is_untouched():
    import torch
    from layer_wise_top_amd import lags
    x = _x(9, 50, "bf16", 1)
    n = lags.lags_ckpt_bytes(9, 50)
    assert n == -(-9 * (64 + 2) // 16) * 16
    big = torch.full((n + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    lags.lags_ckpt_pack(x, big)
    assert (big[n:] == 0x5A).all()


def test_rows_past_32_bits():
    """A matrix of more than 2^32 bytes: its last rows."""
    import torch
    from layer_wise_top_amd import lags
    rows, cols = (1 << 20) + 5, 4096
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-3:] = _x(3, cols, "bf16", 2)
    ck = lags.checkpoint(rows, cols)
    lags.lags_ckpt_pack(x, ck)
    out = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    lags.lags_ckpt_unpack(ck, out)
    ref = torch.from_numpy(R.held(x[-3:].double().cpu().numpy())).to(torch.bfloat16)
    assert torch.equal(out[-3:].cpu(), ref)
    assert not out[:-3].any()


def test_no_rows():
    import torch
    from layer_wise_top_amd import lags
    x = torch.empty(0, 40, device="cuda")
    ck = lags.checkpoint(0, 40)
    lags.lags_ckpt_pack(x, ck)
    lags.lags_ckpt_unpack(ck, x)


def test_other_stream_and_graph():
    """Packed on one stream, unpacked on another after an event; and captured in a graph, every
    replay against the eager result."""
    import torch
    from layer_wise_top_amd import lags
    x = _x(300, 200, "f32", 3)
    want = torch.from_numpy(R.held(x.double().cpu().numpy())).float()
    ck, out = lags.checkpoint(300, 200), torch.zeros_like(x)
    torch.cuda.synchronize()
    s1, s2, ev = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.Event()
    lags.lags_ckpt_pack(x, ck, stream=s1)
    ev.record(s1)
    s2.wait_event(ev)
    lags.lags_ckpt_unpack(ck, out, stream=s2)
    s2.synchronize()
    assert torch.equal(out.cpu(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lags.lags_ckpt_pack(x, ck)
        lags.lags_ckpt_unpack(ck, out)
    for i in range(3):
        x.copy_(_x(300, 200, "f32", 10 + i))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), torch.from_numpy(R.held(x.double().cpu().numpy())).float()), i
