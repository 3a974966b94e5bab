"""Linear layers on the GPU, forward and backward, against float64."""
import numpy as np
import pytest

import act_reference as R
from test_linear_plans import CASES

pytestmark = pytest.mark.gpu
DT = {"f32": "float32", "bf16": "bfloat16", "f16": "float16"}
ACTS = ["none", "relu", "silu", "gelu"]
GELU = 2 * np.sqrt(2 / np.pi)
# rows, cols, outs: one of each, single rows, ragged in every direction, slices of k, every tile
SHAPES = [(1, 1, 1), (1, 2048, 100), (3, 5, 17), (2, 64, 64), (31, 64, 10), (32, 65, 63), (33, 128, 128), (64, 200, 300),
          (65, 257, 1), (100, 31, 70), (257, 129, 200), (7, 4000, 515), (30, 1500, 3001), (128, 512, 512),
          (700, 150, 600), (300, 1031, 77), (513, 256, 260), (1000, 36, 1300), (2100, 72, 2050), (515, 2048, 520),
          (20, 640, 16384)]
LARGE = [(4200, 130, 4100), (3000, 515, 4700), (8200, 264, 1032)]


def _dt(dtype):
    import torch
    return getattr(torch, DT[dtype])


def _np(t):
    return t.double().cpu().numpy()


def _dev(a, dtype):
    import torch
    return torch.from_numpy(np.asarray(a, np.float64)).to(_dt(dtype)).cuda()


def _sig(u):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-u))


def _act(z, kind):
    """act(z), act'(z) in float64, and bounds of the errors of both beside that of z itself: the
    sigmoid's argument is good to a few roundings of its size, as is what is made of it."""
    if kind == "none":
        return z, np.ones_like(z), np.zeros_like(z), np.zeros_like(z)
    if kind == "relu":
        return np.maximum(z, 0), (z > 0).astype(float), np.zeros_like(z), np.zeros_like(z)
    if kind == "silu":
        u, du = z, np.ones_like(z)
    else:
        u, du = GELU * (z + 0.044715 * z ** 3), GELU * (1 + 0.134145 * z ** 2)
    s, r = _sig(u), _sig(-u)
    t = np.minimum(np.abs(u), 90)
    return (z * s, s + z * s * r * du, (16 + 8 * t) * R.U * np.abs(z * s) + 1e-30,
            (16 + 8 * t) * R.U * (s + np.abs(z) * s * r * du) + 1e-30)


def _ws(lin):
    from layer_wise_top_amd import lags
    return lags.linear_workspace(lin).fill_(0xFF)


def _forward(x, w, act="none", bias=None, res=None, keep=False, y=None):
    import torch
    from layer_wise_top_amd import lags
    m, k, n = x.shape[0], x.shape[1], w.shape[0]
    lin = lags.Linear(m, k, n, dtype=x.dtype, act=act)
    y = torch.full((m, n), 7, dtype=x.dtype, device="cuda") if y is None else y
    z = torch.full((m, n), 7, dtype=x.dtype, device="cuda") if keep else None
    print("linear", (m, k, n), x.dtype, x.stride(), w.stride(), act, flush=True)
    lags.lags_linear_forward(lin, x, w, y, _ws(lin), bias=bias, res=res, z=z)
    torch.cuda.synchronize()
    return y, z


def _backward(dy, w, act="none", z=None, bias=True, dx=True, add=None):
    import torch
    from layer_wise_top_amd import lags
    m, n, k = dy.shape[0], dy.shape[1], w.shape[1]
    lin = lags.Linear(m, k, n, dtype=dy.dtype, act=act)
    dz = torch.full((m, n), 7, dtype=dy.dtype, device="cuda") if act != "none" else None
    db = (torch.full((n,), 7.0, device="cuda") if add is None else add) if bias else None
    dxt = torch.full((m, k), 7, dtype=dy.dtype, device="cuda") if dx else None
    print("linear backward", (m, k, n), dy.dtype, dy.stride(), w.stride(), act, flush=True)
    lags.lags_linear_backward(lin, dy, w if dx else None, dxt, _ws(lin), z=z, dz=dz, dbias=db, add=add is not None)
    torch.cuda.synchronize()
    return dz, db, dxt


def _sum_bound(k, dtype):
    """A sum of k products in fp32 in any order has k additions of partial sums no larger than the
    sum of magnitudes; fp32 products round once more.  16-bit products are exact, 16 of them an
    instruction with up to 16 roundings, so the same count."""
    return (k + 8) * R.U


def _check_forward(tag, x, w, act, bias, res, y, z, dtype):
    a, b = _np(x), _np(w)
    want, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    if bias is not None:
        want, mag = want + _np(bias), mag + np.abs(_np(bias))
    ez = _sum_bound(a.shape[1], dtype) * mag
    if z is not None:
        R.check(tag + " z", _np(z), want, ez, dtype)
    v, _, ev, _ = _act(want, act)
    ev = ev + 1.2 * ez                         # the activations' slopes stay below 1.2
    if res is not None:
        v = v + _np(res)
        ev = ev + R.U * (np.abs(v) + np.abs(_np(res)))
    R.check(tag + " y", _np(y), v, ev, dtype)


def _check_backward(tag, dy, w, act, z, dz, db, dx, dtype):
    d, b = _np(dy), _np(w)
    if act != "none":
        _, slope, _, es = _act(_np(z), act)
        want = d * slope
        edz = np.abs(d) * es + R.U * np.abs(want)
        R.check(tag + " dz", _np(dz), want, edz, dtype)
    else:
        want, edz = d, np.zeros_like(d)
    if db is not None:
        # a lane's rows, four waves, then a sixteenth of the chunks, and those: below 256
        R.check(tag + " dbias", _np(db), want.sum(0), (edz + 256 * R.U * np.abs(want)).sum(0))
    if dx is not None:
        held = _np(dz) if act != "none" else d
        R.check(tag + " dx", _np(dx), held @ b, _sum_bound(d.shape[1], dtype) * (np.abs(held) @ np.abs(b)), dtype)


def _inputs(m, k, n, dtype, seed):
    import torch
    rng = np.random.default_rng(seed)
    x = _dev(rng.standard_normal((m, k)) * np.exp(0.5 * rng.standard_normal(k)), dtype)
    w = _dev(rng.standard_normal((n, k)) / np.sqrt(k), dtype)
    bias = torch.from_numpy(0.3 * rng.standard_normal(n)).float().cuda()
    res, dy = _dev(rng.standard_normal((m, n)), dtype), _dev(0.1 * rng.standard_normal((m, n)), dtype)
    return x, w, bias, res, dy


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("m,k,n", SHAPES + LARGE)
def test_shapes(m, k, n, dtype):
    x, w, bias, res, dy = _inputs(m, k, n, dtype, m + k + n)
    i = m + k + n
    act = ACTS[i % 4]
    bias, res = bias if i % 3 else None, res if i % 5 < 2 else None
    y, z = _forward(x, w, act, bias, res, keep=True)
    tag = f"{m}x{k}x{n} {dtype} {act}"
    _check_forward(tag, x, w, act, bias, res, y, z, dtype)
    if act != "none":
        dz, db, dx = _backward(dy, w, act, z, bias is not None)
        _check_backward(tag, dy, w, act, z, dz, db, dx, dtype)
    dz, db, dx = _backward(dy, w, "none")
    _check_backward(tag + " none", dy, w, "none", None, dz, db, dx, dtype)


@pytest.mark.parametrize("dtype,key,shape", CASES)
def test_every_tile(dtype, key, shape):
    """Ragged tiles of every kind, whole and in slices, W as it is and turned round; compared on the GPU in
    float64.  A slice at an odd offset gives the same bits."""
    import torch
    (m, k, n), back = shape, key[0]
    g = torch.Generator(device="cuda").manual_seed(m + k + n)
    inner, outer = (n, k) if back else (k, n)
    a = torch.randn(m, inner, generator=g, device="cuda").to(_dt(dtype))
    w = (torch.randn(n, k, generator=g, device="cuda") / inner ** 0.5).to(_dt(dtype))

    def run(a, w):
        return _backward(a, w, bias=False)[2] if back else _forward(a, w)[0]

    got = run(a, w)
    b = w.double() if back else w.double().t().contiguous()
    want, mag = a.double() @ b, a.double().abs() @ b.abs()
    lim = _sum_bound(inner, dtype) * mag * (1 + R.ROUND[dtype]) + R.ROUND[dtype] * want.abs() + R.TINY[dtype]
    assert ((got.double() - want).abs() <= lim).all()
    assert torch.equal(run(a, w), got)
    for off in (1, 2):
        wide = torch.full((m, inner + 5), float("nan"), dtype=a.dtype, device="cuda")
        wide[:, off:off + inner] = a
        wv = torch.full((n, k + 5), float("nan"), dtype=a.dtype, device="cuda")
        wv[:, off:off + k] = w
        assert torch.equal(run(wide[:, off:off + inner], w), got) and torch.equal(run(a, wv[:, off:off + k]), got)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("has_res", [False, True])
def test_epilogues(act, has_res, dtype):
    """Every activation with and without bias and residual, whole and in slices of k; with and without z."""
    import torch
    for m, k, n in ((90, 64, 75), (40, 5000, 72)):
        x, w, bias, res, dy = _inputs(m, k, n, dtype, 3)
        r = res if has_res else None
        for b in (None, bias):
            y, z = _forward(x, w, act, b, r, keep=True)
            _check_forward(f"{act} {dtype}", x, w, act, b, r, y, z, dtype)
            assert torch.equal(_forward(x, w, act, b, r)[0], y)
            dz, db, dx = _backward(dy, w, act, z if act != "none" else None)
            _check_backward(f"{act} {dtype}", dy, w, act, z, dz, db, dx, dtype)
            only, none, _ = _backward(dy, w, act, z if act != "none" else None, bias=False, dx=False)
            assert none is None and (only is None or torch.equal(only, dz))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("m,k,n", [(37, 70, 45), (300, 136, 264), (70, 64, 129), (25, 3000, 40), (1100, 200, 1064),
                                   (1825, 323, 1288)])
def test_slices_and_pitches(m, k, n, dtype):
    """Operands and results as column slices of wider matrices at odd, even and whole-vector offsets: the
    contiguous call's bits, neighbours (NaN) untouched and unread."""
    import torch
    x, w, bias, res, dy = _inputs(m, k, n, dtype, k)
    y, z = _forward(x, w, "silu", bias, res, keep=True)
    dz, db, dx = _backward(dy, w, "silu", z)

    def wide(t, off, pad):
        a = torch.full((t.shape[0], t.shape[1] + off + pad), float("nan"), dtype=t.dtype, device="cuda")
        a[:, off:off + t.shape[1]] = t
        return a, a[:, off:off + t.shape[1]]

    from layer_wise_top_amd import lags
    lin = lags.Linear(m, k, n, dtype=x.dtype, act="silu")
    for off, pad in ((1, 2), (2, 6), (8, 16), (0, 3)):
        (_, xv), (_, wv), (_, rv), (wy, yv) = (wide(t, off, pad) for t in (x, w, res, y))
        zw, zv = wide(z, off, pad)
        yv.fill_(3), zv.fill_(3)
        lags.lags_linear_forward(lin, xv, wv, yv, _ws(lin), bias=bias, res=rv, z=zv)
        assert torch.equal(yv, y) and torch.equal(zv, z)
        for a, c in ((wy, n), (zw, n)):
            assert torch.isnan(a[:, :off]).all() and torch.isnan(a[:, off + c:]).all()
        lags.lags_linear_forward(lin, xv, wv, rv, _ws(lin), bias=bias, res=rv)          # y is res
        assert torch.equal(rv, y)
        (_, dyv), (dw, dxv), (gw, gv) = wide(dy, off, pad), wide(dx, off, pad), wide(dz, off, pad)
        dxv.fill_(3), gv.fill_(3)
        b2 = torch.empty_like(db)
        lags.lags_linear_backward(lin, dyv, wv, dxv, _ws(lin), z=zv, dz=gv, dbias=b2)
        assert torch.equal(dxv, dx) and torch.equal(gv, dz) and torch.equal(b2, db)
        for a, c in ((dw, k), (gw, n)):
            assert torch.isnan(a[:, :off]).all() and torch.isnan(a[:, off + c:]).all()
        lags.lags_linear_backward(lin, dyv, wv, dxv, _ws(lin), z=zv, dz=zv)              # dz over z
        assert torch.equal(zv, dz)
        lags.lags_linear_backward(lin, dyv, wv, dxv, _ws(lin), z=z, dz=dyv)              # dz over dy
        assert torch.equal(dyv, dz) and torch.equal(dxv, dx)


def test_flat_parameters():
    """W and bias as slices of a flat fp32 buffer at odd offsets; dbias written and added there."""
    import torch
    m, k, n = 50, 33, 47
    x, w, bias, _, dy = _inputs(m, k, n, "f32", 9)
    flat = torch.full((n * k + n + 9,), 2.0, device="cuda")
    wv, bv = flat[1:1 + n * k].view(n, k), flat[3 + n * k:3 + n * k + n]
    wv.copy_(w), bv.copy_(bias)
    y, _ = _forward(x, w, "relu", bias)
    assert torch.equal(_forward(x, wv, "relu", bv)[0], y)
    _, db, dx = _backward(dy, w)
    assert torch.equal(_backward(dy, wv)[2], dx)
    bv.fill_(1)
    _backward(dy, w, add=bv)
    assert torch.equal(bv, 1 + db) and (flat[1 + n * k:3 + n * k] == 2).all() and (flat[-6:] == 2).all()


def test_no_rows():
    import torch
    x, w = torch.empty(0, 20, device="cuda"), torch.ones(30, 20, device="cuda")
    y, _ = _forward(x, w)
    _, db, dx = _backward(y, w)
    assert not db.any() and dx.shape == (0, 20)
    db.fill_(3)
    _backward(y, w, add=db)
    assert (db == 3).all()


def test_gradients_against_differences():
    """fp32: dz, dbias and dx against central differences of the float64 definition."""
    m, k, n = 5, 7, 9
    x, w, bias, res, dy = _inputs(m, k, n, "f32", 11)
    a, b, c, d = _np(x), _np(w), _np(bias), _np(dy)
    for act in ("silu", "gelu"):
        _, z = _forward(x, w, act, bias, res, keep=True)
        _, db, dx = _backward(dy, w, act, z)

        def loss(a, c):
            return (_act(a @ b.T + c, act)[0] * d).sum()

        h = 1e-5
        for got, arr, f in ((_np(dx), a, lambda t: loss(t, c)), (_np(db), c, lambda t: loss(a, t))):
            num = np.empty_like(arr)
            for i in np.ndindex(arr.shape):
                e = np.zeros_like(arr)
                e[i] = h
                num[i] = (f(arr + e) - f(arr - e)) / (2 * h)
            # h^2 truncation, cancellation 1e-16 / h, and fp32's own 1e-6
            assert np.abs(got - num).max() <= 1e-5 * np.abs(num).max(), act


@pytest.mark.parametrize("dtype", list(DT))
def test_values_at_the_edges(dtype):
    """An infinity or NaN of x reaches its row alone, of W its column, of dy its row; the largest finite
    values and infinities of z give the activations' limits."""
    import torch
    m, k, n = 70, 96, 66
    x, w, bias, _, dy = _inputs(m, k, n, dtype, 8)
    w = torch.where(w == 0, torch.ones_like(w), w)
    base = _forward(x, w, "none", bias)[0]
    x2 = x.clone()
    x2[3, 5], x2[9, 95], x2[69, 0] = float("inf"), float("nan"), float("-inf")
    y = _forward(x2, w, "none", bias)[0]
    assert torch.equal(y[3].float(), torch.sign(w[:, 5].float()) * float("inf")) and torch.isnan(y[9]).all()
    assert torch.equal(y[69].float(), -torch.sign(w[:, 0].float()) * float("inf"))
    keep = [i for i in range(m) if i not in (3, 9, 69)]
    assert torch.equal(y[keep], base[keep])
    w2 = w.clone()
    w2[65, 95], w2[1, 0] = float("nan"), float("inf")
    y = _forward(x, w2, "none", bias)[0]
    assert torch.isnan(y[:, 65]).all() and torch.isinf(y[:, 1]).all()
    rest = [i for i in range(n) if i not in (1, 65)]
    assert torch.equal(y[:, rest], base[:, rest])
    _, _, dx0 = _backward(dy, w)
    dy2 = dy.clone()
    dy2[4, 60], dy2[5, 65] = float("inf"), float("nan")
    _, db, dx = _backward(dy2, w)
    assert torch.equal(dx[4].float(), torch.sign(w[60].float()) * float("inf")) and torch.isnan(dx[5]).all()
    assert torch.equal(dx[[0, 1, 69]], dx0[[0, 1, 69]]) and torch.isinf(db[60]) and torch.isnan(db[65])
    assert torch.isfinite(db[:60]).all()
    big = torch.finfo(_dt(dtype)).max
    z = torch.tensor([[float("inf"), big, 0.0, -big, float("-inf"), float("nan")]], dtype=_dt(dtype), device="cuda")
    one = torch.ones(1, 1, dtype=z.dtype, device="cuda")
    for act, low in (("relu", 0), ("silu", 0), ("gelu", 0)):
        ones, eye = torch.ones_like(z), torch.ones(6, 1, dtype=z.dtype, device="cuda")
        got, _, _ = _backward(ones, eye, act, z, bias=False, dx=False)
        assert got[0, 0] == 1 and got[0, 1] == 1 and got[0, 3].abs() <= 1e-30 and got[0, 4].abs() <= 1e-30, act
        assert torch.isnan(got[0, 5])
        y, _ = _forward(one, z.t().contiguous(), act)
        assert torch.isinf(y[0, 0]) and y[0, 1] == big and y[0, 3].abs() <= 1e-30 and y[0, 4].abs() <= 1e-30, act
        assert y[0, 2] == 0 and torch.isnan(y[0, 5])


def test_fp32_keeps_its_digits():
    """One term: the product of two 24-bit values, rounded once."""
    import torch
    rng = np.random.default_rng(0)
    x, w = (torch.from_numpy(rng.standard_normal((64, 1)).astype(np.float32)).cuda() for _ in range(2))
    y, _ = _forward(x, w)
    want = x.double() @ w.double().t()
    assert ((y.double() - want).abs() <= R.U * want.abs()).all()
    big = torch.full((1, 64), 3.4028234e38, device="cuda")
    y, _ = _forward(big[:, :1], torch.ones(70, 1, device="cuda"))
    assert (y == 3.4028234e38).all()


def test_repeats_graphs_and_streams():
    """The same bits every time, in a replayed graph and on another stream; sliced and whole."""
    import torch
    from layer_wise_top_amd import lags
    for m, k, n in ((200, 4096, 136), (2000, 256, 2048)):
        x, w, bias, res, dy = _inputs(m, k, n, "bf16", 2)
        lin = lags.Linear(m, k, n, dtype=x.dtype, act="gelu")
        ws = _ws(lin)
        y, z, dz, dx = (torch.empty(m, c, dtype=x.dtype, device="cuda") for c in (n, n, n, k))
        db = torch.empty(n, device="cuda")

        def step(stream=None):
            lags.lags_linear_forward(lin, x, w, y, ws, bias=bias, res=res, z=z, stream=stream)
            lags.lags_linear_backward(lin, dy, w, dx, ws, z=z, dz=dz, dbias=db, stream=stream)

        step()
        torch.cuda.synchronize()
        base = [t.clone() for t in (y, z, dz, dx, db)]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()

        def check(i):
            torch.cuda.synchronize()
            for got, want in zip((y, z, dz, dx, db), base):
                assert torch.equal(got, want), i
                got.fill_(5)
            ws.fill_(0xFF)
            torch.cuda.synchronize()

        for i in range(4):
            g.replay()
            check(i)
            step()
            check(i)
        step(torch.cuda.Stream())
        check("side")


def test_past_2_31_elements():
    """x, dy and dx of more than 2^31 elements."""
    import torch
    m, k, n = (1 << 21) + 7, 1032, 8
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    x = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x[:4096].normal_(generator=g)
    for i in range(4096, m, 4096):
        x[i:i + 4096] = x[:min(4096, m - i)]
    w = torch.randn(n, k, generator=g, device="cuda").bfloat16()
    y, _ = _forward(x, w)
    assert torch.equal(y[1 << 20:(1 << 20) + 4096], y[:4096]) and torch.equal(y[-7:], y[:7])
    _, db, dx = _backward(y, w)
    assert torch.equal(dx[1 << 20:(1 << 20) + 4096], dx[:4096]) and torch.equal(dx[-7:], dx[:7])
    # and of outs: y, z and dz beyond it
    w2 = torch.randn(1040, 8, generator=g, device="cuda").bfloat16()
    y2, z2 = _forward(y, w2, "relu", keep=True)
    assert torch.equal(y2[-7:], y2[:7]) and torch.equal(z2[1 << 20:(1 << 20) + 4096], z2[:4096])
    dz2, _, dx2 = _backward(y2, w2, "relu", z2)
    assert torch.equal(dz2[-7:], dz2[:7]) and torch.equal(dx2[-7:], dx2[:7])


@pytest.mark.parametrize("m,k,n", [(16448, 72, 262152), (5546, 9, 774729)])
def test_outputs_of_a_large_vocabulary(m, k, n):
    """More than 2^32 outputs, and a backward whose sums over them are split: columns at both ends and past
    2^31 entries, dx whole."""
    import torch
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    g = torch.Generator(device="cuda").manual_seed(m)
    x, w = (torch.randn(r, k, generator=g, device="cuda").bfloat16() for r in (m, n))
    bias = torch.randn(n, generator=g, device="cuda")
    y, _ = _forward(x, w, "none", bias)
    _, db, dx = _backward(y, w)
    for c in (slice(0, 130), slice(n // 2, n // 2 + 70), slice(n - 133, n)):
        _check_forward(f"{m}x{k}x{n} {c}", x, w[c], "none", bias[c], None, y[:, c], None, "bf16")
        d = _np(y[:, c])
        # rows of a lane, waves and chunks, as in _check_backward
        R.check("dbias", _np(db[c]), d.sum(0), 256 * R.U * np.abs(d).sum(0))
    want, mag = (torch.zeros(m, k, dtype=torch.float64, device="cuda") for _ in range(2))
    for i in range(0, n, 16384):
        d, v = y[:, i:i + 16384].double(), w[i:i + 16384].double()
        want += d @ v
        mag += d.abs() @ v.abs()
    R.check("dx", _np(dx), _np(want), _sum_bound(n, "bf16") * _np(mag), "bf16")


def test_rows_of_several_launches():
    """Tiles of more threads than a launch has: x, z, res and y go on where the first launch ends."""
    import torch
    m = (1 << 30) + 77
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    g = torch.Generator(device="cuda").manual_seed(3)
    x, res = (torch.empty(m, 1, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    w = torch.full((1, 1), -1.5, dtype=torch.bfloat16, device="cuda")
    y, z = _forward(x, w, "relu", res=res, keep=True)
    _, _, dx = _backward(res, w, bias=False)
    for i in range(0, m, 1 << 26):
        c = slice(i, i + (1 << 26))
        f = x[c].float() * -1.5                       # exact in fp32
        assert torch.equal(z[c], f.bfloat16()) and torch.equal(y[c], (f.clamp(min=0) + res[c].float()).bfloat16()), i
        assert torch.equal(dx[c], (res[c].float() * -1.5).bfloat16()), i
