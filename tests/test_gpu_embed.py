"""Embedding lookup and the table's gradient on the GPU, against float64."""
import numpy as np
import pytest

import act_reference as R

pytestmark = pytest.mark.gpu
DT = {"f32": "float32", "bf16": "bfloat16", "f16": "float16"}


def _dt(dtype):
    import torch
    return getattr(torch, DT[dtype])


def _dev(a, dtype):
    import torch
    return torch.from_numpy(np.asarray(a, np.float64)).to(_dt(dtype)).cuda()


def _ids(a, wide):
    import torch
    return torch.from_numpy(np.asarray(a, np.int64)).to(torch.int64 if wide else torch.int32).cuda()


def _draw(rng, tokens, vocab, kind):
    if kind == "one":
        return np.full(tokens, rng.integers(vocab))
    if kind == "few":
        return rng.choice(rng.integers(0, vocab, 3), tokens)
    if kind == "text":                  # frequencies fall as 1 / rank
        return np.minimum(np.exp(rng.random(tokens) * np.log(vocab + 1)).astype(np.int64) - 1, vocab - 1)
    if kind == "each":
        return rng.permutation(np.arange(tokens) % vocab)
    a = rng.integers(0, vocab, tokens)  # "holes": padding and ids out of range, on both sides
    bad = rng.random(tokens) < 0.4
    a[bad] = rng.choice([-1, -100, vocab, vocab + 7, 2 ** 31 - 1, -2 ** 31], bad.sum())
    return a


def _grad(ids, dy, vocab, scale=1.0, dtable=None, add=False):
    import torch
    from layer_wise_top_amd import lags
    c = dy.shape[-1]
    ws = lags.embed_workspace(ids.numel(), vocab, c).fill_(0xFF)
    dtable = torch.full((vocab, c), 7.0, device="cuda") if dtable is None else dtable
    print("embed grad", tuple(dy.shape), vocab, dy.dtype, ids.dtype, dy.stride(), flush=True)
    lags.lags_embed_grad(ids, dy, dtable, ws, scale=scale, add=add)
    torch.cuda.synchronize()
    return dtable


def _check_grad(tag, got, ids, dy, vocab, scale):
    """A row's sum: its tokens one after the other up to 256 in all; else at most 16 additions in a
    chunk (of 8 tokens or more), then chains of a quarter of its chunks and three more; the scale is
    one product."""
    d, a = dy.double().cpu().numpy(), np.asarray(ids)
    ok = (a >= 0) & (a < vocab)
    want, mag, n = (np.zeros((vocab, d.shape[1])) for _ in range(3))
    np.add.at(want, a[ok], d[ok])
    np.add.at(mag, a[ok], np.abs(d[ok]))
    np.add.at(n, a[ok], 1)
    s32 = float(np.float32(scale))
    chain = n + 2 if d.shape[0] <= 256 else 16 + n / 32 + 8
    bound = chain * R.U * mag * abs(s32)
    R.check(tag, got.double().cpu().numpy(), want * s32, bound)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("tokens,vocab,cols", [(1, 1, 1), (1, 1000, 8), (5, 3, 7), (64, 10, 33), (700, 10000, 150),
                                               (100, 600, 1500), (33, 50, 2048), (5000, 77, 64), (4100, 300, 1031),
                                               (70, 9, 4099)])
def test_forward(tokens, vocab, cols, dtype):
    import torch
    from layer_wise_top_amd import lags
    rng = np.random.default_rng(tokens + cols)
    for table in {"f32", dtype}:
        for wide in (False, True):
            w = _dev(rng.standard_normal((vocab, cols)), table)
            a = _draw(rng, tokens, vocab, "holes")
            scale = float(rng.choice([1.0, 0.7, 45.25]))
            y = torch.full((tokens, cols), 7, dtype=_dt(dtype), device="cuda")
            print("embed", tokens, vocab, cols, dtype, table, wide, flush=True)
            lags.lags_embed_forward(_ids(a, wide), w, y, scale=scale)
            ok = torch.from_numpy((a >= 0) & (a < vocab)).cuda()
            rows = w[torch.from_numpy(np.where((a >= 0) & (a < vocab), a, 0)).cuda()].float() * scale
            assert torch.equal(y, torch.where(ok[:, None], rows, torch.zeros_like(rows)).to(y.dtype))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("kind", ["one", "few", "text", "each", "holes"])
@pytest.mark.parametrize("tokens,vocab,cols", [(1, 1, 1), (31, 5, 8), (32, 40, 33), (33, 1, 17), (64, 3, 64), (65, 1000, 7),
                                               (700, 10000, 150), (1000, 50, 515), (2500, 513, 2051), (17000, 300, 40)])
def test_gradient(tokens, vocab, cols, kind, dtype):
    rng = np.random.default_rng(tokens + cols + vocab)
    a = _draw(rng, tokens, vocab, kind)
    dy = rng.standard_normal((tokens, cols)) * np.exp(rng.standard_normal((tokens, 1)))
    dy = _dev(dy, dtype)
    scale = float(rng.choice([1.0, 0.3, 39.0]))
    got = _grad(_ids(a, tokens % 2 == 0), dy, vocab, scale)
    _check_grad(f"{tokens} {vocab} {cols} {kind} {dtype}", got, a, dy, vocab, scale)


@pytest.mark.parametrize("kind", ["one", "text", "holes"])
@pytest.mark.parametrize("tokens", [63, 64, 128, 192, 193, 255, 256, 257])
def test_where_one_launch_ends(tokens, kind):
    """Up to 256 tokens and above, written and added at an odd place, all columns of a vector used and not."""
    import torch
    rng = np.random.default_rng(tokens)
    for dtype, vocab, cols in (("bf16", 41, 520), ("f32", 300, 261)):
        a = _draw(rng, tokens, vocab, kind)
        dy = _dev(rng.standard_normal((tokens, cols)), dtype)
        flat = torch.full((vocab * cols + 7,), 0.5, device="cuda")
        at = flat[3:3 + vocab * cols].view(vocab, cols)
        _check_grad(f"{tokens} {kind} {dtype}", _grad(_ids(a, True), dy, vocab, 1.5, at), a, dy, vocab, 1.5)
        once = at.clone()
        _grad(_ids(a, False), dy, vocab, 1.5, at, add=True)
        assert torch.equal(at, 2 * once)
        assert (flat[:3] == 0.5).all() and (flat[3 + vocab * cols:] == 0.5).all()


@pytest.mark.parametrize("tokens", [40, 400])
def test_ids_whose_low_half_is_in_the_table(tokens):
    """64-bit ids outside the table, in each 32-bit half."""
    import torch
    from layer_wise_top_amd import lags
    rng = np.random.default_rng(1)
    vocab, cols = 30, 24
    a = rng.integers(0, vocab, tokens)
    far = a.copy()
    far[::3] = np.resize([2 ** 32 + 3, -2 ** 32 + 3, 2 ** 63 - 1, -2 ** 63, 2 ** 32, 2 ** 40 + 7], len(far[::3]))
    a[::3] = -1
    dy, w = _dev(rng.standard_normal((tokens, cols)), "bf16"), _dev(rng.standard_normal((vocab, cols)), "f32")
    y = torch.full((tokens, cols), 7, dtype=dy.dtype, device="cuda")
    want = torch.full_like(y, 7)
    lags.lags_embed_forward(_ids(far, True), w, y)
    lags.lags_embed_forward(_ids(a, True), w, want)
    assert torch.equal(y, want) and (y[::3] == 0).all()
    assert torch.equal(_grad(_ids(far, True), dy, vocab), _grad(_ids(a, True), dy, vocab))


@pytest.mark.parametrize("vocab", [511, 512, 131072, 131073, 300000])
def test_large_vocabularies(vocab):
    """From one id a workgroup of the sort to its 512 at most, and a last group of any size."""
    rng = np.random.default_rng(vocab)
    a = np.concatenate([_draw(rng, 3000, vocab, "each"), rng.integers(0, vocab, 1500), [0, vocab - 1, vocab - 1]])
    dy = _dev(rng.standard_normal((len(a), 24)), "bf16")
    _check_grad(str(vocab), _grad(_ids(a, True), dy, vocab), a, dy, vocab, 1.0)


def test_many_tokens():
    """Sections of the sort longer than a wave holds in registers."""
    rng = np.random.default_rng(2)
    for kind in ("text", "one"):
        a = _draw(rng, 70001, 3000, kind)
        dy = _dev(rng.standard_normal((len(a), 16)), "f32")
        _check_grad(kind, _grad(_ids(a, False), dy, 3000, 2.0), a, dy, 3000, 2.0)


@pytest.mark.parametrize("dtype", list(DT))
def test_slices_and_flat_gradient(dtype):
    """dy as a slice at an odd offset, y into one; the gradient into a layer's slice of a flat buffer at an
    odd offset, whose neighbours stay; added to, where rows without tokens stay as they are."""
    import torch
    from layer_wise_top_amd import lags
    rng = np.random.default_rng(3)
    t, v, c = 300, 70, 45
    a = _draw(rng, t, v, "text")
    a[::9] = -1
    dy = _dev(rng.standard_normal((t, c)), dtype)
    dy[::9] = float("nan")                                 # padding's gradient is not looked at
    ids = _ids(a, True)
    base = _grad(ids, dy, v, 0.5)
    assert torch.isfinite(base).all()
    wide = torch.full((t, 101), float("nan"), dtype=dy.dtype, device="cuda")
    wide[:, 13:13 + c] = dy
    flat = torch.full((v * c + 10,), 2.0, device="cuda")
    view = flat[3:3 + v * c].view(v, c)
    _grad(ids, wide[:, 13:13 + c], v, 0.5, view)
    assert torch.equal(view, base) and (flat[:3] == 2).all() and (flat[3 + v * c:] == 2).all()
    view.fill_(1)
    _grad(ids, wide[:, 13:13 + c], v, 0.5, view, add=True)
    assert torch.equal(view, 1 + base) and (flat[:3] == 2).all() and (flat[3 + v * c:] == 2).all()
    w = _dev(rng.standard_normal(v * c + 3), "f32")
    y = torch.empty(t, c, dtype=dy.dtype, device="cuda")
    table = w[3:].view(v, c)
    lags.lags_embed_forward(ids, table, y)
    wide.fill_(9)
    lags.lags_embed_forward(ids.view(30, 10), table, wide[:, 13:13 + c])
    assert torch.equal(wide[:, 13:13 + c], y) and (wide[:, :13] == 9).all() and (wide[:, 13 + c:] == 9).all()


def test_no_tokens():
    import torch
    from layer_wise_top_amd import lags
    ids, dy = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, 20, device="cuda")
    lags.lags_embed_forward(ids, torch.ones(5, 20, device="cuda"), dy)
    got = _grad(ids, dy, 5)
    assert not got.any()
    got.fill_(3)
    _grad(ids, dy, 5, dtable=got, add=True)
    assert (got == 3).all()
    # tokens, but none with an id
    ids = torch.full((40,), -1, device="cuda")
    assert not _grad(ids, torch.ones(40, 20, device="cuda"), 5).any()


def test_gradient_is_the_lookups_transpose():
    """<lookup(W), dy> = <W, gradient(dy)> for any W: the derivative, and by differences since it is linear."""
    import torch
    from layer_wise_top_amd import lags
    rng = np.random.default_rng(4)
    t, v, c = 500, 60, 32
    a = _draw(rng, t, v, "holes")
    ids, w, dy = _ids(a, True), _dev(rng.standard_normal((v, c)), "f32"), _dev(rng.standard_normal((t, c)), "f32")
    y = torch.empty(t, c, device="cuda")
    lags.lags_embed_forward(ids, w, y, scale=3.0)
    g = _grad(ids, dy, v, 3.0)
    left, right = (y.double() * dy.double()).sum(), (w.double() * g.double()).sum()
    assert abs(left - right) <= 1e-5 * (y.double() * dy.double()).abs().sum()


def test_infinities_stay_in_their_row_and_channel():
    import torch
    rng = np.random.default_rng(5)
    a = _draw(rng, 400, 30, "text")
    dy = _dev(rng.standard_normal((400, 20)), "bf16")
    base = _grad(_ids(a, True), dy, 30)
    dy[7, 3], dy[11, 4] = float("inf"), float("nan")
    got = _grad(_ids(a, True), dy, 30)
    assert torch.isinf(got[a[7], 3]) and torch.isnan(got[a[11], 4])
    got[a[7], 3], got[a[11], 4] = base[a[7], 3], base[a[11], 4]
    assert torch.equal(got, base)


def test_repeats_graphs_and_streams():
    import torch
    from layer_wise_top_amd import lags
    rng = np.random.default_rng(6)
    t, v, c = 5000, 700, 130
    ids, dy = _ids(_draw(rng, t, v, "text"), True), _dev(rng.standard_normal((t, c)), "bf16")
    w = _dev(rng.standard_normal((v, c)), "f32")
    base = _grad(ids, dy, v)
    y0 = torch.empty(t, c, dtype=dy.dtype, device="cuda")
    lags.lags_embed_forward(ids, w, y0)
    ws, out, y = lags.embed_workspace(t, v, c), torch.empty(v, c, device="cuda"), torch.empty_like(y0)

    def step(stream=None):
        lags.lags_embed_forward(ids, w, y, stream=stream)
        lags.lags_embed_grad(ids, dy, out, ws, stream=stream)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()

    def check(i):
        torch.cuda.synchronize()
        assert torch.equal(out, base) and torch.equal(y, y0), i
        out.fill_(5)
        y.fill_(5)
        ws.fill_(0xFF)
        torch.cuda.synchronize()

    for i in range(4):
        g.replay()
        check(i)
        step()
        check(i)
    step(torch.cuda.Stream())
    check("side")
    # the captured call reads ids and dy anew
    ids.copy_(_ids(_draw(rng, t, v, "each"), True))
    want = _grad(ids, dy, v)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_past_2_31_elements():
    """A table and a gradient of more than 2^31 entries, ids at both ends."""
    import torch
    from layer_wise_top_amd import lags
    v, c = (1 << 20) + 3, 2056
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    w = torch.zeros(v, c, device="cuda")
    ids = torch.tensor([0, v - 1, v - 2, 5, v - 1, -1], device="cuda")
    for i in (0, 5, v - 1, v - 2):
        w[i] = torch.arange(c, device="cuda") + i % 1000
    y = torch.empty(6, c, device="cuda")
    lags.lags_embed_forward(ids, w, y)
    assert torch.equal(y[:5], w[ids[:5]]) and not y[5].any()
    w.fill_(7)
    got = _grad(ids, y, v, dtable=w)
    assert torch.equal(got[v - 1], y[1] + y[4]) and torch.equal(got[v - 2], y[2]) and torch.equal(got[0], y[0])
    assert not got[6:v - 2].any() and not got[1:5].any()


@pytest.mark.parametrize("tokens", [0, 100, 300])
def test_largest_vocabulary(tokens):
    """2^26 ids, in one launch and in three; small whole numbers, so that sums are exact."""
    import torch
    if torch.cuda.mem_get_info()[0] < 10 << 30:
        pytest.skip("needs 10 GB")
    v, c = 1 << 26, 5
    g = torch.Generator(device="cuda").manual_seed(tokens)
    ids = torch.randint(0, v, (tokens,), generator=g, device="cuda")
    if tokens:
        ids[:6] = torch.tensor([0, v - 1, v - 2, v - 1, v, -1])
    dy = torch.randint(-9, 10, (tokens, c), generator=g, device="cuda").float()
    real = (ids >= 0) & (ids < v)
    want = torch.zeros(v, c, device="cuda").index_add_(0, ids[real], dy[real])
    assert torch.equal(_grad(ids, dy, v), want)
    assert torch.equal(_grad(ids, dy, v, scale=2.0, dtable=want.clone(), add=True), 3 * want)


def test_chunks_of_several_joins():
    """More chunks of 16 tokens than one launch of the join has workgroups.  Sums of small whole numbers are
    exact, below 2^24."""
    import torch
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    v, n, c = 1000, (1 << 28) + (1 << 20) + 5, 2
    ids = torch.arange(n, dtype=torch.int32, device="cuda") % v
    g = torch.Generator(device="cuda").manual_seed(1)
    dy = torch.randint(0, 16, (n, c), generator=g, device="cuda", dtype=torch.int8).float()
    got = _grad(ids, dy, v)
    whole = n // v * v
    want = torch.zeros(v, c, dtype=torch.float64, device="cuda")
    for i in range(0, whole, v << 14):
        want += dy[i:min(whole, i + (v << 14))].view(-1, v, c).sum(0, dtype=torch.float64)
    want[:n - whole] += dy[whole:].double()
    assert torch.equal(got.double(), want)
