"""Paths of the activation operators that depend on a shape's plan, on the GPU,
against float64."""
import pytest

from test_act_plans import GROUPS, ROWS, rows_case
from test_gpu_gn import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["none", "relu", "silu"])
@pytest.mark.parametrize("n,s,c,groups", [(1100, 1, 4096, 1), (300, 3, 4096, 2), (150, 4, 2500, 1), (140, 2, 3001, 1),
                                          (3, 2, 4224, 2), (140, 5, 4096, 1)])
def test_fp32_groups_wider_than_2048_channels(n, s, c, groups, act):
    """A column of lanes of its own for each four channels: short samples whole in 1024 lanes, several
    of them a workgroup; five positions, and all of them where samples are few, in chunks."""
    Case(n, s, c, groups, "f32", act, seed=c + s).check_all()


@pytest.mark.parametrize("dtype,act", [("f32", "relu"), ("f32", "silu"), ("bf16", "relu"), ("bf16", "silu"),
                                       ("bf16", "none"), ("f16", "relu"), ("f16", "silu"), ("f16", "none")])
@pytest.mark.parametrize("groups", list(GROUPS))
@pytest.mark.parametrize("rows", list(ROWS))
def test_many_rows_a_thread(rows, groups, dtype, act):
    """8 and 13 register rows, with vectors inside one group and cut by groups, both directions, from x
    and from its checkpoint; then the same through rows of odd pitch at odd offsets (16-bit rows that
    start inside a word) with NaN around them, bit for bit."""
    import torch
    from layer_wise_top_amd import lags
    k = Case(*rows_case(dtype, rows, groups), dtype, act, seed=rows)
    k.check_all()
    n, s, c = k.x.shape
    ck = lags.checkpoint(n * s, c)
    fwd = k.forward(ck)
    bwd = k.backward(fwd[1], fwd[2], x=k.x), k.backward(fwd[1], fwd[2], ckpt=ck)

    def sliced(t, at, width):
        w = torch.full((n, s, width), float("nan"), dtype=t.dtype, device="cuda")
        w[..., at:at + c] = t
        return w[..., at:at + c]

    width = c + 6 + (c + 1) % 2                       # odd
    k.x, k.dy = sliced(k.x, 1, width), sliced(k.dy, 3, width + 2)
    y, dx = sliced(torch.zeros_like(fwd[0]), 2, width), sliced(torch.zeros_like(fwd[0]), 5, width)
    ck2 = lags.checkpoint(n * s, c)
    for a, b in zip(k.forward(ck2, y=y), fwd):
        assert torch.equal(a, b)
    used = lags.lags_ckpt_bytes(n * s, c) // 16 * 16 - 16
    assert torch.equal(ck[:used], ck2[:used])
    for src, want in (({"x": k.x}, bwd[0]), ({"ckpt": ck2}, bwd[1])):
        dx.zero_()
        for a, b in zip(k.backward(fwd[1], fwd[2], dx=dx, **src), want):
            assert torch.equal(a, b)
    for t in (y, dx):
        whole = torch.as_strided(t, (n, s, width), (s * width, width, 1), 0)
        assert int(torch.isnan(whole).sum()) == n * s * (width - c)


@pytest.mark.parametrize("n,s,c,groups", [(70000, 64, 512, 32), (40, 1 << 20, 64, 8)])
def test_group_norm_past_32_bits(n, s, c, groups):
    """More than 2^31 elements, in short samples and in long ones: first and last samples against
    float64, the parameters' gradients against sums on the device."""
    import torch

    import act_reference as R
    from layer_wise_top_amd import lags
    assert n * s * c > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(3)
    x, dy = torch.empty(n, s, c, dtype=torch.bfloat16, device="cuda"), torch.empty(n, s, c, dtype=torch.bfloat16, device="cuda")
    for t in (x, dy):
        t.normal_(generator=g)
    gamma, beta = torch.randn(c, generator=g, device="cuda"), torch.randn(c, generator=g, device="cuda")
    gn = lags.GroupNorm(n, s, c, groups, dtype=torch.bfloat16, act="none")
    ws, ck = lags.gn_workspace(gn), lags.checkpoint(n * s, c)
    y, mean, rstd = torch.full_like(x, 9.0), torch.empty(n, groups, device="cuda"), torch.empty(n, groups, device="cuda")
    print("forward", (n, s, c), flush=True)
    lags.lags_gn_forward(gn, x, gamma, beta, y, mean, rstd, ws, ckpt=ck)
    rows = min(s, 4096)
    at = [0, n // 2 + 1, n - 1]
    want_mean, want_rstd = [], []
    for i in at:
        xi = x[i].double().view(s, groups, c // groups)
        m = xi.mean(dim=(0, 2))
        r = 1 / torch.sqrt(((xi - m[:, None]) ** 2).mean(dim=(0, 2)) + 1e-5)
        # sums of s * c / groups terms near 1 in chains of at most 1100 additions
        assert ((mean[i].double() - m).abs() <= 1100 * R.U).all() and ((rstd[i].double() - r).abs() <= 1100 * R.U).all()
        z = (x[i, -rows:].double() - m.repeat_interleave(c // groups)) * r.repeat_interleave(c // groups) * gamma + beta
        assert ((y[i, -rows:].double() - z).abs() <= 2.0 ** -8 * z.abs() + 1e-3).all()
    dx, dg, db = y.fill_(9.0), torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
    for src in ({"x": x}, {"ckpt": ck}):
        dx.fill_(9.0)
        print("backward", list(src), flush=True)
        lags.lags_gn_backward(gn, dy, gamma, beta, mean, rstd, dx, dg, db, ws, **src)
        sb, sg, mb, mg = (torch.zeros(c, dtype=torch.float64, device="cuda") for _ in range(4))
        step = max(1, (1 << 26) // (s * c))
        held = torch.empty(min(step, n), s, c, device="cuda") if "ckpt" in src else None
        for i in range(0, n, step):
            d = dy[i:i + step].double()
            if held is None:
                v = x[i:i + step].double()
            else:                                       # the same rows packed by themselves
                part, out = x[i:i + step], held[:min(step, n - i)]
                pc = lags.checkpoint(part.shape[0] * s, c)
                lags.lags_ckpt_pack(part, pc)
                lags.lags_ckpt_unpack(pc, out)
                v = out.double()
            cg = c // groups
            m = mean[i:i + step].double().repeat_interleave(cg, 1)[:, None]
            r = rstd[i:i + step].double().repeat_interleave(cg, 1)[:, None]
            xh = (v - m) * r
            sb, sg, mb, mg = sb + d.sum((0, 1)), sg + (d * xh).sum((0, 1)), mb + d.abs().sum((0, 1)), mg + (d * xh).abs().sum((0, 1))
            if i == 0 or i + step >= n:                 # the last sample (or the first) in full
                j = 0 if i == 0 else d.shape[0] - 1
                dz, h = gamma * d[j], xh[j]

                def mean_g(t):
                    return t.view(s, groups, cg).mean((0, 2)).repeat_interleave(cg)
                w = r[j] * (dz - mean_g(dz) - h * mean_g(dz * h))
                got = dx[i + j].double()
                assert ((got - w).abs() <= 2.0 ** -8 * w.abs() + 1e-3).all(), (list(src), i + j)
            del d, v, xh
        # chains of at most 2100 additions
        assert ((db.double() - sb).abs() <= 2100 * R.U * mb).all() and ((dg.double() - sg).abs() <= 2100 * R.U * mg).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weight_gradient_past_32_bits(dtype):
    """dY of more than 2^31 elements: values in the first and the last rows alone, so that the product is
    theirs."""
    import torch

    import act_reference as R
    from layer_wise_top_amd import lags
    m, o, c = (1 << 21) + 77, 1030, 64
    assert m * o > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(5)
    dy = torch.zeros(m, o, dtype=getattr(torch, "bfloat16" if dtype == "bf16" else "float32"), device="cuda")
    x = torch.randn(m, c, generator=g, device="cuda")
    for part in (dy[:200], dy[m // 2:m // 2 + 100], dy[-300:]):
        part.normal_(generator=g)
    ck, val = lags.checkpoint(m, c), torch.empty_like(x)
    lags.lags_ckpt_pack(x, ck)
    lags.lags_ckpt_unpack(ck, val)
    dw = torch.full((o, c), 9.0, device="cuda")
    lags.lags_ckpt_wgrad(dy, ck, dw, lags.wgrad_workspace(m, o, c, dy.dtype))
    d, v = (torch.cat([t[:200], t[m // 2:m // 2 + 100], t[-300:]]).double() for t in (dy, val))
    d = d.t().contiguous()
    want, mag = d @ v, d.abs() @ v.abs()
    assert ((dw.double() - want).abs() <= (600 / 16 + 64) * R.U * mag).all()


def test_group_norm_of_more_samples_than_a_launch_has_threads():
    """2^26 workgroups of 64 threads are more than the 2^32 - 1 threads of one launch: samples of both
    launches, the checkpoint's too."""
    import numpy as np
    import torch

    import act_reference as R
    from layer_wise_top_amd import lags
    n, c = (1 << 26) + 5, 8
    x = torch.zeros(n, 1, c, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, 12345678, (1 << 26) - 2, (1 << 26) - 1, 1 << 26, n - 1], device="cuda")
    x[at] = torch.from_numpy(np.random.default_rng(6).standard_normal((len(at), 1, c))).bfloat16().cuda()
    gamma, beta = torch.linspace(0.5, 2, c, device="cuda"), torch.linspace(-1, 1, c, device="cuda")
    gn = lags.GroupNorm(n, 1, c, 1, dtype=torch.bfloat16, act="silu", eps=1e-5)
    y, mean, rstd = torch.full_like(x, 9.0), torch.full((n, 1), 9.0, device="cuda"), torch.full((n, 1), 9.0, device="cuda")
    ck = lags.checkpoint(n, c)
    lags.lags_gn_forward(gn, x, gamma, beta, y, mean, rstd, lags.gn_workspace(gn), ckpt=ck)
    want, err = R.forward(x[at].double().cpu().numpy(), gamma.double().cpu().numpy(), beta.double().cpu().numpy(), 1,
                          1e-5, "silu")
    for name, got, w, e in zip(("y", "mean", "rstd"), (y, mean, rstd), want, err):
        R.check(name, got[at].double().cpu().numpy(), w, e, "bf16" if name == "y" else "f32")
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[at] = False
    flat = torch.nn.functional.silu(beta).bfloat16()          # a constant group: y = silu(beta)
    assert ((y[rest, 0].float() - flat.float()).abs().amax(dim=0) <= 2.0 ** -8).all()
    assert (mean[rest] == 0).all()
    out = torch.full_like(x, 9.0)
    lags.lags_ckpt_unpack(ck, out)
    ref = torch.from_numpy(R.held(x[at, 0].double().cpu().numpy())).bfloat16()
    assert torch.equal(out[at, 0].cpu(), ref) and not out[rest].any()


def test_checkpoint_of_more_rows_than_a_launch_has_threads():
    """2^31 rows of one column, eight lanes each."""
    import numpy as np
    import torch

    import act_reference as R
    from layer_wise_top_amd import lags
    rows = (1 << 31) + 3
    x = torch.zeros(rows, 1, device="cuda")
    at = torch.tensor([0, 77, (1 << 31) - 129, (1 << 31) - 1, 1 << 31, rows - 1], device="cuda")
    x[at] = torch.from_numpy(np.random.default_rng(7).standard_normal((len(at), 1))).float().cuda()
    ck = lags.checkpoint(rows, 1)
    lags.lags_ckpt_pack(x, ck)
    want = torch.from_numpy(R.held(x[at].double().cpu().numpy())).float()
    x.fill_(9.0)
    lags.lags_ckpt_unpack(ck, x)
    assert torch.equal(x[at].cpu(), want)
    x[at] = 0
    assert not x.any()


# ---- magnitudes at the top of the range ------------------------------------
# From 127.5/128 2^128 up (the largest bf16 value is one of them) a run's largest code is 64 steps of
# 2^122: a value past fp32.  The gradients stay finite and within the format's bound.

TOPS = {"f32": [3.4028234663852886e38, 127.5 / 128 * 2.0 ** 128], "bf16": [255 * 2.0 ** 120]}


def _top_runs(dtype):
    """Rows of one run each with one or more of the largest magnitudes, and ordinary rows."""
    import numpy as np
    import torch
    rng = np.random.default_rng(11)
    rows = [rng.standard_normal(32) for _ in range(4)]
    for t in TOPS[dtype]:
        for sign in (1.0, -1.0):
            r = rng.uniform(-1, 1, 32) * t
            r[3], r[17] = sign * t, 0.0
            rows.append(r)
    x = torch.from_numpy(np.array(rows)).to(getattr(torch, "float32" if dtype == "f32" else "bfloat16"))
    assert torch.isfinite(x).all()
    return x.cuda()


@pytest.mark.parametrize("dtype", list(TOPS))
@pytest.mark.parametrize("dy_dtype", ["f32", "bf16", "f16"])
def test_weight_gradient_of_the_largest_values(dtype, dy_dtype):
    """Finite products, and a zero of dY takes a row out: held values are off by 1/128 of the run's
    largest magnitude at most, sums by their roundings."""
    import torch
    from layer_wise_top_amd import lags
    x = _top_runs(dtype)
    m = x.shape[0]
    ck = lags.checkpoint(m, 32)
    lags.lags_ckpt_pack(x, ck)
    dy = torch.zeros(m, 70, device="cuda")
    dy[torch.arange(m), torch.arange(m)] = 2.0 ** -10        # one row of x each
    dy[:4, 60] = 1.0                                          # the ordinary rows alone
    dy = dy.to({"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dy_dtype])
    dw = torch.full((70, 32), 9.0, device="cuda")
    lags.lags_ckpt_wgrad(dy, ck, dw, lags.wgrad_workspace(m, 70, 32, dy.dtype))
    assert torch.isfinite(dw).all()
    want = dy.double().t() @ x.double()
    bound = dy.double().abs().t() @ (x.double().abs().amax(dim=1, keepdim=True) / 127.5).expand(m, 32)
    assert ((dw.double() - want).abs() <= bound * (1 + 1e-6)).all()


@pytest.mark.parametrize("s", [1, 9000])
@pytest.mark.parametrize("dtype", list(TOPS))
def test_group_norm_backward_of_the_largest_values(dtype, s):
    """Statistics given: rstd = 2^-127 keeps xh about 1, and the bound is the format's error times rstd
    through the formula; a group without such values is as it was."""
    import numpy as np
    import torch
    from layer_wise_top_amd import lags
    rows = _top_runs(dtype)
    n, c = rows.shape[0], 32
    x = torch.zeros(n, s, c, dtype=rows.dtype, device="cuda")
    x[:, 0] = rows
    rng = np.random.default_rng(12)
    dy = torch.from_numpy(rng.standard_normal((n, s, c))).to(rows.dtype).cuda()
    mean = torch.zeros(n, 1, device="cuda")
    rstd = torch.full((n, 1), 2.0 ** -127, device="cuda")
    rstd[:4] = 1.0
    gn = lags.GroupNorm(n, s, c, 1, dtype=rows.dtype, act="none")
    ck = lags.checkpoint(n * s, c)
    lags.lags_ckpt_pack(x, ck)
    dx, dg, db = torch.full_like(x, 9.0), torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
    lags.lags_gn_backward(gn, dy, None, None, mean, rstd, dx, dg, db, lags.gn_workspace(gn), ckpt=ck)
    for t in (dx, dg, db):
        assert torch.isfinite(t).all()
    xh, e = x.double() * rstd.double()[:, None], (x.double().abs().amax(dim=2, keepdim=True) / 127.5) * rstd.double()[:, None]
    d = dy.double()
    # the held xh is off by e, the sums by 2^-16 of their terms at most (chains of up to 100 additions)
    eg = ((d * e).abs() + 2.0 ** -16 * (d * xh).abs()).sum(dim=(0, 1))
    assert ((dg.double() - (d * xh).sum(dim=(0, 1))).abs() <= eg).all()
    s2, es2 = (d * xh).mean(dim=(1, 2), keepdim=True), ((d * e).abs() + 2.0 ** -16 * (d * xh).abs()).mean(dim=(1, 2), keepdim=True)
    s1, es1 = d.mean(dim=(1, 2), keepdim=True), 2.0 ** -16 * d.abs().mean(dim=(1, 2), keepdim=True)
    r = rstd.double()[:, None]
    want = r * (d - s1 - xh * s2)
    bound = r * (es1 + e * (s2.abs() + es2) + xh.abs() * es2 + 2.0 ** -8 * (d.abs() + s1.abs() + (xh * s2).abs())) + 2.0 ** -133
    assert ((dx.double() - want).abs() <= bound).all()


# ---- small gradients -------------------------------------------------------

def test_weight_gradient_of_small_fp32_values():
    """The terms of a 32-bit dY end at bf16's smallest value, 2^-133: what is below it is cut.  Down to
    2^-110 nothing is; sums here have one row, so a product is rounded at most three times."""
    import numpy as np
    import torch
    from layer_wise_top_amd import lags
    rng = np.random.default_rng(13)
    e = np.repeat(np.arange(-126, -94), 4)
    v = (rng.uniform(1, 2, e.size) * 2.0 ** e).astype(np.float32)
    dy = torch.from_numpy(v[None, :]).cuda()
    x = torch.full((1, 32), 2.0 ** 60, device="cuda")
    ck = lags.checkpoint(1, 32)
    lags.lags_ckpt_pack(x, ck)
    dw = torch.empty(e.size, 32, device="cuda")
    lags.lags_ckpt_wgrad(dy, ck, dw, lags.wgrad_workspace(1, e.size, 32, torch.float32))
    want = v.astype(np.float64) * 2.0 ** 60
    off = np.abs(dw.double().cpu().numpy() - want[:, None]).max(axis=1)
    print("relative error by exponent", {int(k): float((off / want)[e == k].max()) for k in np.unique(e)}, flush=True)
    assert (off[e >= -110] <= 3 * 2.0 ** -24 * want[e >= -110]).all()
    assert (off <= 3 * 2.0 ** -24 * want + 2.0 ** (-133 + 60)).all()


@pytest.mark.parametrize("n,s", [(3, 30), (2, 9000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("at", [0, 1, 4000])
def test_group_norm_with_the_lowest_value(dtype, n, s, at):
    """One value of a group is the type's lowest (a mask), resident and in chunks, at a thread's first
    position and later: its square is past fp32, so the variance is infinite, rstd 0 and y act(beta);
    the mean is finite.  So are the gradients; other groups keep their bits."""
    import numpy as np
    import torch

    import act_reference as R
    k = Case(n, s, 64, 8, dtype, "silu", seed=5)
    clean = k.forward()
    at %= s
    lowest = torch.finfo(k.x.dtype).min
    k.x[0, at, 9] = lowest
    y, mean, rstd = k.forward()
    for t in (y, mean, rstd):
        assert torch.isfinite(t).all()
    assert rstd[0, 1] == 0
    want = lowest / (8 * s)                       # the others' part is far below its rounding
    assert abs(float(mean[0, 1]) - want) <= 1e-5 * abs(want)
    flat = R.act(k.b64, "silu")[8:16]
    assert np.abs(y[0, :, 8:16].double().cpu().numpy() - flat).max() <= 2.0 ** -7 * np.abs(flat).max()
    keep = torch.ones(n, 8, dtype=torch.bool, device="cuda")
    keep[0, 1] = False
    assert torch.equal(mean[keep], clean[1][keep]) and torch.equal(rstd[keep], clean[2][keep])
    wide = keep.repeat_interleave(8, 1)[:, None, :].expand(n, s, 64)
    assert torch.equal(y[wide], clean[0][wide])
    for t in k.backward(mean, rstd, x=k.x):
        assert torch.isfinite(t).all()
