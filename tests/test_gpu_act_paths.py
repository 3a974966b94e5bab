"""Paths of the activation operators that depend on a shape's plan, on the GPU,
against float64."""
import pytest

from test_gpu_gn import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["none", "relu", "silu"])
@pytest.mark.parametrize("n,s,c,groups", [(1100, 1, 4096, 1), (300, 3, 4096, 2), (150, 4, 2500, 1), (140, 2, 3001, 1),
                                          (3, 2, 4224, 2), (140, 5, 4096, 1)])
def test_fp32_groups_wider_than_2048_channels(n, s, c, groups, act):
    """A column of lanes of its own for each four channels: short samples whole in 1024 lanes, several
    of them a workgroup; five positions, and all of them where samples are few, in chunks."""
    Case(n, s, c, groups, "f32", act, seed=c + s).check_all()


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
