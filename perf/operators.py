"""The activation operators that are measured: 8-bit activation checkpoints,
group normalisation with an activation (channels last, both directions) and
the weight gradient taken from a checkpoint.

A case names its operator in ``op``:

``ckpt``       an activation packed to 8 bits and unpacked again
``gn_fwd``     y = act(groupnorm(x)), with the statistics the backward needs
``gn_bwd``     dx, dgamma, dbeta from dy and x, or from dy and x's checkpoint
``gn_train``   a forward that also writes x's checkpoint, then the backward
               from that checkpoint alone
``wgrad``      dW = dY^T X with X held as a checkpoint

``own`` chooses between the library's calls and the plain form (elementary
torch operations in 32 bits).  Matrices are [rows, channels], channels last.

The checkpoint of a [rows, cols] matrix is one buffer: int8 codes
[rows][pitch], pitch = cols rounded up to 16, then one scale byte s for each
row's run of 32 columns, [rows][ceil(cols / 32)].  A code q stands for
q * 2^(s - 127); s = 255 marks a run that held an infinity or NaN.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = 32
EPS = 1e-5


def listed():
    return [
        # the last stage of ResNet-20 (8x8x64), a batch of 32 per worker: latency
        dict(name="ckpt-resnet20", op="ckpt", rows=2048, cols=64, dtype="f32"),
        # the hidden activation of the 1.3B transformer's MLP (4 x 2048 wide), 16K tokens
        dict(name="ckpt-mlp", op="ckpt", rows=16384, cols=8192, dtype="bf16"),
        # ResNet-20, last stage: the smallest call
        dict(name="fwd-resnet20", op="gn_fwd", n=32, s=64, groups=8, cg=8, dtype="f32", act="relu"),
        # ResNet-50's first layer, 112x112x64: samples far larger than a compute unit holds
        dict(name="fwd-stem", op="gn_fwd", n=64, s=12544, groups=32, cg=2, dtype="bf16", act="relu"),
        # odd everything: 33x47 positions, 12 channels a group, 3 groups
        dict(name="fwd-odd", op="gn_fwd", n=5, s=1551, groups=3, cg=12, dtype="f16", act="silu"),
        # ResNet-20, middle stage, from the stored input
        dict(name="bwd-resnet20", op="gn_bwd", n=32, s=256, groups=8, cg=4, dtype="f32", act="relu",
             ckpt=False),
        # ResNet-50, 56x56x256, from the checkpoint
        dict(name="bwd-resnet50", op="gn_bwd", n=64, s=3136, groups=32, cg=8, dtype="bf16", act="relu",
             ckpt=True),
        # ResNet-50, 28x28x512, forward and backward of a training step
        dict(name="train-resnet50", op="gn_train", n=64, s=784, groups=32, cg=16, dtype="bf16",
             act="silu"),
        # a 1x1 projection of ResNet-20's size: the smallest weight gradient
        dict(name="wgrad-resnet20", op="wgrad", rows=2048, outs=64, cols=32, dtype="f32"),
        # ResNet-50's first stage, 1x1 convolution 64 -> 256 at 56x56: very many rows, a small product
        dict(name="wgrad-resnet50", op="wgrad", rows=200704, outs=256, cols=64, dtype="bf16"),
        # the LSTM's input-to-gates matrix (1500 -> 4 x 1500), 35 steps of 20 sequences, fp32
        dict(name="wgrad-lstm", op="wgrad", rows=700, outs=6000, cols=1500, dtype="f32"),
        # the 1.3B transformer's fc1 (2048 -> 8192), 16K tokens: matrix rate
        dict(name="wgrad-mlp", op="wgrad", rows=16384, outs=8192, cols=2048, dtype="bf16"),
    ]


def draw(rng):
    """One more case of the same ranges (each operator up to its largest listed one)."""
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["ckpt", "gn_fwd", "gn_bwd", "gn_train", "wgrad"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    if op == "ckpt":
        most = 16384 * 8192 // (2 if dtype == "f32" else 1)
        cols = log_int(8, 8192)
        return dict(op=op, rows=log_int(1, min(200704, most // cols)), cols=cols, dtype=dtype)
    if op == "wgrad":
        outs, cols = log_int(16, 8192), log_int(16, 8192)
        # three matrix passes stand for one where dY has 32 bits, two where it has 16-bit floats
        most = 16384 * 8192 * 2048 // {"f32": 4, "f16": 2, "bf16": 1}[dtype]
        rows = log_int(1, max(1, min(200704, most // (outs * cols))))
        return dict(op=op, rows=rows, outs=outs, cols=cols, dtype=dtype)
    groups, cg, s = log_int(1, 32), log_int(1, 64), log_int(4, 12544)
    if s * cg < 64:     # a group of a few values has a backward that cancels to nothing
        s = -(-64 // cg) + rng.randrange(8)
    most = 64 * 12544 * 64 // ((2 if dtype == "f32" else 1) * (2 if op == "gn_train" else 1))
    n = log_int(1, max(1, min(256, most // (s * groups * cg))))
    case = dict(op=op, n=n, s=s, groups=groups, cg=cg, dtype=dtype)
    if op == "gn_train":
        # no relu here: where its argument rounds to either side of zero the gradient jumps, and this
        # pass computes its own statistics; gn_bwd, which is given them, has it
        case["act"] = rng.choice(["none", "silu"])
    else:
        case["act"] = rng.choice(["none", "relu", "silu"])
    if op == "gn_bwd":
        case["ckpt"] = rng.random() < 0.5
    return case


def work(case):
    e = 4 if case["dtype"] == "f32" else 2

    def packed(rows, cols):
        return rows * cols + rows * -(-cols // BLOCK)

    if case["op"] == "ckpt":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * e + 2 * packed(case["rows"], case["cols"]), "flops": 4 * n}
    if case["op"] == "wgrad":
        m, o, c = case["rows"], case["outs"], case["cols"]
        return {"bytes": m * o * e + packed(m, c) + 4 * o * c, "flops": 2 * m * o * c}
    rows, c = case["n"] * case["s"], case["groups"] * case["cg"]
    n, stats = rows * c, 8 * case["n"] * case["groups"] + 8 * c
    if case["op"] == "gn_fwd":
        return {"bytes": 2 * n * e + stats, "flops": 8 * n}
    if case["op"] == "gn_bwd":
        return {"bytes": 2 * n * e + (packed(rows, c) if case["ckpt"] else n * e) + stats + 8 * c,
                "flops": 20 * n}
    return {"bytes": 4 * n * e + 2 * packed(rows, c) + 2 * stats + 8 * c, "flops": 32 * n}


# ---- inputs ----------------------------------------------------------------

def _generator(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _raw(case, seed):
    """The inputs as they come from the rest of a model, before anything is packed."""
    g = _generator(case, seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    if case["op"] == "ckpt":
        # channels of unlike size, a few of them large
        x = normal(case["rows"], case["cols"]) * torch.exp(0.7 * normal(case["cols"]))
        return {"x": x.to(dt)}
    if case["op"] == "wgrad":
        # a rectified activation and a small gradient
        x = torch.relu(normal(case["rows"], case["cols"]) * torch.exp(0.5 * normal(case["cols"])))
        dy = normal(case["rows"], case["outs"]) * 1e-2
        return {"x": x, "dy": dy.to(dt)}
    n, s, c = case["n"], case["s"], case["groups"] * case["cg"]
    # a convolution's output: each channel with a mean and a spread of its own
    x = normal(n, s, c) * torch.exp(0.5 * normal(c)) + 0.5 * normal(c)
    raw = {"x": x.to(dt), "gamma": 1 + 0.2 * normal(c), "beta": 0.2 * normal(c)}
    if case["op"] != "gn_fwd":
        raw["dy"] = (normal(n, s, c) * 1e-2).to(dt)
    return raw


def _pack(x):
    """The checkpoint buffer of a [rows, cols] matrix, by torch operations."""
    rows, cols = x.shape
    pitch, nb = -(-cols // 16) * 16, -(-cols // BLOCK)
    q, s = _quantise(x.float())
    buf = torch.zeros(-(-(rows * (pitch + nb)) // 16) * 16, dtype=torch.uint8, device=x.device)
    buf[:rows * pitch].view(rows, pitch)[:, :cols] = q.to(torch.int8).view(torch.uint8)
    buf[rows * pitch:rows * (pitch + nb)] = s.to(torch.uint8).reshape(-1)
    return buf


def prepare(case, seed):
    st = _raw(case, seed)
    st["case"] = case
    op = case["op"]
    if op == "ckpt":
        rows, cols = st["x"].shape
    elif op == "wgrad":
        rows, cols = st["x"].shape
        st["ckpt"] = _pack(st.pop("x"))
    else:
        n, s, c = st["x"].shape
        rows, cols = n * s, c
        if op == "gn_bwd":
            xf = st["x"].double().view(n, s, case["groups"], case["cg"])
            mean = xf.mean(dim=(1, 3))
            var = (xf - mean[:, None, :, None]).square().mean(dim=(1, 3))
            st["mean"], st["rstd"] = mean.float(), (1 / torch.sqrt(var + EPS)).float()
            del xf
            if case["ckpt"]:
                st["ckpt"] = _pack(st.pop("x").view(rows, cols))
    if own:
        from layer_wise_top_amd import lags
        dt = DTYPES[case["dtype"]]
        if op == "ckpt":
            st["ckpt"] = lags.checkpoint(rows, cols)
            st["out"] = torch.empty_like(st["x"])
        elif op == "wgrad":
            st["dw"] = torch.empty(case["outs"], cols, device=DEV)
            st["ws"] = lags.wgrad_workspace(rows, case["outs"], cols, dt)
        else:
            st["gn"] = lags.GroupNorm(n, s, c, case["groups"], dtype=dt, act=case["act"], eps=EPS)
            st["ws"] = lags.gn_workspace(st["gn"])
            if op != "gn_bwd":
                st["y"] = torch.empty_like(st["x"])
                st["mean"] = torch.empty(n, case["groups"], device=DEV)
                st["rstd"] = torch.empty(n, case["groups"], device=DEV)
            if op != "gn_fwd":
                st["dx"] = torch.empty_like(st["dy"])
                st["dgamma"], st["dbeta"] = torch.empty(c, device=DEV), torch.empty(c, device=DEV)
            if op == "gn_train":
                st["ckpt"] = lags.checkpoint(rows, cols)
    return st


# ---- the plain form --------------------------------------------------------

def _quantise(x):
    """Codes and scale bytes of an fp32 [rows, cols] matrix, as fp32 and int32."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    xb = torch.nn.functional.pad(x, (0, nb * BLOCK - cols)).view(rows, nb, BLOCK)
    amax = xb.abs().amax(dim=2)
    bad = ~torch.isfinite(xb).all(dim=2)
    bits = torch.where(bad, torch.zeros_like(amax), amax).view(torch.int32)
    # the exponent that takes the largest magnitude to [64, 127.5), so that it rounds to at most 127
    s = (torch.div(bits + 0x10000, 1 << 23, rounding_mode="floor") - 6).clamp(min=1)
    inv = ((254 - s) << 23).view(torch.float32)
    q = torch.round(xb * inv[:, :, None])
    q = torch.where(bad[:, :, None], torch.zeros_like(q), q)
    s = torch.where(bad, torch.full_like(s, 255), s)
    return q.view(rows, nb * BLOCK)[:, :cols], s


def _values(q, s):
    rows, cols = q.shape
    step = (s << 23).view(torch.float32)        # 255 gives infinity, and 0 times that NaN
    return q * step.repeat_interleave(BLOCK, dim=1)[:, :cols]


def _unpack(buf, rows, cols):
    pitch, nb = -(-cols // 16) * 16, -(-cols // BLOCK)
    q = buf[:rows * pitch].view(torch.int8).view(rows, pitch)[:, :cols].float()
    s = buf[rows * pitch:rows * (pitch + nb)].view(rows, nb).to(torch.int32)
    return _values(q, s)


def _plain_stats(xf, case):
    n, s, c = xf.shape
    v = xf.view(n, s, case["groups"], case["cg"])
    mean = v.mean(dim=(1, 3))
    var = (v - mean[:, None, :, None]).square().mean(dim=(1, 3))
    return mean, 1 / torch.sqrt(var + EPS)


def _plain_forward(x, gamma, beta, mean, rstd, case):
    cg = case["cg"]
    m, r = (t.repeat_interleave(cg, dim=1)[:, None, :] for t in (mean, rstd))
    z = (x.float() - m) * r
    z = z * gamma
    z = z + beta
    if case["act"] == "relu":
        z = torch.where(z > 0, z, torch.zeros_like(z))
    elif case["act"] == "silu":
        z = z / (1 + torch.exp(-z))
    return z.to(x.dtype)


def _plain_backward(dy, xf, gamma, beta, mean, rstd, case):
    n, s, c = xf.shape
    groups, cg = case["groups"], case["cg"]
    m, r = (t.repeat_interleave(cg, dim=1)[:, None, :] for t in (mean, rstd))
    xh = (xf - m) * r
    dz = dy.float()
    if case["act"] != "none":
        z = xh * gamma
        z = z + beta
        if case["act"] == "relu":
            dz = torch.where(z > 0, dz, torch.zeros_like(dz))
        else:
            sg = 1 / (1 + torch.exp(-z))
            dz = dz * (sg * (1 + z * (1 - sg)))
    a, b = dz.sum(dim=1), (dz * xh).sum(dim=1)                    # [n, c]
    cnt = s * cg
    s1 = ((a * gamma).view(n, groups, cg).sum(dim=2) / cnt).repeat_interleave(cg, dim=1)[:, None, :]
    s2 = ((b * gamma).view(n, groups, cg).sum(dim=2) / cnt).repeat_interleave(cg, dim=1)[:, None, :]
    dx = r * (gamma * dz - s1 - xh * s2)
    return dx.to(dy.dtype), b.sum(dim=0), a.sum(dim=0)


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "ckpt":
        return _values(*_quantise(st["x"].float())).to(st["x"].dtype)
    if op == "wgrad":
        return st["dy"].float().t() @ _unpack(st["ckpt"], case["rows"], case["cols"])
    n, s, c = case["n"], case["s"], case["groups"] * case["cg"]
    if op == "gn_bwd":
        xf = _unpack(st["ckpt"], n * s, c).view(n, s, c) if case["ckpt"] else st["x"].float()
        dx, dgamma, dbeta = _plain_backward(st["dy"], xf, st["gamma"], st["beta"], st["mean"],
                                            st["rstd"], case)
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    mean, rstd = _plain_stats(st["x"].float(), case)
    y = _plain_forward(st["x"], st["gamma"], st["beta"], mean, rstd, case)
    out = {"y": y, "mean": mean, "rstd": rstd}
    if op == "gn_train":
        xf = _values(*_quantise(st["x"].float().view(n * s, c))).view(n, s, c)
        out["dx"], out["dgamma"], out["dbeta"] = _plain_backward(
            st["dy"], xf, st["gamma"], st["beta"], mean, rstd, case)
    return out


# ---- the library's calls ---------------------------------------------------

def _run_own(st):
    from layer_wise_top_amd import lags
    op = st["case"]["op"]
    if op == "ckpt":
        lags.lags_ckpt_pack(st["x"], st["ckpt"])
        lags.lags_ckpt_unpack(st["ckpt"], st["out"])
        return st["out"]
    if op == "wgrad":
        lags.lags_ckpt_wgrad(st["dy"], st["ckpt"], st["dw"], st["ws"])
        return st["dw"]
    if op == "gn_bwd":
        lags.lags_gn_backward(st["gn"], st["dy"], st["gamma"], st["beta"], st["mean"], st["rstd"],
                              st["dx"], st["dgamma"], st["dbeta"], st["ws"],
                              x=st.get("x"), ckpt=st.get("ckpt"))
        return {"dx": st["dx"], "dgamma": st["dgamma"], "dbeta": st["dbeta"]}
    out = {"y": st["y"], "mean": st["mean"], "rstd": st["rstd"]}
    lags.lags_gn_forward(st["gn"], st["x"], st["gamma"], st["beta"], st["y"], st["mean"], st["rstd"],
                         st["ws"], ckpt=st.get("ckpt"))
    if op == "gn_train":
        lags.lags_gn_backward(st["gn"], st["dy"], st["gamma"], st["beta"], st["mean"], st["rstd"],
                              st["dx"], st["dgamma"], st["dbeta"], st["ws"], ckpt=st["ckpt"])
        out.update(dx=st["dx"], dgamma=st["dgamma"], dbeta=st["dbeta"])
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- the definitions in 64 bits --------------------------------------------

def _held(x):
    """What an 8-bit checkpoint of a finite float64 [rows, cols] matrix stands for: in each run of 32
    columns, multiples of the smallest power of two, 2^-126 at least, that takes every value to at
    most 127 when rounded to the nearest multiple, ties to even."""
    out = torch.empty_like(x)
    for lo in range(0, x.shape[1], BLOCK):
        run_ = x[:, lo:lo + BLOCK]
        top = run_.abs().amax(dim=1, keepdim=True)
        m, e = torch.frexp(top)                   # top = m 2^e, m in [1/2, 1)
        p = e - 7 + (torch.round(m * 128) > 127).to(e.dtype)
        p = torch.where(top > 0, p, torch.full_like(p, -126)).clamp(min=-126)
        unit = ((p.to(torch.int64) + 1023) << 52).view(torch.float64)       # 2^p, exactly
        out[:, lo:lo + BLOCK] = torch.round(run_ / unit) * unit
    return out


def exact(case, seed):
    raw = _raw(case, seed)
    op = case["op"]
    if op == "ckpt":
        return _held(raw["x"].double())
    if op == "wgrad":
        return raw["dy"].double().t().contiguous() @ _held(raw["x"].double())
    n, s, groups, cg = case["n"], case["s"], case["groups"], case["cg"]
    c = groups * cg
    x = raw["x"].double()
    gamma, beta = (raw[k].double().view(groups, cg) for k in ("gamma", "beta"))
    v = x.view(n, s, groups, cg)
    mu = v.sum(dim=(1, 3), keepdim=True) / (s * cg)
    r = ((v - mu).pow(2).sum(dim=(1, 3), keepdim=True) / (s * cg) + EPS).rsqrt()
    out = {}
    if op != "gn_bwd":
        z = gamma * ((v - mu) * r) + beta
        y = {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z)}[case["act"]]()
        out = {"y": y.reshape(n, s, c), "mean": mu.reshape(n, groups), "rstd": r.reshape(n, groups)}
        del z, y
        if op == "gn_fwd":
            return out
    if op == "gn_bwd":      # these are inputs here, in 32 bits
        mu, r = mu.float().double(), r.float().double()
    if op == "gn_train" or case["ckpt"]:
        v = _held(x.view(n * s, c)).view(n, s, groups, cg)
    dy = raw["dy"].double().view(n, s, groups, cg)
    xh = (v - mu) * r
    if case["act"] == "relu":
        dy = dy * (gamma * xh + beta > 0)
    elif case["act"] == "silu":
        z = gamma * xh + beta
        sg = torch.sigmoid(z)
        dy = dy * (sg + z * sg * (1 - sg))
        del z, sg
    dbeta, dgamma = dy.sum(dim=(0, 1)), (dy * xh).sum(dim=(0, 1))
    dxh = gamma * dy
    dx = r * (dxh - dxh.mean(dim=(1, 3), keepdim=True) - xh * (dxh * xh).mean(dim=(1, 3), keepdim=True))
    out.update(dx=dx.reshape(n, s, c), dgamma=dgamma.reshape(c), dbeta=dbeta.reshape(c))
    return out
