"""Plain float64 references of the activation operators, written from their
definitions, and the error bounds their tests use.

u = 2^-24 is fp32's unit roundoff.  A sum of n terms in any order is off by at
most d u sum|terms| where d is the longest chain of additions; the kernels'
chains (rows of a thread, lanes, waves, chunks) stay below `CHAIN`."""
import numpy as np

U = 2.0 ** -24
CHAIN = 64
ROUND = {"f32": 0.0, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}      # one rounding to the type, with slack of 2
TINY = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -24}            # fp16's subnormal spacing
RUN = 32


def quantise(x):
    """Codes [rows, cols] and exponents [rows, runs] of a float64 array; a run that is not finite has
    codes 0 and exponent 128 (scale byte 255)."""
    rows, cols = x.shape
    nrun = -(-cols // RUN)
    v = np.zeros((rows, nrun * RUN))
    v[:, :cols] = x
    v = v.reshape(rows, nrun, RUN)
    bad = ~np.isfinite(v).all(axis=2)
    v = np.where(bad[:, :, None], 0.0, v)
    top = np.abs(v).max(axis=2)
    p = np.full(top.shape, -126)
    some = top > 0
    p[some] = np.maximum(-126, np.floor(np.log2(top[some])).astype(int) - 8)
    while True:                                # the smallest exponent that keeps every code within 127
        over = np.abs(np.rint(np.ldexp(top, -p))) > 127
        if not over.any():
            break
        p[over] += 1
    q = np.rint(np.ldexp(v, -p[:, :, None])).reshape(rows, nrun * RUN)[:, :cols]
    return q, np.where(bad, 128, p)


def held(x):
    """What the 8-bit format holds of a float64 [rows, cols] array (NaN runs where not finite)."""
    q, p = quantise(x)
    e = np.repeat(p, RUN, axis=1)[:, :x.shape[1]]
    return np.where(e == 128, np.nan, np.ldexp(q, np.where(e == 128, 0, e)))


def codes(x):
    """The checkpoint buffer (uint8) of a float64 [rows, cols] array, and its bytes in use."""
    rows, cols = x.shape
    pitch, nrun = -(-cols // 16) * 16, -(-cols // RUN)
    q, p = quantise(x)
    padded = np.zeros((rows, pitch), np.int8)
    padded[:, :cols] = q
    n = rows * (pitch + nrun)
    buf = np.zeros(-(-n // 16) * 16, np.uint8)
    buf[:rows * pitch] = padded.view(np.uint8).reshape(-1)
    buf[rows * pitch:n] = (p + 127).astype(np.uint8).reshape(-1)
    return buf, n


def stats(x, groups, eps):
    """x: float64 [N, S, C] -> mean, rstd [N, G]."""
    n, s, c = x.shape
    v = x.reshape(n, s, groups, c // groups)
    mean = v.mean(axis=(1, 3))
    var = ((v - mean[:, None, :, None]) ** 2).mean(axis=(1, 3))
    return mean, 1 / np.sqrt(var + eps)


def per_channel(t, c):
    """[N, G] -> [N, 1, C]."""
    return np.repeat(t, c // t.shape[1], axis=1)[:, None, :]


def act(z, kind):
    with np.errstate(over="ignore", invalid="ignore"):
        return {"none": z, "relu": np.where(np.isnan(z), z, np.maximum(z, 0)), "silu": z / (1 + np.exp(-z))}[kind]


def z_fp32(x, gamma, beta, mean, rstd):
    """z with every operation rounded to fp32, as defined (x: float32 [N, S, C])."""
    c = x.shape[2]
    f = np.float32
    xh = (x.astype(f) - per_channel(mean.astype(f), c)) * per_channel(rstd.astype(f), c)
    return xh * gamma.astype(f) + beta.astype(f)


def backward(dy, x, gamma, beta, mean, rstd, kind):
    """dx, dgamma, dbeta in float64 from float64 x and the given statistics, and error bounds of
    each.  relu's mask is that of the fp32 z, as defined."""
    n, s, c = x.shape
    groups = mean.shape[1]
    m, r = per_channel(mean, c), per_channel(rstd, c)
    xh = (x - m) * r
    z = xh * gamma + beta
    # error of xh and z: three roundings of values no larger than these
    exh = 4 * U * (np.abs(x) + np.abs(m)) * r
    ez = exh * np.abs(gamma) + 4 * U * (np.abs(xh * gamma) + np.abs(beta))
    if kind == "relu":
        z32 = z_fp32(x.astype(np.float32), gamma, beta, mean, rstd)
        d = (z32 > 0).astype(np.float64)
        ed = np.zeros_like(z)
    elif kind == "silu":
        sg = 1 / (1 + np.exp(-z))
        d = sg * (1 + z * (1 - sg))
        # |d''| < 1; the exponential and the reciprocal are good to a few ulp
        ed = ez + (16 + 4 * np.abs(z)) * U * (sg + np.abs(z) * sg * (1 - sg) + np.abs(d))
    else:
        d, ed = np.ones_like(z), np.zeros_like(z)
    dz = dy * d
    edz = np.abs(dy) * ed + U * np.abs(dz)
    dbeta, dgamma = dz.sum(axis=(0, 1)), (dz * xh).sum(axis=(0, 1))
    edxh = edz * np.abs(xh) + np.abs(dz) * exh + U * np.abs(dz * xh)
    ebeta = (edz + CHAIN * U * np.abs(dz)).sum(axis=(0, 1))
    egamma = (edxh + CHAIN * U * np.abs(dz * xh)).sum(axis=(0, 1))

    def mean_g(t):
        return per_channel(t.reshape(n, s, groups, c // groups).mean(axis=(1, 3)), c)

    g, ag = gamma * dz, np.abs(gamma)
    s1, s2 = mean_g(g), mean_g(g * xh)
    es1 = mean_g(ag * edz + CHAIN * U * np.abs(g))
    es2 = mean_g(ag * edxh + CHAIN * U * np.abs(g * xh))
    dx = r * (g - s1 - xh * s2)
    edx = r * (ag * edz + es1 + np.abs(xh) * es2 + exh * np.abs(s2)
               + 4 * U * (np.abs(g) + np.abs(s1) + np.abs(xh * s2)))
    return (dx, dgamma, dbeta), (edx, egamma, ebeta)


def forward(x, gamma, beta, groups, eps, kind):
    """y, mean, rstd in float64 of a float64 x, and error bounds of each."""
    n, s, c = x.shape
    mean, rstd = stats(x, groups, eps)
    v = x.reshape(n, s, groups, c // groups)
    mag = np.abs(v).mean(axis=(1, 3))
    emean = (CHAIN + 2) * U * mag
    # squared distances: relative error of the sum, and the mean's own error squared
    var = 1 / rstd ** 2
    dist = np.abs(v - mean[:, None, :, None])
    evar = ((CHAIN + 8) * U * (dist ** 2).mean(axis=(1, 3)) + 2 * U * (np.abs(v) * dist).mean(axis=(1, 3))
            + 2 * emean * dist.mean(axis=(1, 3)) * U * CHAIN + emean ** 2)
    erstd = rstd * (0.5 * evar / var + 4 * U)
    m, r = per_channel(mean, c), per_channel(rstd, c)
    xh = (x - m) * r
    exh = (per_channel(emean, c) + 2 * U * (np.abs(x) + np.abs(m))) * r + np.abs(x - m) * per_channel(erstd, c)
    z = xh * gamma + beta
    ez = exh * np.abs(gamma) + 4 * U * (np.abs(xh * gamma) + np.abs(beta))
    y = act(z, kind)
    ey = ez if kind != "silu" else 1.1 * ez + (16 + 4 * np.abs(z)) * U * np.abs(y)
    return (y, mean, rstd), (ey, emean, erstd)


def check(name, got, want, bound, dtype="f32"):
    """got (float64 of the output) within `bound` plus one rounding to `dtype`; NaN where want is."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    bad = np.isnan(want)
    assert np.array_equal(np.isnan(got), bad), f"{name}: NaN in other places"
    inf = np.isinf(want) & ~bad
    assert np.array_equal(got[inf], want[inf]), f"{name}: infinities differ"
    ok = ~bad & ~inf
    lim = np.broadcast_to(bound, want.shape)[ok] * (1 + ROUND[dtype]) + ROUND[dtype] * np.abs(want[ok]) + TINY[dtype]
    err = np.abs(got[ok] - want[ok])
    if err.size and not (err <= lim).all():
        i = int(np.argmax(err - lim))
        raise AssertionError(f"{name}: off by {err[i]:.3g} at most {lim[i]:.3g} (value {want[ok][i]:.6g}), "
                             f"{int((err > lim).sum())} of {err.size}")
