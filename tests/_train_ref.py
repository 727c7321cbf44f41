"""Plain float64 numpy forms of the training operators, for the tests: the
checkpoint format, GroupNorm+SiLU with its derivative, the conv weight gradient
and the token norm around a block with its derivative."""
import numpy as np


def e4m3_values():
    """The 128 magnitudes of e4m3 by code (code 127 is NaN)."""
    v = np.empty(128)
    for code in range(128):
        e, f = code >> 3, code & 7
        v[code] = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
    v[127] = np.nan
    return v


E4M3 = e4m3_values()


def round_e4m3(t):
    """Nearest e4m3 code of |t| <= 448, ties to the even code."""
    mag = np.abs(t)
    hi = np.searchsorted(E4M3[:127], mag)          # first value >= mag
    hi = np.minimum(hi, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = mag - E4M3[lo], E4M3[hi] - mag
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return code + np.where(np.signbit(t), 128, 0)


def quantise(rows):
    """float rows [r, c] -> (codes [r, cp] uint8, scale bytes [r, cp/32] uint8)."""
    rows = np.asarray(rows, dtype=np.float64)
    r, c = rows.shape
    cp = -(-c // 32) * 32
    b = np.zeros((r, cp))
    b[:, :c] = rows
    b = b.reshape(r, cp // 32, 32)
    codes = np.empty(b.shape, dtype=np.uint8)
    scale = np.empty(b.shape[:2], dtype=np.uint8)
    for i in np.ndindex(*scale.shape):
        blk = b[i]
        if not np.isfinite(blk).all():
            scale[i] = 255
            codes[i] = 127
            continue
        top, e = np.abs(blk).max(), -127
        while top > 448 * 2.0 ** e:
            e += 1
        scale[i] = e + 127
        codes[i] = round_e4m3(blk * 2.0 ** -e)
    return codes.reshape(r, cp), scale


def dequantise(codes, scale, c):
    r, cp = codes.shape
    v = E4M3[codes & 127] * np.where(codes & 128, -1.0, 1.0)
    s = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127))
    return (v.reshape(r, cp // 32, 32) * s[:, :, None]).reshape(r, cp)[:, :c]


# ---------------------------------------------------------------- GroupNorm + SiLU
def group_stats(x, groups, eps):
    """x [n, p, c] -> mean, rstd [n, groups]."""
    n, p, c = x.shape
    g = x.reshape(n, p, groups, c // groups)
    mean = g.mean((1, 3))
    var = ((g - mean[:, None, :, None]) ** 2).mean((1, 3))
    return mean, 1 / np.sqrt(var + eps)


def gn_forward(x, groups, eps, gamma, beta, silu):
    n, p, c = x.shape
    mean, rstd = group_stats(x, groups, eps)
    per = lambda a: np.repeat(a, c // groups, 1)[:, None, :]  # noqa: E731
    z = (x - per(mean)) * per(rstd) * gamma + beta
    return z / (1 + np.exp(-z)) if silu else z


def gn_backward(dy, x, mean, rstd, groups, gamma, beta, silu):
    n, p, c = x.shape
    per = lambda a: np.repeat(a, c // groups, 1)[:, None, :]  # noqa: E731
    xh = (x - per(mean)) * per(rstd)
    dz = dy
    if silu:
        z = xh * gamma + beta
        s = 1 / (1 + np.exp(-z))
        dz = dy * s * (1 + z * (1 - s))
    t = dz * gamma
    gm = lambda a: per(a.reshape(n, p, groups, -1).mean((1, 3)))  # noqa: E731
    dx = per(rstd) * (t - gm(t) - xh * gm(t * xh))
    return dx, (dz * xh).sum((0, 1)), dz.sum((0, 1))


# ---------------------------------------------------------------- conv weight gradient
def wgrad(dy, x, k):
    """dy [n, h, w, o], x [n, h, w, c] -> dw [o, c, k, k], dbias [o]."""
    n, h, w, _ = dy.shape
    p = k // 2
    xp = np.pad(x, ((0, 0), (p, p), (p, p), (0, 0)))
    dw = np.zeros((dy.shape[3], x.shape[3], k, k))
    for ky in range(k):
        for kx in range(k):
            dw[:, :, ky, kx] = np.tensordot(dy, xp[:, ky:ky + h, kx:kx + w], ((0, 1, 2),) * 2)
    return dw, dy.sum((0, 1, 2))


# ---------------------------------------------------------------- block norm
def block_norm(u, x, eps, w_post, gate, scale, w_pre):
    """u, x [n, t, c] -> h, y, m, r."""
    f = (1.0 if gate is None else gate[:, None, :]) * (1.0 if scale is None else scale)
    m = 1 / np.sqrt((u * u).mean(-1) + eps)
    h = x + f * w_post * u * m[..., None]
    r = 1 / np.sqrt((h * h).mean(-1) + eps)
    return h, None if w_pre is None else w_pre * h * r[..., None], m, r


def block_norm_backward(dy, dh, u, h, m, r, w_post, gate, scale, w_pre):
    g = np.ones((u.shape[0], u.shape[2])) if gate is None else gate
    sc = np.ones(u.shape[2]) if scale is None else scale
    uh = u * m[..., None]
    dx = np.zeros_like(u) if dh is None else dh.copy()
    out = {}
    if w_pre is not None:
        hh = h * r[..., None]
        t = w_pre * dy
        dx = dx + r[..., None] * (t - hh * (hh * t).mean(-1, keepdims=True))
        out["dw_pre"] = (dy * hh).sum((0, 1))
    t = dx * g[:, None, :] * sc * w_post
    out["dx"] = dx
    out["du"] = m[..., None] * (t - uh * (uh * t).mean(-1, keepdims=True))
    s = (dx * uh).sum(1)
    out["dw_post"] = (g * sc * s).sum(0)
    if gate is not None:
        out["dgate"] = sc * w_post * s
    if scale is not None:
        out["dscale"] = (g * w_post * s).sum(0)
    return out
