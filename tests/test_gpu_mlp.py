"""GPU tests of the MLP operators against float64 forms. Tolerances count roundings:
one of the output's type (finfo.eps / 2), and 2^-24 for each FP32 one before it."""
import numpy as np
import pytest
import torch

import _mlp_ref as R

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DTYPES = list(R.DTYPES)
EPS = 1e-6


@pytest.fixture(scope="module")
def vae():
    import diffusion_vae_decoder_gb300 as pkg
    pkg.load_library()
    return pkg


def rand(seed, *shape, dtype=torch.float32, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def ints(seed, *shape, dtype, top):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda").to(dtype)


def guarded(shape, dtype):
    """(tensor of `shape`, check): a piece of a larger buffer, and a function that
    fails when what lies around it was written."""
    count = int(np.prod(shape))
    buf = torch.full((count + 512,), 3.0, dtype=dtype, device="cuda")
    out = buf[256:256 + count].view(shape)
    out.fill_(float("nan"))

    def check():
        assert (buf[:256] == 3).all() and (buf[256 + count:] == 3).all()
        assert not torch.isnan(out).any()
    return out, check


def close(got, ref, tol, what=""):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    if bad.any():
        i = torch.where(bad, err / (tol + 1e-300), torch.zeros_like(err)).flatten().argmax()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, worst at {int(i)}: "
                             f"{got.flatten()[i].item()} for {ref.flatten()[i].item()}, "
                             f"tolerance {(tol + 0 * err).flatten()[i].item():.3e}")


# ---------------------------------------------------------------- layer norm
NORM_SIZES = [(1, 4), (1, 512), (3, 36), (7, 64), (500, 68), (61, 128), (129, 256), (1221, 700), (300, 1024),
              (65, 2048), (33, 4096), (2, 4100), (9, 8192)]
# A row's sum passes at most 8 x 2 additions in a thread, 1 of a pair, 5 of a warp and
# 16 of a block: 38 roundings of partial sums, each below the sum of the magnitudes.
SUM = 38


def norm_tolerance(x, gamma, beta, mean, rstd, y, dtype):
    top = x.abs().amax(-1, keepdim=True)
    xh = (x - mean) * rstd
    # the mean is off by SUM + 2 roundings of the largest |x|, rstd by half of those of
    # the squares' sum and five of its own; five more in the last products
    return (R.rounding(dtype, y) +
            U * (gamma.abs() * ((SUM + 2) * top * rstd + (SUM / 2 + 10) * xh.abs()) + 2 * y.abs()
                 + (0 if beta is None else beta.abs())))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,c", NORM_SIZES)
def test_layer_norm(vae, rows, c, dtype):
    t = R.DTYPES[dtype]
    x = rand(rows + c, rows, c, dtype=t, std=2.0, mean=0.7)
    gamma = rand(1, c, std=0.2, mean=1.0)
    beta = rand(2, c, std=0.2) if rows % 2 else None
    out, check = guarded((rows, c), t)
    y, stats = vae.vae_layer_norm(x, gamma, beta, eps=EPS, out=out)
    check()
    ref, mean, rstd = R.layer_norm(x.double(), gamma.double(),
                                   None if beta is None else beta.double(), EPS)
    close(y, ref, norm_tolerance(x.double(), gamma, beta, mean, rstd, ref, t), "y")
    close(stats[:, :1], mean, U * (SUM + 2) * x.double().abs().amax(-1, keepdim=True), "mean")
    close(stats[:, 1:], rstd, U * rstd * (SUM / 2 + 8 + 2 * SUM * U), "rstd")
    # in place, and without the statistics
    z = x.clone()
    again, none = vae.vae_layer_norm(z, gamma, beta, eps=EPS, keep=False, out=z)
    assert none is None and again is z
    assert torch.equal(z, y)


def test_layer_norm_of_far_means_and_constant_rows(vae):
    x = rand(5, 64, 512, mean=1000.0)
    x[3] = 0.1
    x[4] = 0.0
    gamma, beta = rand(1, 512, std=0.2, mean=1.0), rand(2, 512, std=0.2)
    y, _ = vae.vae_layer_norm(x, gamma, beta, eps=EPS)
    ref, mean, rstd = R.layer_norm(x.double(), gamma.double(), beta.double(), EPS)
    close(y, ref, norm_tolerance(x.double(), gamma, beta, mean, rstd, ref, x.dtype))
    assert torch.equal(y[4], beta)


def test_layer_norm_keeps_bad_rows_apart(vae):
    for c in (64, 1024):
        x = rand(6, 40, c)
        gamma = rand(1, c, std=0.2, mean=1.0)
        want, _ = vae.vae_layer_norm(x, gamma)
        x[7, 3], x[21, c - 1], x[39, 0] = float("nan"), float("inf"), -float("inf")
        y, _ = vae.vae_layer_norm(x, gamma)
        bad = torch.zeros(40, dtype=torch.bool, device="cuda")
        bad[[7, 21, 39]] = True
        assert torch.isnan(y[bad]).all()
        assert torch.equal(y[~bad], want[~bad])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,c", NORM_SIZES + [(2048, 512), (2049, 512), (5000, 32), (2500, 1024)])
def test_layer_norm_backward(vae, rows, c, dtype):
    t = R.DTYPES[dtype]
    x = rand(rows + c, rows, c, dtype=t, std=2.0, mean=0.7)
    dy = rand(rows + c + 1, rows, c, dtype=t, std=0.1)
    dres = rand(rows + c + 2, rows, c, dtype=t, std=0.1) if rows % 2 else None
    gamma = rand(1, c, std=0.2, mean=1.0)
    stats = vae.vae_layer_norm(x, gamma, eps=EPS)[1]
    out, check = guarded((rows, c), t)
    dx, dgamma, dbeta = vae.vae_layer_norm_backward(dy, x, stats, gamma, dres=dres, out=out)
    check()
    mean, rstd = stats.double()[:, :1], stats.double()[:, 1:]
    x64, dy64, g64 = x.double(), dy.double(), gamma.double()
    ref, rg, rb = R.layer_norm_backward(dy64, x64, mean, rstd, g64,
                                        None if dres is None else dres.double())
    xh, tt = (x64 - mean) * rstd, dy64 * g64
    m1, m2 = tt.abs().mean(-1, keepdim=True), (tt * xh).abs().mean(-1, keepdim=True)
    # xh two roundings, t one, the two means SUM + 4 each, six in the last products
    tol = (R.rounding(t, ref) + U * rstd.abs() *
           (6 * tt.abs() + (SUM + 6) * m1 + xh.abs() * (SUM + 12) * m2) +
           U * (2 * ref.abs() + (0 if dres is None else dres.double().abs())))
    close(dx, ref, tol, "dx")
    # a column: rows / blocks numbers in a thread, then at most 32 + 10 + 5 sums; few
    # rows: rows / 32 in a thread, then 64 threads
    chain = max(rows / 304 * max(1, 256 * 8 / c) + 64, rows / 32 + 64)
    close(dgamma, rg, U * (chain + 4) * (dy64 * xh).abs().sum(0), "dgamma")
    close(dbeta, rb, U * chain * dy64.abs().sum(0), "dbeta")
    # dx over dy, and over dres
    over = dy.clone()
    vae.vae_layer_norm_backward(over, x, stats, gamma, dres=dres, out=over)
    assert torch.equal(over, dx)
    if dres is not None:
        over = dres.clone()
        vae.vae_layer_norm_backward(dy, x, stats, gamma, dres=over, out=over)
        assert torch.equal(over, dx)


def test_layer_norm_backward_against_differences(vae):
    rows, c, h = 5, 36, 1e-6
    x, dy = rand(1, rows, c).double(), rand(2, rows, c)
    gamma, beta = rand(3, c, std=0.2, mean=1.0), rand(4, c)
    stats = vae.vae_layer_norm(x.float(), gamma, beta)[1]
    dx, dgamma, dbeta = vae.vae_layer_norm_backward(dy, x.float(), stats, gamma)

    def value(x, gamma, beta):
        return (R.layer_norm(x, gamma, beta, EPS)[0] * dy.double()).sum()

    g64, b64 = gamma.double(), beta.double()
    for i in range(0, rows * c, 7):
        d = torch.zeros_like(x).view(-1)
        d[i] = h
        d = d.view_as(x)
        want = (value(x + d, g64, b64) - value(x - d, g64, b64)) / (2 * h)
        assert abs(dx.view(-1)[i].double() - want) < 1e-4  # h^2 and 2^-53 / h are below 1e-8
    for i in range(c):
        d = torch.zeros_like(g64)
        d[i] = h
        assert abs(dgamma[i] - (value(x, g64 + d, b64) - value(x, g64 - d, b64)) / (2 * h)) < 1e-4
        assert abs(dbeta[i] - (value(x, g64, b64 + d) - value(x, g64, b64 - d)) / (2 * h)) < 1e-4


# ---------------------------------------------------------------- dropout
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("count,p", [(1, 0.5), (7, 0.5), (8, 0.1), (9, 0.1), (1000, 0.0),
                                     (1003, 1.0), (135173, 0.3), (2 ** 20 + 4, 0.1)])
def test_dropout(vae, count, p, residual, dtype):
    t = R.DTYPES[dtype]
    seed, offset = 0xFEDCBA9876543210, 2 ** 32 - 3
    x = rand(count, count, dtype=t)
    x[x == 0] = 1
    r = rand(count + 1, count, dtype=t, std=2.0) if residual else None
    out, check = guarded((count,), t)
    y = vae.vae_dropout(x, p, seed=seed, offset=offset, residual=r, out=out)
    check()
    keep = torch.from_numpy(R.kept(count, p, seed, offset)).cuda()
    q = R.threshold(p)
    kept = x.double() * (65536 / (65536 - q) if q < 65536 else 0)
    ref = torch.where(keep, kept, torch.zeros_like(kept))
    if residual:
        ref = ref + r.double()
        assert torch.equal(y[~keep], r[~keep])
    else:
        assert torch.equal(y != 0, keep)
    # the scale and the sum are rounded in FP32
    close(y, ref, R.rounding(t, ref) + U * (kept.abs() + ref.abs()))
    # over its input, and over the residual
    over = x.clone()
    vae.vae_dropout(over, p, seed=seed, offset=offset, residual=r, out=over)
    assert torch.equal(over, y)
    if residual:
        over = r.clone()
        vae.vae_dropout(x, p, seed=seed, offset=offset, residual=over, out=over)
        assert torch.equal(over, y)


def test_dropout_backward_is_the_same_mask(vae):
    x, dy = rand(1, 100, 48), rand(2, 100, 48)
    ones = vae.vae_dropout(torch.ones_like(x), 0.4, seed=9, offset=5)
    assert torch.equal(vae.vae_dropout(dy, 0.4, seed=9, offset=5), dy * ones)
    other = vae.vae_dropout(torch.ones_like(x), 0.4, seed=9, offset=5 + 100 * 48 // 8)
    both = ((ones == 0) & (other == 0)).double().mean().item()
    assert abs(both - 0.16) < 6 * (0.16 * 0.84 / 4800) ** 0.5  # independent


def test_dropout_of_bad_numbers_and_of_unaligned_views(vae):
    x = torch.full((1, 4096), float("nan"), device="cuda")
    y = vae.vae_dropout(x, 0.5, seed=3)
    keep = torch.from_numpy(R.kept(4096, 0.5, 3, 0)).cuda().view(1, -1)
    assert (y[~keep] == 0).all() and torch.isnan(y[keep]).all()
    for t in R.DTYPES.values():
        base = rand(4, 1000, dtype=t)
        step = 16 // base.element_size()
        v = base[step:step + 805]
        assert torch.equal(vae.vae_dropout(v, 0.3, seed=1), vae.vae_dropout(v.clone(), 0.3, seed=1))
        with pytest.raises(vae.VaeError):
            vae.vae_dropout(base[1:9], 0.3, seed=1)


def test_dropout_state_moves_between_replays(vae):
    x = torch.ones(1000, 24, device="cuda")
    state = torch.tensor([77, 0], dtype=torch.int64, device="cuda")
    out = torch.empty_like(x)
    vae.vae_dropout(x, 0.3, state=state, offset=40, out=out)
    assert torch.equal(out, vae.vae_dropout(x, 0.3, seed=77, offset=40))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        vae.vae_dropout(x, 0.3, state=state, offset=40, out=out)
        state[1] += 3000
    for i in range(3):
        g.replay()
        assert torch.equal(out, vae.vae_dropout(x, 0.3, seed=77, offset=40 + 3000 * i))
    state.copy_(torch.tensor([-1, -1]))  # all ones: 2^64 - 1, and offset 39
    g.replay()
    assert torch.equal(out, vae.vae_dropout(x, 0.3, seed=2 ** 64 - 1, offset=39))


# ---------------------------------------------------------------- linear: exact integers
# Small integers make every product and sum exact, and every result a number of the
# type: the operators have to agree to the last bit at every size.
LINEAR_SIZES = [(1, 8, 8), (1, 264, 512), (2, 512, 264), (3, 2048, 128), (5, 64, 40), (8, 72, 1000),
                (9, 520, 72), (127, 128, 128), (128, 136, 64), (129, 264, 200), (257, 120, 520),
                (1000, 1032, 72), (300, 512, 2056), (4575, 256, 128), (2049, 2048, 520),
                (1000, 2056, 2048), (4100, 1032, 2048), (8, 4096, 2048), (7, 4104, 2048)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n,k", LINEAR_SIZES)
def test_linear_exact(vae, rows, n, k, dtype):
    t = R.DTYPES[dtype]
    # sums of k numbers up to 1: |z| <= 2^8 for bf16 with sparse weights
    x, w = ints(rows, rows, k, dtype=t, top=1), ints(n, n, k, dtype=t, top=1)
    if dtype == "bf16":
        w *= (torch.arange(k, device="cuda") % max(1, k // 64) == 0).to(t)
    bias = ints(1, n, dtype=torch.float32, top=3)
    res = ints(2, rows, n, dtype=t, top=9)
    z = x.double() @ w.double().t() + bias.double()
    assert z.abs().max() + 9 <= (256 if dtype == "bf16" else 2048)
    out, check = guarded((rows, n), t)
    y, kept = vae.vae_linear(x, w, bias=bias, residual=res, keep=True, out=out)
    check()
    assert torch.equal(kept.double(), z)
    assert torch.equal(y.double(), z + res.double())
    y, kept = vae.vae_linear(x, w)
    assert kept is None and torch.equal(y.double(), z - bias.double())
    vae.vae_linear(x, w, bias=bias, residual=res, out=res)
    assert torch.equal(res, out)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n,k", LINEAR_SIZES)
def test_linear_dgrad_exact(vae, rows, n, k, dtype):
    t = R.DTYPES[dtype]
    dy, w = ints(rows, rows, n, dtype=t, top=1), ints(n, n, k, dtype=t, top=1)
    if dtype == "bf16":
        dy *= (torch.arange(n, device="cuda") % max(1, n // 64) == 0).to(t)
    ref = dy.double() @ w.double()
    assert ref.abs().max() <= (256 if dtype == "bf16" else 2048)
    out, check = guarded((rows, k), t)
    vae.vae_linear_dgrad(dy, w, out=out)
    check()
    assert torch.equal(out.double(), ref)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n,k", LINEAR_SIZES)
def test_linear_wgrad_exact(vae, rows, n, k, dtype):
    t = R.DTYPES[dtype]
    dy, x = ints(rows, rows, n, dtype=t, top=4), ints(n, rows, k, dtype=t, top=4)
    dw, db = vae.vae_linear_wgrad(dy, x)
    assert dw.dtype == db.dtype == torch.float32
    assert torch.equal(dw.double(), dy.double().t() @ x.double())
    assert torch.equal(db.double(), dy.double().sum(0))
    again, none = vae.vae_linear_wgrad(dy, x, bias=False)
    assert none is None and torch.equal(again, dw)


@pytest.mark.parametrize("rows,n,k", [(3, 264, 512), (300, 264, 512), (2500, 2048, 256)])
def test_linear_of_subnormal_halves(vae, rows, n, k):
    """f16 numbers below the smallest normal one, as gradients are, lose nothing."""
    tiny = 2.0 ** -24  # the smallest f16
    x = (ints(1, rows, k, dtype=torch.float32, top=9) * tiny).half()
    w = ints(2, n, k, dtype=torch.float16, top=2)
    z = x.double() @ w.double().t()
    assert (z.abs() < 2.0 ** -13).all()  # (exact in f16)
    assert torch.equal(vae.vae_linear(x, w)[0].double(), z)
    dw, db = vae.vae_linear_wgrad(x, w[:1].expand(rows, k).contiguous())
    assert torch.equal(dw.double(), x.double().t() @ w[:1].double().expand(rows, k))
    assert torch.equal(db.double(), x.double().sum(0))


@pytest.mark.parametrize("rows,n,k", [(3, 264, 512), (300, 264, 512), (2500, 2048, 256)])
def test_float_products_scale_with_powers_of_two(vae, rows, n, k):
    """All three parts of a float keep their numbers over float's range."""
    x, w = rand(1, rows, k), rand(2, n, k, std=k ** -0.5)
    want, _ = vae.vae_linear(x, w)
    for e in (-80, 90):
        got, _ = vae.vae_linear(x * 2.0 ** e, w)
        assert torch.equal(got, want * 2.0 ** e)


# ---------------------------------------------------------------- linear: numbers
# The tensor core cuts its running sum once every 16 products, by at most 2^-22 of it
# (2^-23 where the products are aligned and 2^-23 where they are added); a float's sum
# leaves it every 32 steps and is rounded there. Floats' left-out products are 2^-24.
def sum_tolerance(k, magnitude, exact16, to_float):
    steps = -(-k // 16)
    if exact16 and not to_float:
        return magnitude * steps * 2.0 ** -22
    chains = -(-steps * (1 if exact16 else 6) // 32) + 8
    return magnitude * (2 * U + min(32, 6 * steps) * 2.0 ** -22 + chains * U)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("rows,n,k", [(1, 512, 264), (6, 72, 2048), (200, 136, 520),
                                      (700, 1024, 512), (2305, 2048, 256)])
def test_linear(vae, rows, n, k, act, dtype):
    t = R.DTYPES[dtype]
    x, w = rand(1, rows, k, dtype=t, std=2.0), rand(2, n, k, dtype=t, std=k ** -0.5)
    bias, res = rand(3, n), rand(4, rows, n, dtype=t)
    code = {"none": vae.VAE_ACT_NONE, "silu": vae.VAE_ACT_SILU, "gelu": vae.VAE_ACT_GELU}[act]
    y, z = vae.vae_linear(x, w, bias=bias, act=code, residual=res, keep=True)
    z64 = x.double() @ w.double().t() + bias.double()
    tol = sum_tolerance(k, x.double().abs() @ w.double().abs().t() + bias.double().abs(),
                        t != torch.float32, t == torch.float32) + 2 * U * z64.abs()
    close(z, z64, tol + R.rounding(t, z64), "z")
    a = R.activation(z64, act)
    ref = a + res.double()
    # |act'| < 1.2; the sigmoid's exponential and reciprocal: for floats 2^-22 and 4 |v|
    # 2^-24 (v is rounded four times), for 16-bit results 2^-20 and 2^-22 |v|
    v = z64 if act == "none" else R.gate(z64, act)[0]
    rel = (4 * U + 4 * U * v.abs()) if t == torch.float32 else 2.0 ** -20 + 2.0 ** -22 * v.abs()
    out = 1.2 * tol + a.abs() * torch.clamp(rel, max=1.0) + 2 * U * ref.abs()
    close(y, ref, out + R.rounding(t, ref) + 1e-30, "y")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("rows,n,k", [(1, 264, 512), (200, 136, 520), (2294, 264, 520),
                                      (700, 512, 2048), (4100, 264, 2048)])
def test_linear_dgrad(vae, rows, n, k, act, dtype):
    t = R.DTYPES[dtype]
    dy, w = rand(1, rows, n, dtype=t, std=0.1), rand(2, n, k, dtype=t, std=k ** -0.5)
    z = None if act == "none" else rand(3, rows, k, dtype=t, std=3.0)
    code = {"none": vae.VAE_ACT_NONE, "silu": vae.VAE_ACT_SILU, "gelu": vae.VAE_ACT_GELU}[act]
    dx = vae.vae_linear_dgrad(dy, w, z=z, act=code)
    s64 = dy.double() @ w.double()
    sl = torch.ones_like(s64) if z is None else R.slope(z.double(), act)
    tol = sum_tolerance(n, dy.double().abs() @ w.double().abs(), t != torch.float32,
                        t == torch.float32) * sl.abs()
    if z is not None:
        # s + w s (1 - s), w = z v': s as in test_linear, 1 - s = e s with it, e off by
        # 4 |v| 2^-24 and its unit's 2^-22, five more roundings; z is held at -10 (SiLU:
        # -87), where the derivative is 2.8e-36 at most
        v, dv = R.gate(z.double(), act)
        s, far = torch.sigmoid(v), torch.sigmoid(-v)
        w = (z.double() * dv).abs()
        rel = 4 * U if t == torch.float32 else 2.0 ** -20 + 2.0 ** -22 * v.abs().clamp(max=88)
        tol = tol + s64.abs() * (rel * (s + 2 * w * s * far) + U * (8 + 4 * v.abs()) * s * far
                                 * (1 + w) + 8 * U * (s + w * s * far) + 1e-35)
    ref = s64 * sl
    close(dx, ref, tol + R.rounding(t, ref) + 4 * U * ref.abs())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n,k", [(1, 64, 72), (77, 136, 520), (4575, 256, 128),
                                      (20000, 512, 264), (3000, 2048, 2056), (20011, 520, 1032),
                                      (30000, 64, 40)])
def test_linear_wgrad(vae, rows, n, k, dtype):
    t = R.DTYPES[dtype]
    dy, x = rand(1, rows, n, dtype=t, std=0.1), rand(2, rows, k, dtype=t)
    dw, db = vae.vae_linear_wgrad(dy, x)
    ref = dy.double().t() @ x.double()
    close(dw, ref, sum_tolerance(rows, dy.double().abs().t() @ x.double().abs(),
                                 t != torch.float32, True) + U * ref.abs(), "dw")
    close(db, dy.double().sum(0), U * (rows / 8 + 64) * dy.double().abs().sum(0), "dbias")


def test_derivative_at_the_far_ends(vae):
    z = torch.tensor([float("inf"), 1e30, 100.0, 33.0, -33.0, -100.0, -1e30, -float("inf")],
                     device="cuda").view(1, 8)
    dy = torch.zeros(1, 8, device="cuda")
    dy[0, 0] = 1
    w = torch.zeros(8, 8, device="cuda")
    w[0] = 1
    for act in (vae.VAE_ACT_SILU, vae.VAE_ACT_GELU):
        for t in R.DTYPES.values():
            dx = vae.vae_linear_dgrad(dy.to(t), w.to(t), z=z.to(t), act=act)[0]
            assert (dx[:4] == 1).all()
            assert (dx[4:].float().abs() < 1e-12).all()  # (1e-12 is no half)
            bad = vae.vae_linear_dgrad(dy.to(t), w.to(t), z=torch.full_like(z, float("nan")).to(t),
                                       act=act)
            assert torch.isnan(bad).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", [(2, 64), (200, 64), (2500, 2048)])
def test_activation_at_the_far_ends(vae, rows, n, dtype):
    t = R.DTYPES[dtype]
    top = 6e4 if dtype == "f16" else 1e30
    ends = torch.tensor([top, 3e4, 100.0, -100.0, -3e4, -top, float("inf"), -float("inf")],
                        device="cuda")
    bias = ends.repeat(n // 8)
    x, w = torch.zeros(rows, 64, dtype=t, device="cuda"), rand(1, n, 64, dtype=t)
    for act in (vae.VAE_ACT_SILU, vae.VAE_ACT_GELU):
        y, z = vae.vae_linear(x, w, bias=bias, act=act, keep=True)
        assert torch.equal(z, bias.to(t).expand(rows, n))
        y = y.view(rows, -1, 8)
        assert torch.equal(y[..., :3], ends[:3].to(t).expand_as(y[..., :3]))
        assert torch.isinf(y[..., 6]).all() and (y[..., 6] > 0).all()
        assert (y[..., [3, 4, 5, 7]].float().abs() < 1e-30).all()


@pytest.mark.parametrize("rows", [4, 300])
@pytest.mark.parametrize("dtype", DTYPES)
def test_bad_numbers_stay_in_their_row_and_column(vae, rows, dtype):
    t = R.DTYPES[dtype]
    x, w = rand(1, rows, 136, dtype=t), rand(2, 264, 136, dtype=t)
    want, _ = vae.vae_linear(x, w)
    x[2, 5] = float("nan")
    w[100, 9] = float("inf")
    got, _ = vae.vae_linear(x, w)
    assert torch.isnan(got[2]).all()
    assert not torch.isfinite(got[:, 100]).any()
    got[2], got[:, 100] = want[2], want[:, 100]
    assert torch.equal(got, want)


def same_bad_numbers(got, ref, want, rows=(), cols=()):
    """Infinities and NaN are float64's; everything outside the rows and columns that they
    reach is `want`, and so is what they leave finite in them."""
    bad = ~torch.isfinite(ref)
    assert torch.equal(~torch.isfinite(got), bad)
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    inf = torch.isinf(ref)
    assert torch.equal(got[inf].double(), ref[inf])
    clean = torch.ones_like(bad)
    clean[list(rows)] = False
    clean[:, list(cols)] = False
    assert not bad[clean].any() and torch.equal(got[clean], want[clean])


def spoil(a, b):
    """Infinities of either sign in a row of a, alone, together and on b's zero, infinity
    and smallest numbers; infinities and a NaN in rows of b. (rows of a, of b) reached."""
    inf = float("inf")
    a[1, 5], a[2, 5], a[3, 7], a[3, 8] = inf, -inf, inf, inf
    b[17, 9], b[7, 5], b[33, 11] = -inf, inf, float("nan")
    b[20, 5], b[21, 5], b[22, 5] = 0.0, 1e-45, -1e-42
    return (1, 2, 3), (17, 7, 33, 20, 21, 22)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n,k", [(4, 264, 136), (8, 264, 136), (9, 264, 136), (300, 264, 136),
                                      (2500, 2048, 512)])
def test_bad_numbers_are_those_of_float(vae, rows, n, k, dtype):
    """The same infinities and NaN whichever kernel the number of rows takes."""
    t = R.DTYPES[dtype]
    x, w = rand(1, rows, k, dtype=t), rand(2, n, k, dtype=t)
    dy, wt = rand(3, rows, k, dtype=t), rand(4, k, n, dtype=t)
    want, back = vae.vae_linear(x, w)[0], vae.vae_linear_dgrad(dy, wt)
    ra, rb = spoil(x, w)
    same_bad_numbers(vae.vae_linear(x, w)[0], x.double() @ w.double().t(), want, ra, rb)
    ra, rb = spoil(dy, wt.t())
    same_bad_numbers(vae.vae_linear_dgrad(dy, wt), dy.double() @ wt.double(), back, ra, rb)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n,k", [(40, 64, 72), (4575, 256, 128), (8192, 2048, 512)])
def test_bad_numbers_of_the_weights_gradient(vae, rows, n, k, dtype):
    t = R.DTYPES[dtype]
    dy, x = rand(1, rows, n, dtype=t), rand(2, rows, k, dtype=t)
    want, sums = vae.vae_linear_wgrad(dy, x)
    ra, rb = spoil(dy.t(), x.t())
    dw, db = vae.vae_linear_wgrad(dy, x)
    same_bad_numbers(dw, dy.double().t() @ x.double(), want, ra, rb)
    same_bad_numbers(db.view(-1, 1), dy.double().sum(0).view(-1, 1), sums.view(-1, 1), ra)


@pytest.mark.parametrize("dtype", DTYPES)
def test_arrays_next_to_one_another(vae, dtype):
    """Inputs and outputs cut from one buffer without a gap are taken; shifted ones not."""
    t = R.DTYPES[dtype]
    rows, c = 40, 64
    buf = rand(1, 5 * rows, c, dtype=t)
    x, w, r, y, more = buf.split(rows)
    w = rand(2, c, c, dtype=t)
    gamma = rand(3, c, std=0.2, mean=1.0)
    want = vae.vae_linear(x.clone(), w, residual=r.clone())[0]
    assert torch.equal(vae.vae_linear(x, w, residual=r, out=y)[0], want)
    stats = vae.vae_layer_norm(x.clone(), gamma)[1]
    want = vae.vae_layer_norm_backward(y.clone(), x.clone(), stats, gamma, dres=r.clone())[0]
    assert torch.equal(vae.vae_layer_norm_backward(y, x, stats, gamma, dres=r, out=more)[0], want)
    want = vae.vae_linear_dgrad(x.clone(), w, z=r.clone(), act=vae.VAE_ACT_SILU)
    assert torch.equal(vae.vae_linear_dgrad(x, w, z=r, act=vae.VAE_ACT_SILU, out=y), want)
    want = vae.vae_linear_dgrad(x, w, z=r.clone(), act=vae.VAE_ACT_SILU)
    over = r.clone()  # the derivative's numbers, written over
    assert torch.equal(vae.vae_linear_dgrad(x, w, z=over, act=vae.VAE_ACT_SILU, out=over), want)
    before, shifted = buf.clone(), buf[8:8 + rows]
    for call in (lambda: vae.vae_linear(x, w, out=shifted),
                 lambda: vae.vae_linear(y, w, residual=x, out=shifted),
                 lambda: vae.vae_layer_norm(x, gamma, out=shifted),
                 lambda: vae.vae_layer_norm_backward(y, more, stats, gamma, dres=x, out=shifted),
                 lambda: vae.vae_dropout(x, 0.1, seed=1, out=shifted),
                 lambda: vae.vae_linear_dgrad(y, w, z=x, act=vae.VAE_ACT_SILU, out=shifted)):
        with pytest.raises(vae.VaeError):
            call()
    assert torch.equal(buf, before)


# ---------------------------------------------------------------- all of them
def mlp_ref(x, gamma, beta, w1, b1, w2, b2, keep, scale):
    """float64 MLP block with autograd."""
    h = torch.nn.functional.layer_norm(x, x.shape[-1:], gamma, beta, EPS)
    z = h @ w1.t() + b1
    u = R.activation(z, "gelu") @ w2.t() + b2
    return x + keep * scale * u


class Mlp:
    """x + dropout(linear(gelu(linear(norm(x))))) and its gradients, as a user writes it."""

    def __init__(self, vae, c, hidden, dtype, p):
        self.vae, self.p, self.seed, self.offset = vae, p, 1234, 2 ** 33 + 5
        self.gamma, self.beta = rand(1, c, std=0.2, mean=1.0), rand(2, c, std=0.2)
        self.w1 = rand(3, hidden, c, dtype=dtype, std=c ** -0.5)
        self.w2 = rand(4, c, hidden, dtype=dtype, std=hidden ** -0.5)
        self.b1, self.b2 = rand(5, hidden, std=0.1), rand(6, c, std=0.1)

    def forward(self, x):
        v = self.vae
        self.x = x
        self.h, self.stats = v.vae_layer_norm(x, self.gamma, self.beta, eps=EPS)
        self.a, self.z = v.vae_linear(self.h, self.w1, bias=self.b1, act=v.VAE_ACT_GELU, keep=True)
        u, _ = v.vae_linear(self.a, self.w2, bias=self.b2)
        return v.vae_dropout(u, self.p, seed=self.seed, offset=self.offset, residual=x)

    def backward(self, dy):
        v = self.vae
        du = v.vae_dropout(dy, self.p, seed=self.seed, offset=self.offset)
        dw2, db2 = v.vae_linear_wgrad(du, self.a)
        dz = v.vae_linear_dgrad(du, self.w2, z=self.z, act=v.VAE_ACT_GELU)
        dw1, db1 = v.vae_linear_wgrad(dz, self.h)
        dh = v.vae_linear_dgrad(dz, self.w1)
        dx, dgamma, dbeta = v.vae_layer_norm_backward(dh, self.x, self.stats, self.gamma, dres=dy)
        return dict(dx=dx, dgamma=dgamma, dbeta=dbeta, dw1=dw1, db1=db1, dw2=dw2, db2=db2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,tokens,c", [(1, 1, 64), (2, 333, 136), (1, 1024, 512)])
def test_mlp_block(vae, n, tokens, c, dtype):
    t = R.DTYPES[dtype]
    m = Mlp(vae, c, 4 * c, t, 0.25)
    x, dy = rand(8, n, tokens, c, dtype=t), rand(9, n, tokens, c, dtype=t, std=0.1)
    y, grads = m.forward(x), None
    grads = m.backward(dy)
    leaves = [a.double().requires_grad_() for a in (x, m.gamma, m.beta, m.w1, m.b1, m.w2, m.b2)]
    keep = torch.from_numpy(R.kept(x.numel(), 0.25, m.seed, m.offset)).cuda().view(x.shape)
    ref = mlp_ref(*leaves, keep.double(), 1 / 0.75)
    want = torch.autograd.grad(ref, leaves, dy.double())
    # every tensor between two operators is rounded once to t: six of them on the
    # longest way, each off by half a step at most
    bound = 6 * R.half_step(t) + 2e-6

    def off(a, b):
        return ((a.double() - b).norm() / b.norm()).item()
    assert off(y, ref.detach()) < bound
    for (name, g), r in zip(
            [(k, grads[k]) for k in ("dx", "dgamma", "dbeta", "dw1", "db1", "dw2", "db2")], want):
        assert g.shape == r.shape
        assert off(g, r) < bound, name
    # the same bits again, and from a captured graph on other numbers
    again = m.backward(dy)
    assert all(torch.equal(again[k], grads[k]) for k in grads)
    sx, sdy = x.clone(), dy.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sy = m.forward(sx)
        sg = m.backward(sdy)
    sx.copy_(rand(18, n, tokens, c, dtype=t))
    sdy.copy_(rand(19, n, tokens, c, dtype=t, std=0.1))
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    ey = m.forward(sx.clone())
    eg = m.backward(sdy.clone())
    assert torch.equal(sy, ey) and all(torch.equal(sg[k], eg[k]) for k in eg)


def test_two_streams_at_once(vae):
    t = torch.float32  # (its products use the workspace)
    a, b = Mlp(vae, 264, 520, t, 0.1), Mlp(vae, 136, 1032, t, 0.1)
    xa, xb = rand(1, 700, 264), rand(2, 900, 136)
    want = [m.backward(m.forward(x)) for m, x in ((a, xa), (b, xb))]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            ga = a.backward(a.forward(xa))
        with torch.cuda.stream(s2):
            gb = b.backward(b.forward(xb))
        torch.cuda.synchronize()
        for got, ref in ((ga, want[0]), (gb, want[1])):
            assert all(torch.equal(got[k], ref[k]) for k in ref)
    # each call handed a stream
    y, _ = vae.vae_linear(xa, a.w1, bias=a.b1, stream=s1)
    dw, db = vae.vae_linear_wgrad(y, xa, stream=s1)
    s1.synchronize()
    y2, _ = vae.vae_linear(xa, a.w1, bias=a.b1)
    dw2, db2 = vae.vae_linear_wgrad(y2, xa)
    assert torch.equal(y, y2) and torch.equal(dw, dw2) and torch.equal(db, db2)


def test_next_to_the_decoders_kernels(vae):
    """Products on one stream while convs and a weight gradient, which take tensor memory
    as well, run on another."""
    x, w = rand(1, 3000, 512, dtype=torch.bfloat16), rand(2, 2048, 512, dtype=torch.bfloat16)
    xf, wf = rand(3, 700, 264), rand(4, 520, 264)
    img, cw = rand(5, 1, 64, 64, 128), rand(6, 128, 128, 3, 3, std=0.03)
    dy = rand(7, 1, 64, 64, 128, std=0.01)
    ckpt = vae.vae_ckpt_pack(img)

    def mine():
        y, z = vae.vae_linear(x, w, act=vae.VAE_ACT_GELU, keep=True)
        return y, z, *vae.vae_linear_wgrad(y, x), vae.vae_linear(xf, wf)[0]

    def others():
        return vae.vae_conv2d(img, cw, layout=vae.VAE_NHWC), *vae.vae_conv2d_wgrad(
            dy, ckpt, 3, layout=vae.VAE_NHWC)

    want = mine(), others()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            a = [mine() for _ in range(3)][-1]
        with torch.cuda.stream(s2):
            b = [others() for _ in range(3)][-1]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a, want[0]))
        assert all(torch.equal(p, q) for p, q in zip(b, want[1]))
    assert vae.vae_device_error() == 0


def test_beyond_32_bit_offsets(vae):
    """More than 2^31 elements: the last rows are right, and so are the first."""
    t = torch.bfloat16
    rows, c = 2 ** 31 // 4096 + 300, 4096
    x = torch.empty(rows, c, dtype=t, device="cuda").normal_()
    gamma = rand(1, c, std=0.2, mean=1.0)
    y, stats = vae.vae_layer_norm(x, gamma)
    ends = torch.cat([torch.arange(5), torch.arange(rows - 5, rows)]).cuda()
    want, wst = vae.vae_layer_norm(x[ends].contiguous(), gamma)
    assert torch.equal(y[ends], want) and torch.equal(stats[ends], wst)
    dx, _, _ = vae.vae_layer_norm_backward(y, x, stats, gamma)
    part, _, _ = vae.vae_layer_norm_backward(want, x[ends].contiguous(), wst, gamma)
    assert torch.equal(dx[ends], part)
    vae.vae_dropout(x, 0.5, seed=3, offset=7, out=dx)
    tail = vae.vae_dropout(x[rows - 5:].contiguous(), 0.5, seed=3, offset=7 + (rows - 5) * c // 8)
    assert torch.equal(dx[rows - 5:], tail)
    # a layer from c to 64 numbers and back
    w = rand(2, 64, c, dtype=t, std=c ** -0.5)
    z, _ = vae.vae_linear(x, w)
    some = torch.cat([torch.arange(200), torch.arange(rows - 200, rows)]).cuda()
    ref = x[some].double() @ w.double().t()
    tol = sum_tolerance(c, x[some].double().abs() @ w.double().abs().t(), True, False)
    close(z[some], ref, tol + R.rounding(t, ref))
    vae.vae_linear_dgrad(z, w, out=dx)
    ref = z[some].double() @ w.double()
    tol = sum_tolerance(64, z[some].double().abs() @ w.double().abs(), True, False)
    close(dx[some], ref, tol + R.rounding(t, ref))
    dw, db = vae.vae_linear_wgrad(z, x)
    cut = 100000  # the gradient is the sum of two parts'
    d1, b1 = vae.vae_linear_wgrad(z[:cut].contiguous(), x[:cut].contiguous())
    d2, b2 = vae.vae_linear_wgrad(z[cut:].contiguous(), x[cut:].contiguous())
    mag = torch.zeros(64, c, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 65536):
        mag += z[i:i + 65536].double().abs().t() @ x[i:i + 65536].double().abs()
    close(dw, d1.double() + d2.double(), 3 * sum_tolerance(rows, mag, True, True), "dw")


@pytest.mark.parametrize("op", ["linear", "linear_large", "dgrad_large", "wgrad", "wgrad_large"])
def test_waits_that_run_out(vae, op):
    """With a limit of a nanosecond some of the products' waits may give up: the call
    then reports it, and leaves a device on which the next one is right."""
    t = torch.bfloat16
    rows, n, k = (2500, 2048, 512) if "large" in op else (300, 264, 520)
    x, w, dy = rand(1, rows, k, dtype=t), rand(2, n, k, dtype=t), rand(3, rows, n, dtype=t)
    z = rand(4, rows, k, dtype=t)

    def call():
        if op.startswith("linear"):
            return vae.vae_linear(x, w)[0]
        if op.startswith("dgrad"):
            return vae.vae_linear_dgrad(dy, w, z=z, act=vae.VAE_ACT_GELU)
        return torch.cat([v.flatten() for v in vae.vae_linear_wgrad(dy, x)])

    want = call()
    assert vae.vae_device_error() == 0
    vae.vae_debug_set_wait_limit(1)
    try:
        got = call()
        code = vae.vae_device_error()
    finally:
        vae.vae_debug_set_wait_limit(0)
    assert code in (0, -6)
    if code == 0:
        assert torch.equal(got, want)
    assert torch.equal(call(), want)
    assert vae.vae_device_error() == 0


def test_python_refusals(vae):
    t = torch.bfloat16
    x, w, g = rand(1, 8, 64, dtype=t), rand(2, 72, 64, dtype=t), rand(3, 64)
    bad = [
        lambda: vae.vae_layer_norm(x, g.to(t)), lambda: vae.vae_layer_norm(x, g[:60]),
        lambda: vae.vae_layer_norm(x.t(), g), lambda: vae.vae_layer_norm(x.double(), g),
        lambda: vae.vae_layer_norm(x, g, out=x.float()),
        lambda: vae.vae_layer_norm_backward(x, x.float(), rand(1, 8, 2), g),
        lambda: vae.vae_layer_norm_backward(x, x, rand(1, 7, 2), g),
        lambda: vae.vae_layer_norm_backward(x, x, rand(1, 8, 2), g, dres=x.float()),
        lambda: vae.vae_dropout(x, 0.1), lambda: vae.vae_dropout(x, 1.5, seed=1),
        lambda: vae.vae_dropout(x, 0.1, seed=-1), lambda: vae.vae_dropout(x, 0.1, seed=2 ** 64),
        lambda: vae.vae_dropout(x, 0.1, seed=1, state=torch.zeros(2, dtype=torch.int64).cuda()),
        lambda: vae.vae_dropout(x, 0.1, state=torch.zeros(3, dtype=torch.int64).cuda()),
        lambda: vae.vae_dropout(x, 0.1, seed=1, offset=-1),
        lambda: vae.vae_dropout(x, 0.1, seed=1, residual=x.float()),
        lambda: vae.vae_linear(x, w.float()), lambda: vae.vae_linear(x, w[:, :56].contiguous()),
        lambda: vae.vae_linear(x, w, bias=rand(1, 64)), lambda: vae.vae_linear(x, w[0]),
        lambda: vae.vae_linear(x, w, bias=rand(1, 72).to(t)),
        lambda: vae.vae_linear(x, w, residual=x), lambda: vae.vae_linear(x, w, act=5),
        lambda: vae.vae_linear(x, w[:66]), lambda: vae.vae_linear(x, w, out=x),
        lambda: vae.vae_linear(x, w[:64], out=x),
        lambda: vae.vae_linear_dgrad(x, w), lambda: vae.vae_linear_dgrad(x[:, :8], w[:8]),
        lambda: vae.vae_linear_dgrad(x, w.t().contiguous(), z=rand(1, 8, 72, dtype=t)),
        lambda: vae.vae_linear_dgrad(x, w.t().contiguous(), act=vae.VAE_ACT_SILU),
        lambda: vae.vae_linear_wgrad(x, x.float()), lambda: vae.vae_linear_wgrad(x, x[:4]),
        lambda: vae.vae_linear_wgrad(x[:0], x[:0]), lambda: vae.vae_layer_norm(x[:0], g),
        lambda: vae.vae_dropout(x[:0], 0.5, seed=1),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError, vae.VaeError)):
            call()
            pytest.fail(f"call {i} was taken")
    assert vae.vae_device_error() == 0
