"""The training operators on the GPU against float64 forms (tests/_train_ref.py).

Checkpoints are compared bit by bit: a power-of-two scale makes everything but
the rounding to e4m3 exact, and the checkpoints of computed tensors (y, h) are
the quantisation of the float32 output itself. Weight gradients of small
integers are exact as well. Floating outputs are held to bounds counted in
half-steps of float32, H = 2^-24, relative to the largest terms that enter:
each test states its count."""
import numpy as np
import pytest

from tests import _train_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
H = 2.0 ** -24
SENTINEL = -12345.0


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import diffusion_vae_decoder_gb300 as p
    p.load_library()
    yield
    assert p.vae_device_error() == 0


def pkg():
    import diffusion_vae_decoder_gb300 as p
    return p


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


def host(t):
    return t.cpu().numpy().astype(np.float64)


def to_layout(a, layout):
    """[n, ..., c] -> the layout the op is called with."""
    return a if layout == pkg().VAE_NHWC else np.moveaxis(a, -1, 1)


def from_layout(a, layout):
    return a if layout == pkg().VAE_NHWC else np.moveaxis(a, 1, -1)


def parts(k):
    """(codes, scale bytes) of a Checkpoint."""
    return (k.payload.view(torch.uint8).cpu().numpy(), k.scale.view(torch.uint8).cpu().numpy())


def same_codes(k, rows):
    """The checkpoint holds exactly what float32 rows [r, c] quantise to."""
    codes, scale = parts(k)
    want_codes, want_scale = R.quantise(rows)
    assert (scale == want_scale).all()
    nan = (want_codes & 127) == 127
    assert ((codes & 127) == 127)[nan].all()
    assert (codes[~nan] == want_codes[~nan]).all()


LAYOUTS = [0, 1]


# ---------------------------------------------------------------- checkpoints
def awkward_rows(r, c, seed):
    g = np.random.default_rng(seed)
    v = (g.normal(size=(r, c)) * 2.0 ** g.integers(-30, 30, size=(r, 1))).astype(np.float32)
    v[g.random((r, c)) < 0.1] = 0
    return v


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n,h,w,c", [(1, 1, 1, 1), (2, 3, 5, 31), (1, 7, 1, 32), (3, 2, 2, 33),
                                     (1, 9, 15, 100), (2, 16, 8, 128), (1, 1, 2, 516)])
def test_pack_and_unpack_exactly(layout, n, h, w, c):
    rows = awkward_rows(n * h * w, c, 1)
    x = dev(to_layout(rows.reshape(n, h, w, c), layout))
    k = pkg().vae_ckpt_pack(x, layout=layout)
    same_codes(k, rows)
    back = pkg().vae_ckpt_unpack(k, x.shape, layout=layout)
    want = R.dequantise(*parts(k), c).reshape(n, h, w, c)
    assert (host(back) == to_layout(want, layout)).all()


def test_pack_edges_of_the_format():
    """Zeros, the scale's borders (448 and the next float), ties, the smallest
    and largest floats, subnormals, -0, infinities and NaN."""
    tiny, big = 2.0 ** -149, float(np.finfo(np.float32).max)
    rows = np.zeros((14, 32), dtype=np.float32)
    rows[1, 0] = 448
    rows[2, 0] = np.nextafter(np.float32(448), np.float32(500))
    rows[3] = np.float32(1.0625) * np.where(np.arange(32) % 2, 1, -1)
    rows[3, 5] = 400
    rows[4] = tiny * np.arange(32)
    rows[5, :3] = [big, -big, 1]
    rows[6, :4] = [np.inf, 1, 2, 3]
    rows[7, :4] = [1, np.nan, -2, 0]
    rows[8] = 2.0 ** -126 * np.linspace(-1, 1, 32)
    rows[9, 0], rows[9, 1] = 448 * 2.0 ** -127, -1e-40
    rows[10] = -0.0
    rows[11] = np.linspace(-448, 448, 32)
    rows[12, 0], rows[12, 1:] = 256, np.arange(31) * 2.0 ** -10
    rows[13, 0] = -np.inf
    k = pkg().vae_ckpt_pack(dev(rows[None, None]), layout=pkg().VAE_NHWC)
    same_codes(k, rows)
    back = pkg().vae_ckpt_unpack(k, (1, 1, 14, 32), layout=pkg().VAE_NHWC)
    want = R.dequantise(*parts(k), 32).astype(np.float32)
    got = back.cpu().numpy()[0, 0]
    assert (np.isnan(got) == np.isnan(want)).all()
    assert (got[~np.isnan(want)] == want[~np.isnan(want)]).all()


# ---------------------------------------------------------------- GroupNorm + SiLU
GN = [(1, 8, 8, 128, 32), (2, 5, 7, 32, 32), (1, 1, 1, 64, 32), (3, 3, 11, 96, 32),
      (1, 37, 29, 48, 8), (2, 16, 33, 512, 32), (1, 4, 9, 1024, 1), (1, 130, 70, 36, 9)]
# one launch at its largest, several rounds of blocks, a slab of all channels, many
# samples; then three launches
GN_LARGE = [(1, 64, 64, 512, 32), (4, 64, 64, 512, 32), (1, 64, 64, 96, 32), (300, 4, 4, 64, 32),
            (1, 96, 100, 64, 32), (1, 150, 160, 64, 32), (2, 190, 180, 32, 8)]


def gn_data(n, h, w, c, seed):
    g = np.random.default_rng(seed)
    x = (g.normal(size=(n, h, w, c)) * np.exp(0.5 * g.normal(size=c)) + g.normal(size=c))
    return (x.astype(np.float32), g.normal(1, 0.1, c).astype(np.float32),
            g.normal(0, 0.1, c).astype(np.float32))


def gn_out_bound(x, rstd, gamma, beta):
    # mean and rstd: tree sums, under 24 half-steps each of max|x| rstd; the
    # affine 4; exp, 1 + e and the quotient under 24 for |z| <= 12.
    return 64 * H * (np.abs(gamma).max() * np.abs(x).max() * rstd.max() + np.abs(beta).max() + 1)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("n,h,w,c,groups", GN)
def test_groupnorm_ckpt(layout, silu, n, h, w, c, groups):
    x, gamma, beta = gn_data(n, h, w, c, 2)
    eps = 1e-3
    y, kx, ky, stats = pkg().vae_groupnorm_silu_ckpt(
        dev(to_layout(x, layout)), dev(gamma), dev(beta), groups=groups, eps=eps, apply_silu=silu,
        layout=layout)
    x64 = x.reshape(n, h * w, c).astype(np.float64)
    mean, rstd = R.group_stats(x64, groups, eps)
    st = host(stats)
    assert np.abs(st[..., 0] - mean).max() <= 24 * H * np.abs(x).max()
    # d rstd = rstd^3 / 2 d var, and the variance is off by 48 half-steps of max x^2 at most
    assert (np.abs(st[..., 1] - rstd) <= 4 * H * rstd + 24 * H * rstd ** 3 *
            np.abs(x).max() ** 2).all()
    want = R.gn_forward(x64, groups, eps, gamma, beta, silu)
    got = from_layout(host(y), layout).reshape(n, h * w, c)
    # the variance enters z once more, times |x|
    bound = gn_out_bound(x, rstd, gamma, beta) * (1 + (np.abs(x).max() * rstd.max()) ** 2)
    assert np.abs(got - want).max() <= bound
    same_codes(kx, x.reshape(-1, c))
    same_codes(ky, got.reshape(-1, c))


def test_groupnorm_ckpt_keeps_what_is_asked_and_writes_in_place():
    x, gamma, beta = gn_data(2, 6, 5, 64, 3)
    for layout in LAYOUTS:
        xt = dev(to_layout(x, layout))
        y, kx, ky, st = pkg().vae_groupnorm_silu_ckpt(xt, dev(gamma), dev(beta), layout=layout)
        z, nx, ny, st2 = pkg().vae_groupnorm_silu_ckpt(xt, dev(gamma), dev(beta), layout=layout,
                                                       keep_x=False, keep_y=False)
        assert nx is None and ny is None and torch.equal(y, z) and torch.equal(st, st2)
        w, kx2, ky2, _ = pkg().vae_groupnorm_silu_ckpt(xt, dev(gamma), dev(beta), layout=layout,
                                                       out=xt)
        assert w.data_ptr() == xt.data_ptr() and torch.equal(w, y)
        for a, b in ((kx, kx2), (ky, ky2)):
            assert all((p == q).all() for p, q in zip(parts(a), parts(b)))


def test_groupnorm_ckpt_agrees_with_vae_groupnorm_silu():
    x, gamma, beta = gn_data(1, 40, 33, 128, 4)
    for layout in LAYOUTS:
        xt = dev(to_layout(x, layout))
        y = pkg().vae_groupnorm_silu_ckpt(xt, dev(gamma), dev(beta), layout=layout)[0]
        z = pkg().vae_groupnorm_silu(xt, dev(gamma), dev(beta), layout=layout)
        # two evaluations, each within the forward's bound
        _, rstd = R.group_stats(x.reshape(1, -1, 128).astype(np.float64), 32, 1e-6)
        assert float((y - z).abs().max()) <= 2 * gn_out_bound(x, rstd, gamma, beta) * (
            1 + (np.abs(x).max() * rstd.max()) ** 2)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n,h,w,c,groups", GN_LARGE)
def test_groupnorm_pair_on_larger_tensors(layout, n, h, w, c, groups):
    """Against float64 torch on the GPU; the same bounds as below."""
    g = torch.Generator(device="cuda").manual_seed(21)
    f = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rows, dyr = f(n, h * w, c) * 2 + 1, f(n, h * w, c)
    gamma, beta, eps = 1 + 0.1 * f(c), 0.1 * f(c), 1e-4

    def lay(t):
        t = t.view(n, h, w, c)
        return t if layout == 1 else t.permute(0, 3, 1, 2).contiguous()

    def unlay(t):
        return (t if layout == 1 else t.permute(0, 2, 3, 1)).reshape(n, h * w, c).double()

    y, kx, ky, st = pkg().vae_groupnorm_silu_ckpt(lay(rows), gamma, beta, groups=groups, eps=eps,
                                                  layout=layout)
    ga, be, per = gamma.double(), beta.double(), lambda a: a.repeat_interleave(  # noqa: E731
        c // groups, 1)[:, None]
    x = rows.double().view(n, h * w, groups, -1)
    mean, var = x.mean((1, 3)), x.var((1, 3), unbiased=False)
    rstd = (var + eps).rsqrt()
    z = (rows.double() - per(mean)) * per(rstd) * ga + be
    top = float(rows.abs().max() * rstd.max())
    bound = 64 * H * (1.5 * top + 2) * (1 + top ** 2)
    assert float((unlay(y) - z * z.sigmoid()).abs().max()) <= bound
    assert float((st[..., 1].double() - rstd).abs().max()) <= bound
    # the checkpoints are those of a separate pack of x and y
    for kept, t in ((kx, lay(rows)), (ky, y)):
        again = pkg().vae_ckpt_pack(t, layout=layout)
        assert (parts(kept)[0] == parts(again)[0]).all() and (
            parts(kept)[1] == parts(again)[1]).all()
    dx, dgamma, dbeta = pkg().vae_groupnorm_silu_backward(lay(dyr), kx, st, gamma, beta,
                                                          groups=groups, layout=layout)
    xt = unlay(pkg().vae_ckpt_unpack(kx, y.shape, layout=layout))
    xh = (xt - per(st[..., 0].double())) * per(st[..., 1].double())
    z = xh * ga + be
    s = z.sigmoid()
    dz = dyr.double() * s * (1 + z * (1 - s))
    t = (dz * ga).view(n, h * w, groups, -1)
    m = lambda a: a.reshape(n, h * w, groups, -1).mean((1, 3))  # noqa: E731
    want = per(st[..., 1].double()) * (dz * ga - per(m(t)) - xh * per(m(t * xh.view_as(t))))
    limit = 256 * H * float(rstd.max()) * 1.1 * float(dyr.abs().max()) * 1.5 * (
        2 + float(xh.abs().max())) ** 2
    assert float((unlay(dx) - want).abs().max()) <= limit
    size = 1.1 * dyr.double().abs().sum((0, 1))
    assert bool(((dgamma.double() - (dz * xh).sum((0, 1))).abs() <=
                 256 * H * size * (1 + float(xh.abs().max()))).all())
    assert bool(((dbeta.double() - dz.sum((0, 1))).abs() <= 256 * H * size).all())


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("n,h,w,c,groups", GN)
def test_groupnorm_backward(layout, silu, n, h, w, c, groups):
    x, gamma, beta = gn_data(n, h, w, c, 5)
    eps = 1e-3
    g = np.random.default_rng(6)
    dy = g.normal(size=x.shape).astype(np.float32)
    dres = g.normal(size=x.shape).astype(np.float32)
    kx = pkg().vae_ckpt_pack(dev(to_layout(x, layout)), layout=layout)
    x64 = x.reshape(n, h * w, c).astype(np.float64)
    stats = np.stack(R.group_stats(x64, groups, eps), -1).astype(np.float32)
    xt = R.dequantise(*parts(kx), c).reshape(n, h * w, c)
    mean, rstd = (stats[..., i].astype(np.float64) for i in range(2))
    want = R.gn_backward(dy.reshape(n, h * w, c).astype(np.float64), xt, mean, rstd, groups,
                         gamma, beta, silu)
    per = np.repeat(rstd, c // groups, 1)[:, None, :]
    xh = (xt - np.repeat(mean, c // groups, 1)[:, None, :]) * per
    # xh 3 half-steps, the sigmoid's derivative under 64 (|z| <= 16), sums over
    # at most 64 values a thread, then trees: 256 half-steps of the largest terms
    top = 1.1 * np.abs(dy).max() * np.abs(gamma).max()
    bound = 256 * H * rstd.max() * top * (2 + np.abs(xh).max()) ** 2
    for res in (None, dres):
        dx, dgamma, dbeta = pkg().vae_groupnorm_silu_backward(
            dev(to_layout(dy, layout)), kx, dev(stats), dev(gamma), dev(beta), groups=groups,
            apply_silu=silu, layout=layout, dres=None if res is None else dev(to_layout(res, layout)))
        got = from_layout(host(dx), layout).reshape(n, h * w, c)
        add = 0 if res is None else res.reshape(n, h * w, c)
        assert np.abs(got - want[0] - add).max() <= bound + H * (0 if res is None else 10)
        size = 1.1 * np.abs(dy).sum((0, 1, 2))
        assert (np.abs(host(dgamma) - want[1]) <= 256 * H * size * (1 + np.abs(xh).max())).all()
        assert (np.abs(host(dbeta) - want[2]) <= 256 * H * size).all()


def test_groupnorm_backward_is_the_same_in_place_and_again():
    x, gamma, beta = gn_data(2, 19, 23, 64, 7)
    dy = np.random.default_rng(8).normal(size=x.shape)
    for layout in LAYOUTS:
        xt, d = dev(to_layout(x, layout)), dev(to_layout(dy, layout))
        _, kx, _, st = pkg().vae_groupnorm_silu_ckpt(xt, dev(gamma), dev(beta), layout=layout)
        args = (kx, st, dev(gamma), dev(beta))
        a = pkg().vae_groupnorm_silu_backward(d, *args, layout=layout)
        b = pkg().vae_groupnorm_silu_backward(d, *args, layout=layout)
        r = d.clone()
        c = pkg().vae_groupnorm_silu_backward(d, *args, layout=layout, dres=r, out=r)
        e = pkg().vae_groupnorm_silu_backward(d, *args, layout=layout, out=d)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        assert all(torch.equal(p, q) for p, q in zip(a, e)) and e[0].data_ptr() == d.data_ptr()
        # one rounding of a sum of two values
        assert float((c[0] - a[0] - dev(to_layout(dy, layout))).abs().max()) <= 4 * H * float(
            c[0].abs().max() + a[0].abs().max())


def silu_of(betas, layout, pixels):
    """vae_groupnorm_silu_ckpt of a constant: z is beta to the bit, every pixel alike."""
    x = torch.zeros((1, pixels, 1, 64) if layout == 1 else (1, 64, pixels, 1), device="cuda")
    rows = []
    for b in betas.split(64):
        y, _, _, _ = pkg().vae_groupnorm_silu_ckpt(x, torch.ones_like(b), b, groups=2,
                                                   layout=layout)
        y = y.reshape(pixels, 64) if layout == 1 else y.reshape(64, pixels).t()
        assert bool(((y == y[0]) | (y != y)).all())
        rows.append(y[0])
    return torch.cat(rows)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("pixels", [1, 24000])  # one launch, three
def test_silu_is_as_precise_where_it_is_small(layout, pixels):
    """Half-steps of y for |z| <= 12: the exp2 unit 4, its correction 1 and ln 2's
    rounding 0.6, the sum with 1 one, the reciprocal 2, the product 1."""
    z = torch.linspace(-12, 12, 64 * 60, device="cuda")
    want = z.double() * torch.sigmoid(z.double())
    got = silu_of(z, layout, pixels).double()
    assert float(((got - want).abs() / want.abs().clamp(min=1e-30)).max()) <= 10 * H


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("pixels", [1, 24000])
def test_silu_of_the_largest_and_of_non_finite_values(layout, pixels):
    big = [88.0, 104.0, 200.0, 1e6, 2.0 ** 24, 1e9, 1e30, 2.4e38, 3.4e38, float("inf")]
    z = torch.zeros(64, device="cuda")
    z[:10], z[10:20], z[20] = torch.tensor(big), -torch.tensor(big), float("nan")
    got = silu_of(z, layout, pixels)
    want = z / (1 + torch.exp(-z))
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan) and int(nan.sum()) == 2  # -infinity and NaN
    # e^-88 is a small normal number's reciprocal, which may be taken for 0
    assert bool((got[~nan] - want[~nan]).abs().le(2.0 ** -119 + 10 * H * want[~nan].abs())
                .logical_or(got[~nan] == want[~nan]).all())


def leave_nan_in_shared_memory():
    """An ordinary call after which the start of every SM's shared memory holds NaN:
    1024 one-block samples of NaN, whose channels' affines lie there."""
    x = torch.full((1024, 1, 1, 1024), float("nan"), device="cuda")
    v = torch.ones(1024, device="cuda")
    pkg().vae_groupnorm_silu_ckpt(x, v, v, groups=1, layout=pkg().VAE_NHWC, keep_x=False,
                                  keep_y=False)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("n,h,w,c,groups", [(1, 8, 8, 36, 9), (2, 5, 7, 40, 8), (1, 16, 16, 100, 25),
                                            (3, 1, 1, 48, 8), (1, 3, 5, 1020, 5), (1, 2, 2, 4, 1)])
def test_padding_channels_do_not_depend_on_what_ran_before(layout, silu, n, h, w, c, groups):
    """c is no multiple of 32: the last block of y's checkpoint ends in padding."""
    x, gamma, beta = gn_data(n, h, w, c, 30)
    args = dev(to_layout(x, layout)), dev(gamma), dev(beta)
    leave_nan_in_shared_memory()
    y, kx, ky, _ = pkg().vae_groupnorm_silu_ckpt(*args, groups=groups, apply_silu=silu,
                                                 layout=layout)
    same_codes(kx, x.reshape(-1, c))
    same_codes(ky, from_layout(y.cpu().numpy(), layout).reshape(-1, c))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("h,w,c,groups", [(5, 7, 64, 16), (5, 7, 48, 12), (150, 100, 64, 16),
                                          (130, 120, 48, 12)])  # one launch; three
def test_groupnorm_pair_keeps_non_finite_values_apart(layout, value, h, w, c, groups):
    """One value of sample 1, group 3: its group of outputs is lost, and in the backward
    pass the sample's groups that share the checkpoint block. Every other number is, to
    the bit, what it is without it."""
    x, gamma, beta = gn_data(2, h, w, c, 34)
    dy = dev(to_layout(np.random.default_rng(35).normal(size=x.shape), layout))
    args = dev(gamma), dev(beta)
    out = []
    for bad in (False, True):
        x[1, h // 2, w // 3, 13] = value if bad else 0.5
        xt = dev(to_layout(x, layout))
        y, kx, ky, st = pkg().vae_groupnorm_silu_ckpt(xt, *args, groups=groups, layout=layout)
        for kept, t in ((kx, xt), (ky, y)):
            again = pkg().vae_ckpt_pack(t, layout=layout)
            assert all((a == b).all() for a, b in zip(parts(kept), parts(again)))
        dx, dga, dbe = pkg().vae_groupnorm_silu_backward(dy, kx, st, *args, groups=groups,
                                                         layout=layout)
        flat = lambda t: from_layout(t.cpu().numpy(), layout).reshape(2, h * w, c)  # noqa: E731
        out.append([flat(y), st.cpu().numpy(), flat(dx), dga.cpu().numpy(), dbe.cpu().numpy()])
    (y, st, dx, dga, dbe), (yb, stb, dxb, dgab, dbeb) = out
    lost = np.zeros((2, c), dtype=bool)
    lost[1, 12:16] = True
    assert np.isnan(yb[1, :, 12:16]).all() and np.isnan(stb[1, 3, 1])
    assert (yb == y)[:, :, ~lost[1]].all() and (yb[0] == y[0]).all()
    ok = ~lost.reshape(2, groups, -1).any(2)
    assert (stb == st)[ok].all()
    block = np.arange(c) < 32
    assert np.isnan(dxb[1][:, block]).all() and np.isnan(dgab[block]).all()
    assert (dxb[0] == dx[0]).all() and (dxb[1] == dx[1])[:, ~block].all()
    assert (dgab == dga)[~block].all() and (dbeb == dbe)[~block].all()


# ---------------------------------------------------------------- conv weight gradient
WG = [(1, 1, 1, 32, 32), (1, 1, 1, 1, 4), (2, 3, 5, 16, 12), (1, 8, 8, 64, 64), (1, 7, 33, 96, 20),
      (2, 13, 129, 40, 132), (1, 64, 1, 130, 64), (1, 1, 300, 33, 8), (3, 20, 17, 160, 72),
      (1, 40, 90, 128, 128)]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("k", [1, 3])
@pytest.mark.parametrize("n,h,w,cin,cout", WG)
def test_wgrad_exact_integers(layout, k, n, h, w, cin, cout):
    """Integers of at most four bits are exact in e4m3, and their products' sums
    in float32: every element is compared for equality."""
    g = np.random.default_rng(9)
    x = g.integers(-8, 9, size=(n, h, w, cin)).astype(np.float32)
    dy = g.integers(-4, 5, size=(n, h, w, cout)).astype(np.float32)
    kx = pkg().vae_ckpt_pack(dev(x), layout=1)
    dw, dbias = pkg().vae_conv2d_wgrad(dev(to_layout(dy, layout)), kx, k, layout=layout)
    want, wb = R.wgrad(dy.astype(np.float64), x.astype(np.float64), k)
    assert (host(dw) == want).all()
    assert (host(dbias) == wb).all()


def wgrad_bound(dy, xt, k):
    # dy: two parts, off by 2^-22; a chain of 128 truncating steps in each of two
    # accumulators, 2^-23 of the running sum at most each; then rounded sums.
    a, _ = R.wgrad(np.abs(dy), np.abs(xt), k)
    return (2.0 ** -22 + 2 * 128 * 2.0 ** -23 + 64 * H) * a


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("k", [1, 3])
@pytest.mark.parametrize("n,h,w,cin,cout", [(2, 13, 129, 40, 132), (1, 96, 100, 160, 72),
                                            (1, 5, 6, 64, 300)])
def test_wgrad_values(layout, k, n, h, w, cin, cout):
    g = np.random.default_rng(10)
    x = g.normal(size=(n, h, w, cin)) * np.exp2(g.integers(-6, 6, size=(n, h, w, 1)))
    dy = (g.normal(size=(n, h, w, cout)) * 10.0 ** g.integers(-20, 20, size=cout)).astype(
        np.float32)
    kx = pkg().vae_ckpt_pack(dev(x), layout=1)
    xt = R.dequantise(*parts(kx), cin).reshape(x.shape)
    dw, dbias = pkg().vae_conv2d_wgrad(dev(to_layout(dy, layout)), kx, k, layout=layout)
    want, wb = R.wgrad(dy.astype(np.float64), xt, k)
    assert (np.abs(host(dw) - want) <= wgrad_bound(dy.astype(np.float64), xt, k)).all()
    assert (np.abs(host(dbias) - wb) <= 256 * H * np.abs(dy).sum((0, 1, 2))).all()


def test_wgrad_zero_tiny_huge_and_non_finite():
    g = np.random.default_rng(11)
    x = g.normal(size=(1, 6, 7, 64)).astype(np.float32)
    x[0, 2, 3, :32] = 0
    dy = g.normal(size=(1, 6, 7, 16)).astype(np.float32)
    dy[..., 0] = 0
    dy[..., 1] *= 2.0 ** -140   # subnormal
    dy[..., 2] *= 2.0 ** 110
    dy[0, 3, 3, 3] = np.inf
    dy[0, 1, 1, 4] = np.nan
    kx = pkg().vae_ckpt_pack(dev(x), layout=1)
    xt = R.dequantise(*parts(kx), 64).reshape(x.shape)
    dw, dbias = (host(t) for t in pkg().vae_conv2d_wgrad(dev(dy), kx, 3, layout=1))
    fine = [i for i in range(16) if i not in (3, 4)]
    want, wb = R.wgrad(dy[..., fine].astype(np.float64), xt, 3)
    # results under the smallest normal number round to its last subnormal place
    bound = wgrad_bound(dy[..., fine].astype(np.float64), xt, 3) + 2.0 ** -149
    assert (np.abs(dw[fine] - want) <= bound).all()
    assert (dw[0] == 0).all() and dbias[0] == 0
    assert not np.isfinite(dw[3, :, 1, 1]).any() and not np.isfinite(dw[4, :, 1, 1]).any()
    assert dbias[3] == np.inf and np.isnan(dbias[4])
    # a block of NaNs reaches its own 32 input channels and no others
    x[0, 2, 2, 40] = np.nan
    kx = pkg().vae_ckpt_pack(dev(x), layout=1)
    dw2 = host(pkg().vae_conv2d_wgrad(dev(dy[..., :3].repeat(2, -1)[..., :4]), kx, 3, layout=1)[0])
    assert np.isnan(dw2[0, 32:, 1, 1]).all() and np.isfinite(dw2[:, :32]).all()


def test_wgrad_of_zeros_is_zero():
    kx = pkg().vae_ckpt_pack(torch.zeros(1, 9, 9, 32, device="cuda"), layout=1)
    for d in (torch.zeros(1, 9, 9, 8, device="cuda"), torch.ones(1, 9, 9, 8, device="cuda")):
        dw, _ = pkg().vae_conv2d_wgrad(d, kx, 3, layout=1)
        assert (dw == 0).all()


def test_wgrad_many_chains_and_pieces():
    """Pixels for several accumulator chains a piece, against float64 torch."""
    g = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn(1, 512, 640, 32, generator=g, device="cuda")
    dy = torch.randn(1, 512, 640, 32, generator=g, device="cuda")
    kx = pkg().vae_ckpt_pack(x, layout=1)
    xt = pkg().vae_ckpt_unpack(kx, x.shape, layout=1)
    dw, dbias = pkg().vae_conv2d_wgrad(dy, kx, 3, layout=1)
    again, _ = pkg().vae_conv2d_wgrad(dy, kx, 3, layout=1)
    assert torch.equal(dw, again)
    xp = torch.nn.functional.pad(xt.double(), (0, 0, 1, 1, 1, 1))
    d = dy.double().reshape(-1, 32)
    for ky in range(3):
        for kx_ in range(3):
            b = xp[:, ky:ky + 512, kx_:kx_ + 640].reshape(-1, 32)
            want, size = d.t() @ b, d.abs().t() @ b.abs()
            err = (dw[:, :, ky, kx_].double() - want).abs()
            assert bool((err <= (2.0 ** -22 + 2 * 128 * 2.0 ** -23 + 64 * H) * size).all())


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("k", [1, 3])
@pytest.mark.parametrize("below,off", [(21, 0.0), (30, 2.0 ** -39), (60, 2.0 ** -31)])
def test_wgrad_of_activations_far_below_the_largest(layout, k, below, off):
    """One pixel of ones, where dy is 0, and activations 2^below under it everywhere
    else, so that nothing hides what they lose. The scales of blocks are d = below - 2
    to below + 1 binades under the largest; with that at 2^7 in half precision, e4m3
    times 2^(7 - d) is a multiple of 2^(-2 - d): exact for d <= 22, rounded to a multiple
    of 2^-24 for d <= 31 (2^-25 of the scaled largest, at least 224 * 2^7: 2^-39), and
    nothing, 448 * 2^-25 at most, from d = 32 on (2^-31)."""
    g = np.random.default_rng(32)
    n, h, w, cin, cout = 1, 24, 37, 40, 12
    down = np.exp2(g.integers(0, 3, size=(n, h, w, 1)) - float(below))
    x = g.uniform(0.5, 1, size=(n, h, w, cin)) * g.choice([-1, 1], size=(n, h, w, cin)) * down
    x = x.astype(np.float32)
    x[0, 11, 17] = np.where(np.arange(cin) % 2, 1, -1)
    dy = g.normal(size=(n, h, w, cout)).astype(np.float32)
    dy[0, 10:13, 16:19] = 0
    kx = pkg().vae_ckpt_pack(dev(x), layout=1)
    xt = R.dequantise(*parts(kx), cin).reshape(x.shape)
    dw, _ = pkg().vae_conv2d_wgrad(dev(to_layout(dy, layout)), kx, k, layout=layout)
    d64 = dy.astype(np.float64)
    want, _ = R.wgrad(d64, xt, k)
    per, _ = R.wgrad(np.abs(d64), np.full_like(xt, np.abs(xt).max()), k)
    assert (np.abs(host(dw) - want) <= wgrad_bound(d64, xt, k) + off * per).all()


@pytest.mark.parametrize("layout", LAYOUTS)
def test_wgrad_both_parts_of_dy_in_every_chain(layout):
    """Integers of 13 bits need both halves of dy, and x~ is 0 or +-1 in so few pixels
    that every sum of magnitudes stays below 2^24: exact in any order, over several
    chains a piece. Without the second half, in any chain, the sums differ."""
    g = torch.Generator(device="cuda").manual_seed(31)
    h, w, c = 512, 640, 32
    r = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda")  # noqa: E731
    dy = (r(4096, 8192, 1, h, w, c) * (2 * r(0, 2, 1, h, w, c) - 1)).float()
    x = (r(0, 200, 1, h, w, c) == 0).float() * (2 * r(0, 2, 1, h, w, c) - 1)
    kx = pkg().vae_ckpt_pack(x, layout=1)
    d_in = dy if layout == 1 else dy.permute(0, 3, 1, 2).contiguous()
    dw, dbias = pkg().vae_conv2d_wgrad(d_in, kx, 3, layout=layout)
    xp = torch.nn.functional.pad(x.double(), (0, 0, 1, 1, 1, 1))
    d = dy.double().reshape(-1, c)
    first = d.to(torch.float16).double()  # 11 significant bits
    for ky in range(3):
        for kx_ in range(3):
            b = xp[:, ky:ky + h, kx_:kx_ + w].reshape(-1, c)
            assert float((d.abs().t() @ b.abs()).max()) < 2 ** 24
            want = d.t() @ b
            assert torch.equal(dw[:, :, ky, kx_].double(), want)
            # what a chain of 2048 positions would lose: it shows
            rows = slice(200 * 640, 203 * 640)
            lost = (d - first)[rows].t() @ b[rows]
            assert float((lost != 0).double().mean()) > 0.5
    # a value passes 34 additions in a thread, 64 in a block, 10 + 5 behind it at most
    assert float((dbias.double() - d.sum(0)).abs().max()) <= 113 * H * float(d.abs().sum(0).max())


# ---------------------------------------------------------------- block norm
BN = [(1, 1, 4), (1, 1, 512), (2, 3, 32), (1, 17, 100), (3, 5, 128), (2, 9, 256), (1, 40, 512),
      (2, 33, 516), (1, 7, 1024), (2, 11, 1536), (1, 19, 2048), (1, 9, 4096), (5, 1, 2052)]


def bn_data(n, t, c, gate, scale, pre, seed):
    g = np.random.default_rng(seed)
    f = lambda *s, std=1.0, mean=0.0: g.normal(mean, std, s).astype(np.float32)  # noqa: E731
    return dict(u=f(n, t, c) * np.exp(f(c, std=0.3)), x=f(n, t, c, std=2.0),
                w_post=f(c, std=0.1, mean=1.0), gate=f(n, c) if gate else None,
                scale=f(c, std=0.1, mean=0.3) if scale else None,
                w_pre=f(c, std=0.1, mean=1.0) if pre else None)


def bn_call(a, **kw):
    t = {k: None if v is None else dev(v) for k, v in a.items()}
    return pkg().vae_block_norm(t["u"], t["x"], t["w_post"], gate=t["gate"], scale=t["scale"],
                                w_pre=t["w_pre"], **kw)


OPTIONS = [(True, True, True), (False, False, False), (True, False, True), (False, True, True),
           (True, True, False)]


@pytest.mark.parametrize("gate,scale,pre", OPTIONS)
@pytest.mark.parametrize("n,t,c", BN)
def test_block_norm(n, t, c, gate, scale, pre):
    a = bn_data(n, t, c, gate, scale, pre, 13)
    eps = 1e-4
    h, y, ku, kh, rstd = bn_call(a, eps=eps)
    b = {k: None if v is None else v.astype(np.float64) for k, v in a.items()}
    wh, wy, m, r = R.block_norm(b["u"], b["x"], eps, b["w_post"], b["gate"], b["scale"],
                                b["w_pre"])
    # a row's sum of squares: 16 values a lane, then a tree, under 32 half-steps;
    # its root, the factors and the sum another 16
    hb = 48 * H * (np.abs(wh).max() + np.abs(wh - b["x"]).max())
    assert np.abs(host(h) - wh).max() <= hb
    st = host(rstd).reshape(2, n, t)
    assert (np.abs(st[0] - m) <= 32 * H * m).all()
    same_codes(ku, a["u"].reshape(-1, c))
    if pre:
        top = np.abs(b["w_pre"]).max() * r.max()
        assert np.abs(host(y) - wy).max() <= 2 * top * hb + 48 * H * np.abs(wy).max() * (
            1 + r.max() * hb / H / 48)
        same_codes(kh, h.cpu().numpy().reshape(-1, c))
    else:
        assert y is None and kh is None
    # serving keeps nothing and gives the same
    h2, y2, *none = bn_call(a, eps=eps, keep=False)
    assert none == [None, None, None] and torch.equal(h, h2)
    assert y is None or torch.equal(y, y2)


def test_block_norm_in_place():
    a = bn_data(2, 7, 260, True, True, True, 14)
    h, y, ku, kh, rstd = bn_call(a)
    t = {k: dev(v) for k, v in a.items()}
    h2, y2, ku2, kh2, r2 = pkg().vae_block_norm(
        t["u"], t["x"], t["w_post"], gate=t["gate"], scale=t["scale"], w_pre=t["w_pre"],
        out_h=t["x"], out_y=t["u"])
    assert h2.data_ptr() == t["x"].data_ptr() and y2.data_ptr() == t["u"].data_ptr()
    assert torch.equal(h, h2) and torch.equal(y, y2) and torch.equal(rstd, r2)
    assert all((p == q).all() for p, q in zip(parts(ku) + parts(kh), parts(ku2) + parts(kh2)))


def test_block_norm_zero_and_nan_rows_stay_apart():
    a = bn_data(1, 4, 64, True, True, True, 15)
    a["u"][0, 1] = 0
    a["u"][0, 2, 5] = np.nan
    h, y, ku, kh, _ = bn_call(a)
    assert (host(h)[0, 1] == a["x"][0, 1]).all()
    assert np.isnan(host(h)[0, 2]).all() and np.isnan(host(y)[0, 2]).all()
    assert np.isfinite(host(y)[0, [0, 1, 3]]).all()
    same_codes(ku, a["u"].reshape(-1, 64))


@pytest.mark.parametrize("gate,scale,pre", OPTIONS)
@pytest.mark.parametrize("n,t,c", BN + [(2, 700, 64), (400, 2, 36)])
def test_block_norm_backward(n, t, c, gate, scale, pre):
    a = bn_data(n, t, c, gate, scale, pre, 16)
    _, _, ku, kh, rstd = bn_call(a, eps=1e-4)
    g = np.random.default_rng(17)
    dy = g.normal(size=(n, t, c)).astype(np.float32) if pre else None
    u = R.dequantise(*parts(ku), c).reshape(n, t, c)
    h = R.dequantise(*parts(kh), c).reshape(n, t, c) if pre else None
    m, r = host(rstd).reshape(2, n, t)
    b = {k: None if v is None else v.astype(np.float64) for k, v in a.items()}
    d = {k: None if v is None else dev(v) for k, v in a.items()}
    for dh in (g.normal(size=(n, t, c)).astype(np.float32), None):
        if dh is None and not pre:
            continue
        got = pkg().vae_block_norm_backward(
            None if dy is None else dev(dy), None if dh is None else dev(dh), ku, kh, rstd,
            d["w_post"], gate=d["gate"], scale=d["scale"], w_pre=d["w_pre"])
        want = R.block_norm_backward(dy, None if dh is None else dh.astype(np.float64), u, h, m, r,
                                     b["w_post"], b["gate"], b["scale"], b["w_pre"])
        uh = np.abs(u * m[..., None]).max()
        hh = np.abs(h * r[..., None]).max() if pre else 0.0
        up = (0 if dy is None else np.abs(dy * b["w_pre"]).max() * r.max() * (1 + hh * hh))
        up += 0 if dh is None else np.abs(dh).max()
        # two row sums of under 40 half-steps each, a dozen products
        xb = 64 * H * up
        assert np.abs(host(got["dx"]) - want["dx"]).max() <= xb
        f = np.abs(b["w_post"]).max() * (1 if not gate else np.abs(b["gate"]).max()) * (
            1 if not scale else np.abs(b["scale"]).max())
        assert np.abs(host(got["du"]) - want["du"]).max() <= 4 * m.max() * f * (1 + uh * uh) * xb
        # column sums: at most 32 rows a thread, then trees, of terms off by xb
        cb = (xb + 128 * H * np.abs(want["dx"]).max()) * uh * n * t
        others = dict(dw_post=f / np.abs(b["w_post"]).max(), dgate=f, dscale=f)
        if gate:
            others["dgate"] = f / np.abs(b["gate"]).max()
        if scale:
            others["dscale"] = f / np.abs(b["scale"]).max()
        for name in ("dw_post", "dgate", "dscale"):
            if name not in want:
                assert got[name] is None
                continue
            assert np.abs(host(got[name]) - want[name]).max() <= cb * others[name]
        if pre:
            assert np.abs(host(got["dw_pre"]) - want["dw_pre"]).max() <= (
                160 * H * np.abs(dy).max() * hh * n * t)
        else:
            assert got["dw_pre"] is None


# ---------------------------------------------------------------- streams, graphs, memory
def all_ops(n=2, h=24, w=20, c=64):
    """One call of each operator on fixed inputs; returns its tensors. The default
    GroupNorms are one launch each, those of the second of `SIZES` three."""
    p = pkg()
    g = torch.Generator(device="cuda").manual_seed(18)
    f = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, dy, ga, be = f(n, h, w, c), f(n, h, w, c), f(c), f(c)
    u, v, wpo, wpr, sc, gate = f(2, 50, 128), f(2, 50, 128), f(128), f(128), f(128), f(2, 128)
    torch.cuda.synchronize()

    def run(stream=None):
        y, kx, ky, st = p.vae_groupnorm_silu_ckpt(x, ga, be, layout=1, stream=stream)
        dx, dga, dbe = p.vae_groupnorm_silu_backward(dy, kx, st, ga, be, layout=1, dres=x,
                                                     stream=stream)
        dw, db = p.vae_conv2d_wgrad(dx, ky, 3, layout=1, stream=stream)
        h, z, ku, kh, rs = p.vae_block_norm(u, v, wpo, gate=gate, scale=sc, w_pre=wpr,
                                            stream=stream)
        gr = p.vae_block_norm_backward(z, h, ku, kh, rs, wpo, gate=gate, scale=sc, w_pre=wpr,
                                       stream=stream)
        kept = [getattr(k, v).view(torch.uint8) for k in (kx, ky, ku, kh)
                for v in ("payload", "scale")]
        return [y, st, dx, dga, dbe, dw, db, h, z, rs, *gr.values(), *kept]
    return run


SIZES = [(2, 24, 20, 64), (1, 150, 160, 64)]


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("size", SIZES)
def test_ops_on_another_stream(size):
    run = all_ops(*size)
    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = run(stream=side)
    side.synchronize()
    assert same(want, got)
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert same(want, got)


def test_a_streams_results_are_not_in_memory_that_another_stream_still_writes():
    p = pkg()
    u = torch.randn(1, 4096, 512, device="cuda")
    w, side = torch.ones(512, device="cuda"), torch.cuda.Stream()
    want = p.vae_block_norm(u, u, w, keep=False)[0]
    torch.cuda.synchronize()
    for _ in range(3):
        late = torch.empty_like(u)
        torch.cuda._sleep(50_000_000)  # some 25 ms
        late.fill_(SENTINEL)
        del late  # free for the current stream, which has yet to write it
        got = p.vae_block_norm(u, u, w, keep=False, stream=side)[0]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del got


def test_a_result_freed_early_stays_until_the_callers_stream_has_read_it():
    p = pkg()
    u = torch.randn(1, 4096, 512, device="cuda")
    w, side = torch.ones(512, device="cuda"), torch.cuda.Stream()
    want = p.vae_block_norm(u, u, w, keep=False)[0]
    torch.cuda.synchronize()
    got = p.vae_block_norm(u, u, w, keep=False, stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(50_000_000)
    read = got.clone()
    del got
    for _ in range(3):
        p.vae_block_norm(u, 2 * u, w, keep=False, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(read, want)


def test_a_temporary_stays_until_the_other_stream_has_read_it():
    """Inputs whose last reference goes with the call, behind a delay on the call's
    stream; the caller's stream then allocates and fills as much."""
    p = pkg()
    n, h, w, c = 1, 64, 64, 128
    x = torch.randn(n, h, w, c, device="cuda")
    t, v, side = x.view(n, h * w, c), torch.randn(c, device="cuda"), torch.cuda.Stream()
    _, kx, _, st = p.vae_groupnorm_silu_ckpt(x, v, v, layout=1)
    _, _, ku, kh, rs = p.vae_block_norm(t, t, v, w_pre=v)

    def again(k):
        """A checkpoint of its own around copied bytes."""
        buf = torch.zeros(p.Checkpoint.nbytes(k.rows, k.c), dtype=torch.uint8, device="cuda")
        out = p.Checkpoint(buf, k.rows, k.c)
        out.payload.view(torch.uint8).copy_(k.payload.view(torch.uint8))
        out.scale.view(torch.uint8).copy_(k.scale.view(torch.uint8))
        return out

    calls = [
        (lambda **kw: lambda a: p.vae_groupnorm_silu_ckpt(a, v, v, layout=1, **kw),
         lambda: (2 * x,)),
        (lambda **kw: lambda a, k: p.vae_groupnorm_silu_backward(a, k, st, v, v, layout=1, **kw),
         lambda: (2 * x, again(kx))),
        (lambda **kw: lambda a, k: p.vae_conv2d_wgrad(a, k, 3, layout=1, **kw),
         lambda: (2 * x, again(kx))),
        (lambda **kw: lambda a, b: p.vae_block_norm(a, b, v, w_pre=v, **kw),
         lambda: (2 * t, 3 * t)),
        (lambda **kw: lambda a, b, k, m: p.vae_block_norm_backward(a, b, k, m, rs, v, w_pre=v, **kw),
         lambda: (2 * t, 3 * t, again(ku), again(kh))),
        (lambda **kw: lambda a: p.vae_ckpt_pack(a, layout=1, **kw), lambda: (2 * x,)),
        (lambda **kw: lambda k: p.vae_ckpt_unpack(k, x.shape, layout=1, **kw), lambda: (again(kx),)),
    ]

    def flat(r):
        if isinstance(r, p.Checkpoint):
            return [r.payload.view(torch.uint8), r.scale.view(torch.uint8)]
        if isinstance(r, (tuple, dict)):
            return [f for e in (r.values() if isinstance(r, dict) else r) for f in flat(e)]
        return [] if r is None else [r]

    for call, inputs in calls:
        want = flat(call()(*inputs()))
        args = inputs()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(50_000_000)
        got = call(stream=side)(*args)
        del args
        junk = [torch.full_like(x, float("nan")) for _ in range(8)]
        junk += [torch.full((p.Checkpoint.nbytes(h * w, c),), 255, dtype=torch.uint8,
                            device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        assert same(want, flat(got))
        del junk, got


@pytest.mark.parametrize("size", SIZES)
def test_calls_of_two_threads_on_one_stream(size):
    import threading
    runs = [all_ops(*size), all_ops(1, 9, 7, 32)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        for _ in range(6):
            got[i].append(runs[i]())

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(len(g) == 6 and all(same(w, r) for r in g) for w, g in zip(want, got))


@pytest.mark.parametrize("size", SIZES)
def test_two_graphs_replayed_at_once(size):
    run = all_ops(*size)
    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(run())
    torch.cuda.synchronize()
    for _ in range(4):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(same(want, o) for o in outs)


def test_two_runs_at_once():
    run = all_ops()
    want = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [[] for _ in streams]
    for _ in range(4):
        for s, g in zip(streams, got):
            g.append(run(stream=s))
    torch.cuda.synchronize()
    assert all(same(want, r) for g in got for r in g)


@pytest.mark.parametrize("size", SIZES)
def test_captured_and_replayed(size):
    run = all_ops(*size)
    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for t in got:
        t.fill_(0)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert same(want, got)


def shifted(t):
    """A copy that starts 16 bytes behind a 32-byte boundary."""
    buf = torch.empty(t.numel() + 16, device="cuda")
    first = (4 - buf.data_ptr() // 4) % 8
    out = buf[first:first + t.numel()].view(t.shape)
    assert out.data_ptr() % 32 == 16
    return out.copy_(t)


@pytest.mark.parametrize("size", SIZES)
def test_tensors_on_16_byte_boundaries(size):
    """256-bit accesses are taken on 32-byte boundaries only; elsewhere two of 128
    bits bring the same numbers in the same order."""
    p = pkg()
    n, h, w, c = size
    g = torch.Generator(device="cuda").manual_seed(23)
    f = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, dy, ga, be = f(n, h, w, c), f(n, h, w, c), f(c), f(c)
    a = p.vae_groupnorm_silu_ckpt(x, ga, be, layout=1)
    b = p.vae_groupnorm_silu_ckpt(shifted(x), shifted(ga), shifted(be), layout=1,
                                  out=shifted(x))
    bits = lambda k: [k.payload.view(torch.uint8), k.scale.view(torch.uint8)]  # noqa: E731
    assert same([a[0], a[3], *bits(a[1]), *bits(a[2])], [b[0], b[3], *bits(b[1]), *bits(b[2])])
    a2 = p.vae_groupnorm_silu_backward(dy, a[1], a[3], ga, be, layout=1, dres=x)
    b2 = p.vae_groupnorm_silu_backward(shifted(dy), b[1], shifted(b[3]), ga, be, layout=1,
                                       dres=shifted(x), out=shifted(dy))
    assert same(a2, b2)
    for k in (1, 3):
        assert same(p.vae_conv2d_wgrad(dy, a[2], k, layout=1),
                    p.vae_conv2d_wgrad(shifted(dy), b[2], k, layout=1))
    u, v = x.view(n, h * w, c), dy.view(n, h * w, c)
    a = p.vae_block_norm(u, v, ga, w_pre=be)
    b = p.vae_block_norm(shifted(u), shifted(v), shifted(ga), w_pre=shifted(be),
                         out_h=shifted(u), out_y=shifted(u))
    assert same([a[0], a[1], a[4], *bits(a[2]), *bits(a[3])],
                [b[0], b[1], b[4], *bits(b[2]), *bits(b[3])])
    a2 = p.vae_block_norm_backward(v, u, a[2], a[3], a[4], ga, w_pre=be)
    b2 = p.vae_block_norm_backward(shifted(v), shifted(u), b[2], b[3], b[4], ga, w_pre=be)
    assert all(a2[k] is b2[k] or torch.equal(a2[k], b2[k]) for k in a2)


# ---------------------------------------------------------------- offsets past 32 bits
def test_block_norm_and_checkpoints_past_2_to_32_elements():
    """Rows are independent: the last ones are what a call on them alone gives."""
    p = pkg()
    t, c, tail = (1 << 20) + 37, 4096, 64
    u = torch.empty(1, t, c, device="cuda").uniform_(-1, 1)
    w, wp = torch.full((c,), 0.5, device="cuda"), torch.full((c,), 2.0, device="cuda")
    end = u[:, -tail:].contiguous()
    want = p.vae_block_norm(end, end, w, w_pre=wp)
    got = p.vae_block_norm(u, u, w, w_pre=wp)
    bits = lambda k: [k.payload.view(torch.uint8), k.scale.view(torch.uint8)]  # noqa: E731
    last = lambda ts, axis: [v.narrow(axis, v.shape[axis] - tail, tail) for v in ts]  # noqa: E731
    assert same(want[:2], last(got[:2], 1))
    assert same([*bits(want[2]), *bits(want[3])], last([*bits(got[2]), *bits(got[3])], 0))
    grads = p.vae_block_norm_backward(u, u, *got[2:], w, w_pre=wp)
    alone = p.vae_block_norm_backward(end, end, *want[2:], w, w_pre=wp)
    assert same([alone["du"], alone["dx"]], last([grads["du"], grads["dx"]], 1))
    del got, grads
    k = p.vae_ckpt_pack(u, layout=1)
    assert same(bits(p.vae_ckpt_pack(end, layout=1)), last(bits(k), 0))
    back = p.vae_ckpt_unpack(k, u.shape, layout=1)
    assert same([p.vae_ckpt_unpack(p.vae_ckpt_pack(end, layout=1), end.shape, layout=1)],
                last([back], 1))


@pytest.mark.parametrize("layout", LAYOUTS)
def test_groupnorm_pair_past_2_to_32_elements(layout):
    """Two samples of over 2^31 numbers; the second's results against the call on it
    alone, which cuts its sums differently. A thread adds up under 2^13 numbers in a
    row, so sums are off by 2^-11 of their terms' sizes: deviations up to 2 and
    squares up to 4 (mean 2^-10, variance 2^-7, rstd = 1.73 2^-6, y 2^-5; both calls:
    twice that). dx, of size up to 3, has four such terms. A wrong offset gives
    differences of the order of the values."""
    p = pkg()
    c, spatial = 256, (1 << 23) + 40
    shape = (2, spatial, c) if layout == 1 else (2, c, spatial)
    x = torch.empty(shape, device="cuda").uniform_(-1, 1)
    ga, be = torch.full((c,), 1.5, device="cuda"), torch.full((c,), 0.5, device="cuda")
    y, kx, ky, st = p.vae_groupnorm_silu_ckpt(x, ga, be, layout=layout)
    one = x[1:].contiguous()
    y1, kx1, ky1, st1 = p.vae_groupnorm_silu_ckpt(one, ga, be, layout=layout)
    bits = lambda k: [k.payload.view(torch.uint8), k.scale.view(torch.uint8)]  # noqa: E731
    assert all(torch.equal(a[spatial:], b) for a, b in zip(bits(kx), bits(kx1)))
    assert float((st[1] - st1[0]).abs().max()) <= 2.0 ** -5
    assert float((y[1] - y1[0]).abs().max()) <= 2.0 ** -4
    del y, y1, ky, ky1, one
    dx, dga, dbe = p.vae_groupnorm_silu_backward(x, kx, st, ga, be, layout=layout)
    dx1, _, _ = p.vae_groupnorm_silu_backward(x[1:].contiguous(), kx1, st1, ga, be, layout=layout)
    assert float((dx[1] - dx1[0]).abs().max()) <= 2.0 ** -2


def test_groupnorm_statistics_of_long_planes_nchw():
    """A plane of one value behind 256 zeros, which are the first numbers of its first
    256 threads: their sums of deviations lose the same amount at every step. A thread
    adds up at most 2^12 numbers, step i off by i H of the value: half of 2^12 H of the
    mean, and 64 H for the division and the merges behind it."""
    n, c, side = 5, 32, 1 << 23
    value = 1 + 2.0 ** -10 - 2.0 ** -14
    x = torch.full((n, c, side), value, device="cuda")
    x[:, :, :256] = 0
    v = torch.ones(c, device="cuda")
    _, _, _, st = pkg().vae_groupnorm_silu_ckpt(x, v, v, groups=c, layout=pkg().VAE_NCHW, out=x,
                                                keep_x=False, keep_y=False)
    want = value * (1 - 256 / side)
    assert float((st[..., 0].double() - want).abs().max()) <= (2048 + 64) * H * value


@pytest.mark.parametrize("layout", LAYOUTS)
def test_groupnorm_backward_sums_past_2_to_32_elements(layout):
    """Values of -1, 0 and 1, mean 0, rstd 1 and no SiLU: every sum is a whole number
    below 2^24, exact in any order. The parameters' gradients are the sums of the
    samples', and a sample's dx is that of a call on it alone."""
    p = pkg()
    g = torch.Generator(device="cuda").manual_seed(33)
    n, c, spatial = 2, 256, (1 << 23) - 40
    shape = (n, spatial, c) if layout == 1 else (n, c, spatial)
    draw = lambda *s: torch.randint(  # noqa: E731
        -1, 2, s, generator=g, device="cuda", dtype=torch.int8).float()
    kx = [p.vae_ckpt_pack(draw(1, spatial, c), layout=1) for _ in range(n)]
    both = p.Checkpoint(torch.empty(p.Checkpoint.nbytes(n * spatial, c), dtype=torch.uint8,
                                    device="cuda"), n * spatial, c)
    for part in ("payload", "scale"):
        torch.cat([getattr(k, part).view(torch.uint8) for k in kx],
                  out=getattr(both, part).view(torch.uint8))
    dy = draw(*shape)
    st = torch.tensor([0.0, 1.0], device="cuda").expand(n, 32, 2).contiguous()
    ga, be = torch.full((c,), 1.5, device="cuda"), torch.full((c,), 0.5, device="cuda")
    dx, dga, dbe = p.vae_groupnorm_silu_backward(dy, both, st, ga, be, apply_silu=False,
                                                 layout=layout)
    sums = torch.zeros(2, c, device="cuda")
    for i in range(n):
        dx1, dga1, dbe1 = p.vae_groupnorm_silu_backward(dy[i:i + 1], kx[i], st[i:i + 1], ga, be,
                                                        apply_silu=False, layout=layout)
        assert torch.equal(dx[i], dx1[0])
        sums += torch.stack([dga1, dbe1])
    assert torch.equal(torch.stack([dga, dbe]), sums)
    assert torch.equal(dbe.double(), dy.sum((0, 1) if layout == 1 else (0, 2), dtype=torch.float64))


@pytest.mark.parametrize("layout", LAYOUTS)
def test_wgrad_past_2_to_32_elements(layout):
    """Small integers, whose sums stay below 2^24, are exact whatever their order:
    the whole is the sum of its samples."""
    p = pkg()
    n, h, w, cin, cout = 2, 2048, 2056, 512, 512  # 2^32 + bytes of payload, numbers of dy
    g = torch.Generator(device="cuda").manual_seed(24)
    shape = (n, h, w, cout) if layout == 1 else (n, cout, h, w)
    dy = torch.randint(-1, 2, shape, generator=g, device="cuda", dtype=torch.int8).float()
    x = torch.randint(-1, 2, (n, h * w, cin), generator=g, device="cuda", dtype=torch.int8).float()
    dw, db = p.vae_conv2d_wgrad(dy, p.vae_ckpt_pack(x, layout=1), 1, layout=layout)
    parts_ = [p.vae_conv2d_wgrad(dy[i:i + 1].contiguous(),
                                 p.vae_ckpt_pack(x[i:i + 1].contiguous(), layout=1), 1,
                                 layout=layout) for i in range(n)]
    assert torch.equal(dw, parts_[0][0] + parts_[1][0])
    assert torch.equal(db, parts_[0][1] + parts_[1][1])


# ---------------------------------------------------------------- memory
def test_nothing_is_written_behind_the_outputs():
    """Outputs inside larger buffers, through the C ABI: what lies behind stays."""
    p, lib = pkg(), pkg().load_library()
    n, h, w, c, groups, guard = 1, 5, 7, 40, 8, 4096
    rows = n * h * w
    g = torch.Generator(device="cuda").manual_seed(19)
    f = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, dy, ga, be = f(n, h, w, c), f(n, h, w, c), f(c), f(c)
    nb = lib.vae_ckpt_bytes(rows, c)
    at = (rows * 64 + 255) // 256 * 256  # of the scales; c = 40 fills up to 64
    two = lambda k: (k.data_ptr(), k.data_ptr() + at)  # noqa: E731

    def floats(count):
        return torch.full((count + guard,), SENTINEL, device="cuda")

    def kept():
        return torch.full((nb + guard,), 77, dtype=torch.uint8, device="cuda")

    def workspace(size):
        return torch.full((size + guard,), 77, dtype=torch.uint8, device="cuda")

    y, kx, ky, st = floats(rows * c), kept(), kept(), floats(2 * n * groups)
    size = lib.vae_groupnorm_silu_ckpt_workspace_size(n, c, h * w, 1, groups)
    assert size == 0  # the guard then has to stay untouched from its first byte
    ws = workspace(size)
    assert lib.vae_groupnorm_silu_ckpt(
        x.data_ptr(), n, c, h * w, 1, groups, 1e-6, ga.data_ptr(), be.data_ptr(), 1, y.data_ptr(),
        *two(kx), *two(ky), st.data_ptr(), ws.data_ptr(), size, None) == 0
    size_b = lib.vae_groupnorm_silu_backward_workspace_size(n, c, h * w, 1, groups)
    ws_b, dx, dga, dbe = workspace(size_b), floats(rows * c), floats(c), floats(c)
    assert lib.vae_groupnorm_silu_backward(
        dy.data_ptr(), *two(kx), st.data_ptr(), n, c, h * w, 1, groups, ga.data_ptr(),
        be.data_ptr(), 1, None, dx.data_ptr(), dga.data_ptr(), dbe.data_ptr(), ws_b.data_ptr(),
        size_b, None) == 0
    size_w = lib.vae_conv2d_wgrad_workspace_size(n, c, h, w, 1, c, 3)
    ws_w, dw, db = workspace(size_w), floats(c * c * 9), floats(c)
    assert lib.vae_conv2d_wgrad(dy.data_ptr(), *two(ky), n, c, h, w, 1, c, 3, dw.data_ptr(),
                                db.data_ptr(), ws_w.data_ptr(), size_w, None) == 0
    hh, z, ku, kh, rs = floats(rows * c), floats(rows * c), kept(), kept(), floats(2 * rows)
    assert lib.vae_block_norm(x.data_ptr(), dy.data_ptr(), n, rows, c, 1e-6, ga.data_ptr(), None,
                              None, be.data_ptr(), hh.data_ptr(), z.data_ptr(), *two(ku),
                              *two(kh), rs.data_ptr(), None) == 0
    size_n = lib.vae_block_norm_backward_workspace_size(n, rows, c, 0)
    ws_n, du, dx2, g1, g2 = (workspace(size_n), floats(rows * c), floats(rows * c), floats(c),
                             floats(c))
    assert lib.vae_block_norm_backward(
        dy.data_ptr(), dy.data_ptr(), *two(ku), *two(kh), rs.data_ptr(), n, rows, c,
        ga.data_ptr(), None, None, be.data_ptr(), du.data_ptr(), dx2.data_ptr(), g1.data_ptr(),
        None, None, g2.data_ptr(), ws_n.data_ptr(), size_n, None) == 0
    torch.cuda.synchronize()
    for t in (y, st, dx, dga, dbe, dw, db, hh, z, rs, du, dx2, g1, g2):
        assert (t[-guard:] == SENTINEL).all() and not (t[:-guard] == SENTINEL).any()
    for t in (kx, ky, ku, kh, ws, ws_b, ws_w, ws_n):
        assert (t[-guard:] == 77).all()
    k = p.Checkpoint(kx, rows, c)
    same_codes(k, x.cpu().numpy().reshape(rows, c))


def test_refusals_of_the_binding():
    p = pkg()
    x = torch.randn(2, 4, 4, 64, device="cuda")
    v = torch.ones(64, device="cuda")
    k = p.vae_ckpt_pack(x, layout=1)
    st = torch.zeros(2, 32, 2, device="cuda")
    with pytest.raises(ValueError):
        p.vae_groupnorm_silu_ckpt(x, v[:32], v, layout=1)
    with pytest.raises(ValueError):
        p.vae_groupnorm_silu_backward(x, p.vae_ckpt_pack(x[:1], layout=1), st, v, v, layout=1)
    with pytest.raises(ValueError):
        p.vae_groupnorm_silu_backward(x, k, st[:1], v, v, layout=1)
    with pytest.raises(TypeError):
        p.vae_groupnorm_silu_backward(x, k.payload, st, v, v, layout=1)
    with pytest.raises(TypeError):
        p.vae_ckpt_pack(x.half(), layout=1)
    with pytest.raises(TypeError):
        p.vae_ckpt_pack(x.transpose(1, 2), layout=1)
    with pytest.raises(ValueError):
        p.vae_conv2d_wgrad(x[:1].contiguous(), k, 3, layout=1)
    with pytest.raises(p.VaeError):
        p.vae_conv2d_wgrad(x, k, 5, layout=1)
    with pytest.raises(p.VaeError):
        p.vae_groupnorm_silu_ckpt(x, v, v, groups=24, layout=1)
    with pytest.raises(ValueError):
        p.Checkpoint(torch.zeros(64, dtype=torch.uint8, device="cuda"), 32, 64)
    t = x.view(2, 16, 64)
    with pytest.raises(ValueError):
        p.vae_block_norm(t, t[:, :8].contiguous(), v)
    with pytest.raises(ValueError):
        p.vae_block_norm(t, t, v, gate=v)
    with pytest.raises(ValueError):
        p.vae_block_norm_backward(t, None, k, k, torch.zeros(2, 32, device="cuda"), v)
    with pytest.raises(ValueError):
        p.vae_ckpt_unpack(k, (1, 4, 4, 64))


# ---------------------------------------------------------------- a step of a resnet
@pytest.mark.parametrize("layout", LAYOUTS)
def test_resnet_step(layout):
    """x + conv2(silu(norm2(conv1(silu(norm1(x)))))) through a 1x1 shortcut, forward
    and backward, as a training step calls it; every gradient against the
    float64 forms on the same checkpoints and saved values. The convs and the
    data gradients are TF32 products (per-layer relative L2 1e-3)."""
    p = pkg()
    n, h, w, ci, co = 2, 12, 18, 64, 96
    g = np.random.default_rng(20)
    f = lambda *s, std=1.0, mean=0.0: g.normal(mean, std, s).astype(np.float32)  # noqa: E731
    x = dev(to_layout(f(n, h, w, ci), layout))
    w1, w2, ws = f(co, ci, 3, 3, std=(9 * ci) ** -0.5), f(co, co, 3, 3, std=(9 * co) ** -0.5), f(
        co, ci, 1, 1, std=ci ** -0.5)
    ga1, be1, ga2, be2 = f(ci, std=0.1, mean=1), f(ci, std=0.1), f(co, std=0.1, mean=1), f(
        co, std=0.1)
    a1, kx, ka1, st1 = p.vae_groupnorm_silu_ckpt(x, dev(ga1), dev(be1), layout=layout)
    v = p.vae_conv2d(a1, dev(w1), layout=layout)
    a2, kv, ka2, st2 = p.vae_groupnorm_silu_ckpt(v, dev(ga2), dev(be2), layout=layout)
    p.vae_conv2d(a2, dev(w2), sc_x=x, sc_w=dev(ws), layout=layout)
    dy = dev(to_layout(f(n, h, w, co), layout))

    def flipped(t):
        return dev(np.ascontiguousarray(t[:, :, ::-1, ::-1].transpose(1, 0, 2, 3)))

    dw2, db2 = p.vae_conv2d_wgrad(dy, ka2, 3, layout=layout)
    dws, _ = p.vae_conv2d_wgrad(dy, kx, 1, layout=layout)
    da2 = p.vae_conv2d(dy, flipped(w2), layout=layout)
    dv, dga2, dbe2 = p.vae_groupnorm_silu_backward(da2, kv, st2, dev(ga2), dev(be2),
                                                   layout=layout)
    dw1, db1 = p.vae_conv2d_wgrad(dv, ka1, 3, layout=layout)
    da1 = p.vae_conv2d(dv, flipped(w1), layout=layout)
    dskip = p.vae_conv2d(dy, flipped(ws), layout=layout)
    dx, dga1, dbe1 = p.vae_groupnorm_silu_backward(da1, kx, st1, dev(ga1), dev(be1),
                                                   layout=layout, dres=dskip)
    torch.cuda.synchronize()

    # the same chain in float64
    read = lambda k, c: R.dequantise(*parts(k), c)  # noqa: E731
    dyr = from_layout(host(dy), layout)

    def dgrad(d, wt):
        k = wt.shape[2]
        dp = np.pad(d, ((0, 0), (k // 2,) * 2, (k // 2,) * 2, (0, 0)))
        out = np.zeros(d.shape[:3] + (wt.shape[1],))
        for ky in range(k):
            for kx_ in range(k):
                out += dp[:, ky:ky + h, kx_:kx_ + w] @ wt[:, :, k - 1 - ky, k - 1 - kx_].astype(
                    np.float64)
        return out

    def gnb(d, k, st, ga, be, c):
        s = host(st)
        o = R.gn_backward(d.reshape(n, h * w, c), read(k, c).reshape(n, h * w, c), s[..., 0],
                          s[..., 1], 32, ga, be, True)
        return o[0].reshape(n, h, w, c), o[1], o[2]

    want = {}
    want["dw2"], want["db2"] = R.wgrad(dyr, read(ka2, co).reshape(n, h, w, co), 3)
    want["dws"], _ = R.wgrad(dyr, read(kx, ci).reshape(n, h, w, ci), 1)
    rv, want["dga2"], want["dbe2"] = gnb(dgrad(dyr, w2), kv, st2, ga2, be2, co)
    want["dw1"], want["db1"] = R.wgrad(rv, read(ka1, ci).reshape(n, h, w, ci), 3)
    rx, want["dga1"], want["dbe1"] = gnb(dgrad(rv, w1), kx, st1, ga1, be1, ci)
    want["dx"] = rx + dgrad(dyr, ws)
    got = dict(dw2=dw2, db2=db2, dws=dws, dga2=dga2, dbe2=dbe2, dw1=dw1, db1=db1, dga1=dga1,
               dbe1=dbe1, dx=dx)
    for name, t in got.items():
        a = from_layout(host(t), layout) if name == "dx" else host(t)
        rel = np.linalg.norm(a - want[name]) / np.linalg.norm(want[name])
        assert rel <= (1e-6 if name in ("dw2", "db2", "dws") else 3e-3), (name, rel)
