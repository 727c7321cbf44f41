"""Host-side checks of the training operators (no GPU): their entry points
refuse bad calls before anything is launched, workspace sizes, the checkpoint's
size, and the float64 forms the GPU tests compare with, against differences."""
import ctypes
import os

import numpy as np
import pytest

from tests import _train_ref as R

OK, EINVAL, EUNSUPPORTED, EWORKSPACE = 0, -1, -2, -3
P = ctypes.c_void_p(256)     # never read: every call here is refused
ODD = ctypes.c_void_p(260)   # not 16-byte aligned
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    import diffusion_vae_decoder_gb300 as pkg
    if not os.path.exists(pkg.LIB_PATH):
        from diffusion_vae_decoder_gb300 import _build
        _build.build()
    return pkg.load_library()


def test_ckpt_bytes(lib):
    for rows, c in ((1, 1), (1, 32), (7, 33), (100, 128), (4096, 512), (3, 1000)):
        cp = (c + 31) // 32 * 32
        assert lib.vae_ckpt_bytes(rows, c) == (rows * cp + 255) // 256 * 256 + rows * cp // 32
    import diffusion_vae_decoder_gb300 as pkg
    for rows, c in ((1, 1), (7, 33), (4096, 512)):
        assert pkg.Checkpoint.nbytes(rows, c) == lib.vae_ckpt_bytes(rows, c)
    for rows, c in ((0, 32), (-1, 32), (4, 0), (1 << 31, 32), (1, 65537)):
        assert lib.vae_ckpt_bytes(rows, c) == 0


@pytest.mark.parametrize("fn", ["vae_ckpt_pack", "vae_ckpt_unpack"])
@pytest.mark.parametrize("args,status", [
    (dict(x=None), EINVAL), (dict(q=None), EINVAL), (dict(s=None), EINVAL), (dict(n=0), EINVAL),
    (dict(c=0), EINVAL), (dict(sp=0), EINVAL), (dict(lay=2), EINVAL), (dict(x=ODD), EINVAL),
    (dict(q=ODD), EINVAL), (dict(s=ODD), EINVAL), (dict(n=65536), EUNSUPPORTED),
    (dict(n=2, sp=1 << 30), EUNSUPPORTED), (dict(c=65537), EUNSUPPORTED)])
def test_pack_and_unpack_refuse(lib, fn, args, status):
    a = dict(x=P, q=P, s=P, n=1, c=32, sp=4, lay=0) | args
    size = (a["n"], a["c"], a["sp"], a["lay"])
    if fn == "vae_ckpt_pack":
        assert lib.vae_ckpt_pack(a["x"], *size, a["q"], a["s"], None) == status
    else:
        assert lib.vae_ckpt_unpack(a["q"], a["s"], *size, a["x"], None) == status


def gn_fwd(lib, x=P, n=1, c=64, sp=1 << 20, lay=1, g=32, ga=P, be=P, y=P, kx=P, sx=P, ky=P, sy=P,
           st=P, ws=P, nb=BIG):
    return lib.vae_groupnorm_silu_ckpt(x, n, c, sp, lay, g, 1e-6, ga, be, 1, y, kx, sx, ky, sy, st,
                                       ws, nb, None)


def gn_bwd(lib, dy=P, kx=P, sx=P, st=P, n=1, c=64, sp=1 << 20, lay=1, g=32, ga=P, be=P, res=None,
           dx=P, ws=P, nb=BIG):
    return lib.vae_groupnorm_silu_backward(dy, kx, sx, st, n, c, sp, lay, g, ga, be, 1, res, dx, P,
                                           P, ws, nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), EINVAL), (dict(c=0), EINVAL), (dict(sp=0), EINVAL), (dict(lay=2), EINVAL),
    (dict(g=0), EINVAL), (dict(g=24), EUNSUPPORTED), (dict(c=1056), EUNSUPPORTED),
    (dict(c=66, g=33), EUNSUPPORTED), (dict(n=65536), EUNSUPPORTED),
    (dict(sp=1 << 31), EUNSUPPORTED), (dict(nb=8), EWORKSPACE), (dict(ws=None), EINVAL),
    (dict(ws=ODD), EINVAL), (dict(st=None), EINVAL), (dict(ga=None), EINVAL),
    (dict(be=None), EINVAL)])
def test_groupnorm_pair_refuses(lib, kw, status):
    assert gn_fwd(lib, **kw) == status
    assert gn_bwd(lib, **kw) == status


@pytest.mark.parametrize("kw", [dict(x=None), dict(y=None), dict(x=ODD), dict(y=ODD),
                                dict(kx=ODD), dict(ky=ODD), dict(kx=None), dict(sx=None),
                                dict(ky=None), dict(sy=None), dict(sx=ODD), dict(sy=ODD)])
def test_groupnorm_forward_refuses_pointers(lib, kw):
    assert gn_fwd(lib, **kw) == EINVAL


@pytest.mark.parametrize("kw", [dict(dy=None), dict(kx=None), dict(sx=None), dict(dx=None), dict(dy=ODD),
                                dict(kx=ODD), dict(res=ODD), dict(dx=ODD)])
def test_groupnorm_backward_refuses_pointers(lib, kw):
    assert gn_bwd(lib, **kw) == EINVAL


def wgrad(lib, dy=P, k8=P, s8=P, n=1, cin=32, h=8, w=8, lay=1, cout=32, k=3, dw=P, ws=P, nb=BIG):
    return lib.vae_conv2d_wgrad(dy, k8, s8, n, cin, h, w, lay, cout, k, dw, None, ws, nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), EINVAL), (dict(k8=None), EINVAL), (dict(s8=None), EINVAL), (dict(s8=ODD), EINVAL), (dict(dw=None), EINVAL),
    (dict(ws=None), EINVAL), (dict(n=0), EINVAL), (dict(cin=0), EINVAL), (dict(h=0), EINVAL),
    (dict(w=-1), EINVAL), (dict(cout=0), EINVAL), (dict(lay=3), EINVAL), (dict(dy=ODD), EINVAL),
    (dict(k8=ODD), EINVAL), (dict(ws=ODD), EINVAL), (dict(k=2), EUNSUPPORTED),
    (dict(k=5), EUNSUPPORTED), (dict(cin=4097), EUNSUPPORTED), (dict(cout=4100), EUNSUPPORTED),
    (dict(h=65536), EUNSUPPORTED), (dict(w=65536), EUNSUPPORTED),
    (dict(h=32768, w=32768), EUNSUPPORTED), (dict(cout=6), EUNSUPPORTED),
    (dict(nb=64), EWORKSPACE)])
def test_wgrad_refuses(lib, kw, status):
    assert wgrad(lib, **kw) == status


def bn_fwd(lib, u=P, x=P, n=1, t=4, c=64, wpo=P, gate=None, sc=None, wpr=P, h=P, y=P, ku=P, su=P,
           kh=P, sh=P, rs=P):
    return lib.vae_block_norm(u, x, n, t, c, 1e-6, wpo, gate, sc, wpr, h, y, ku, su, kh, sh, rs,
                              None)


@pytest.mark.parametrize("kw,status", [
    (dict(u=None), EINVAL), (dict(x=None), EINVAL), (dict(wpo=None), EINVAL),
    (dict(h=None), EINVAL), (dict(y=None), EINVAL), (dict(wpr=None), EINVAL),
    (dict(ku=None), EINVAL), (dict(kh=None), EINVAL), (dict(rs=None), EINVAL),
    (dict(su=None), EINVAL), (dict(sh=None), EINVAL), (dict(kh=None, sh=None), EINVAL),
    (dict(ku=None, su=None), EINVAL), (dict(wpr=None, y=None), EINVAL), (dict(n=0), EINVAL), (dict(t=0), EINVAL),
    (dict(c=0), EINVAL), (dict(u=ODD), EINVAL), (dict(gate=ODD), EINVAL), (dict(kh=ODD), EINVAL),
    (dict(c=66), EUNSUPPORTED), (dict(c=4100), EUNSUPPORTED), (dict(n=65536), EUNSUPPORTED),
    (dict(n=4, t=1 << 29), EUNSUPPORTED)])
def test_block_norm_refuses(lib, kw, status):
    assert bn_fwd(lib, **kw) == status


def bn_bwd(lib, dy=P, dh=P, ku=P, su=P, kh=P, sh=P, rs=P, n=1, t=4, c=64, wpo=P, gate=P, sc=P, wpr=P, du=P,
           dx=P, dwpo=P, dgate=P, dsc=P, dwpr=P, ws=P, nb=BIG):
    return lib.vae_block_norm_backward(dy, dh, ku, su, kh, sh, rs, n, t, c, wpo, gate, sc, wpr, du, dx,
                                       dwpo, dgate, dsc, dwpr, ws, nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), EINVAL), (dict(kh=None), EINVAL), (dict(wpr=None), EINVAL),
    (dict(dy=None, dh=None, kh=None, sh=None, wpr=None, dwpr=None), EINVAL), (dict(ku=None), EINVAL),
    (dict(rs=None), EINVAL), (dict(wpo=None), EINVAL), (dict(du=None), EINVAL),
    (dict(dx=None), EINVAL), (dict(ws=None), EINVAL), (dict(gate=None), EINVAL),
    (dict(sc=None), EINVAL), (dict(dy=None, kh=None, sh=None, wpr=None), EINVAL),
    (dict(su=None), EINVAL), (dict(sh=None), EINVAL), (dict(dh=ODD), EINVAL),
    (dict(n=0), EINVAL), (dict(c=2), EUNSUPPORTED), (dict(nb=4), EWORKSPACE)])
def test_block_norm_backward_refuses(lib, kw, status):
    assert bn_bwd(lib, **kw) == status


def test_workspace_sizes(lib):
    assert lib.vae_conv2d_wgrad_workspace_size(1, 128, 64, 64, 1, 128, 3) > 0
    assert lib.vae_conv2d_wgrad_workspace_size(1, 128, 64, 64, 1, 128, 2) == 0
    assert lib.vae_groupnorm_silu_ckpt_workspace_size(1, 64, 1 << 20, 1, 32) > 0
    assert lib.vae_groupnorm_silu_ckpt_workspace_size(1, 64, 64, 1, 32) == 0  # none is used
    assert lib.vae_groupnorm_silu_ckpt_workspace_size(1, 64, 64, 1, 24) == 0
    assert lib.vae_groupnorm_silu_backward_workspace_size(1, 64, 1 << 20, 0, 32) > 0
    assert lib.vae_groupnorm_silu_backward_workspace_size(2, 64, 64, 0, 32) > 0
    assert lib.vae_groupnorm_silu_backward_workspace_size(1, 64, 0, 0, 32) == 0
    one = lib.vae_block_norm_backward_workspace_size(1, 4096, 512, 0)
    assert 0 < one and lib.vae_block_norm_backward_workspace_size(0, 4096, 512, 0) == 0
    # without a gate all rows are one sample, with one the samples' sums are apart
    assert lib.vae_block_norm_backward_workspace_size(512, 8, 512, 1) > one


def test_python_refuses_what_is_not_on_the_gpu():
    torch = pytest.importorskip("torch")
    import diffusion_vae_decoder_gb300 as pkg
    t = torch.zeros(1, 4, 32)
    with pytest.raises(TypeError):
        pkg.vae_block_norm(t, t, t[0, 0])
    with pytest.raises(TypeError):
        pkg.vae_ckpt_pack(t)
    with pytest.raises(TypeError):
        pkg.Checkpoint(torch.zeros(512, dtype=torch.uint8), 1, 32)
    with pytest.raises(TypeError):
        pkg.vae_conv2d_wgrad(t, None, 3)
    with pytest.raises(ValueError):
        pkg.vae_block_norm_backward(None, None, None, None, None, t[0, 0])


def test_a_call_on_another_stream_records_what_it_reads_and_returns(monkeypatch):
    """Inputs, buffers for results and checkpoints belong to the caller's stream: the
    allocator has to be told that the other stream uses them, or a temporary's
    memory is given away while the kernel still reads it."""
    import contextlib
    torch = pytest.importorskip("torch")
    import diffusion_vae_decoder_gb300 as pkg

    class Stream:
        device = "cuda:0"

    here, side = Stream(), Stream()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: here)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    seen = []

    class Fake:
        device = "cuda:0"

        def __init__(self, name):
            self.name = name

        def record_stream(self, stream):
            seen.append((self.name, "side" if stream is side else "here"))

    def checkpoint(name, packed):
        k = pkg.Checkpoint.__new__(pkg.Checkpoint)
        k.rows, k.c = 1, 32
        k._bytes = Fake(name) if packed else None
        k._payload, k._scale = (None, None) if packed else (Fake(name + ".q"), Fake(name + ".s"))
        return k

    result = (Fake("y"), None, checkpoint("kept", False), dict(g=Fake("g"), none=None))
    call = lambda *args: result  # noqa: E731
    args = (Fake("x"), None, 32, 1e-6, True, (1, 2, 3), checkpoint("a", True),
            checkpoint("b", False), Fake("out"))
    assert pkg._on(side, call, *args) is result
    assert sorted(seen) == sorted(
        [(n, "side") for n in ("x", "a", "b.q", "b.s", "out")] +
        [(n, "here") for n in ("y", "kept.q", "kept.s", "g")])
    seen.clear()
    pkg._on(here, call, *args)  # the caller's own stream: nothing to tell
    assert not seen

    def failing(*args):
        raise pkg.VaeError("op", -5)  # perhaps behind its first kernel

    with pytest.raises(pkg.VaeError):
        pkg._on(side, failing, *args)
    assert sorted(seen) == [(n, "side") for n in ("a", "b.q", "b.s", "out", "x")]


# ---------------------------------------------------------------- the float64 forms
def _difference(f, a, d, step=1e-5):
    """Central difference of f along d at a."""
    return (f(a + step * d) - f(a - step * d)) / (2 * step)


def test_round_e4m3_is_nearest_even():
    assert [int(R.round_e4m3(np.float64(v))) for v in (0.0, 1.0, 1.0625, 1.1875, 448.0, 2 ** -10,
                                                       1.5 * 2 ** -9)] == [
        0, 56, 56, 58, 126, 0, 2]
    codes = np.arange(127)
    assert (R.round_e4m3(R.E4M3[:127]) == codes).all()


@pytest.mark.parametrize("silu", [False, True])
def test_groupnorm_gradient_formula_against_differences(silu):
    r = np.random.default_rng(1)
    x, dy = r.normal(size=(2, 5, 12)), r.normal(size=(2, 5, 12))
    gamma, beta = r.normal(1, 0.2, 12), r.normal(0, 0.2, 12)
    mean, rstd = R.group_stats(x, 4, 1e-3)
    dx, dgamma, dbeta = R.gn_backward(dy, x, mean, rstd, 4, gamma, beta, silu)
    loss = lambda a, g, b: (dy * R.gn_forward(a, 4, 1e-3, g, b, silu)).sum()  # noqa: E731
    # second-order remainder of a central difference at 1e-5 plus float64 rounding: ~1e-9
    d = r.normal(size=x.shape)
    assert abs(_difference(lambda a: loss(a, gamma, beta), x, d) - (dx * d).sum()) < 1e-7
    d = r.normal(size=12)
    assert abs(_difference(lambda a: loss(x, a, beta), gamma, d) - (dgamma * d).sum()) < 1e-7
    assert abs(_difference(lambda a: loss(x, gamma, a), beta, d) - (dbeta * d).sum()) < 1e-7


@pytest.mark.parametrize("with_pre", [False, True])
def test_block_norm_gradient_formula_against_differences(with_pre):
    r = np.random.default_rng(2)
    a = dict(u=r.normal(size=(2, 3, 8)), x=r.normal(size=(2, 3, 8)), w_post=r.normal(1, 0.2, 8),
             gate=r.normal(size=(2, 8)), scale=r.normal(0.3, 0.1, 8),
             w_pre=r.normal(1, 0.2, 8) if with_pre else None)
    dy, dh = r.normal(size=(2, 3, 8)), r.normal(size=(2, 3, 8))

    def loss(**kw):
        b = {**a, **kw}
        h, y, _, _ = R.block_norm(b["u"], b["x"], 1e-3, b["w_post"], b["gate"], b["scale"],
                                  b["w_pre"])
        return (dh * h).sum() + (0 if y is None else (dy * y).sum())

    h, _, m, rr = R.block_norm(a["u"], a["x"], 1e-3, a["w_post"], a["gate"], a["scale"],
                               a["w_pre"])
    got = R.block_norm_backward(dy, dh, a["u"], h, m, rr, a["w_post"], a["gate"], a["scale"],
                                a["w_pre"])
    for name, v in a.items():
        if v is None:
            continue
        d = r.normal(size=v.shape)
        want = _difference(lambda t: loss(**{name: t}), v, d)
        assert abs(want - (got["d" + name] * d).sum()) < 1e-7, name


@pytest.mark.parametrize("k", [1, 3])
def test_wgrad_formula_against_differences(k):
    import oracle as O
    r = np.random.default_rng(3)
    x, w = r.normal(size=(2, 3, 4, 5)), r.normal(size=(2, 3, k, k))
    dy = r.normal(size=(2, 2, 4, 5))
    dw, dbias = R.wgrad(np.moveaxis(dy, 1, -1), np.moveaxis(x, 1, -1), k)
    d, b = r.normal(size=w.shape), np.zeros(2)
    # the conv is linear in its weights: a unit step is the derivative, to the
    # oracle's float64 rounding
    y0, y1 = O.conv2d(x, w, b), O.conv2d(x, w + d, b)
    assert abs((dy * (y1 - y0)).sum() - (dw * d).sum()) < 1e-4 * np.abs(dw * d).sum()
    assert np.allclose(dbias, dy.sum((0, 2, 3)))
