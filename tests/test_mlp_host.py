"""CPU tests of the MLP operators: the generator's published answers, the split of a
float into three bf16 parts, and every refusal of the C ABI (checks run before any
CUDA call, so that no device is needed)."""
import ctypes
import os

import numpy as np
import pytest
import torch

import _mlp_ref as R


@pytest.fixture(scope="module")
def lib():
    import diffusion_vae_decoder_gb300 as pkg
    if not os.path.exists(pkg.LIB_PATH):
        from diffusion_vae_decoder_gb300 import _build
        _build.build()
    return pkg.load_library()


# The known answers that the generator's authors publish with it.
@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
])
def test_generator_known_answers(counter, key, words):
    assert tuple(R.philox(counter, key)) == words


def test_mask_is_the_generators():
    seed, offset = 0x123456789ABCDEF0, 2 ** 32 - 2
    got = R.kept(61, 0.3, seed, offset)
    for i in range(61):
        block = offset + i // 8
        w = R.philox((block & 0xFFFFFFFF, block >> 32, 0, 0), (seed & 0xFFFFFFFF, seed >> 32))
        bits = w[i % 8 // 2] >> (16 if i % 2 else 0) & 0xFFFF
        assert got[i] == (bits >= R.threshold(0.3))


def test_mask_rate():
    # 2^20 independent draws: six deviations of sqrt(p (1 - p) / 2^20)
    for p in (0.1, 0.5, 0.9):
        rate = 1 - R.kept(2 ** 20, p, 7, 11).mean()
        assert abs(rate - p) < 6 * (p * (1 - p) / 2 ** 20) ** 0.5 + 2 ** -17


def test_three_bf16_parts_are_the_float():
    g = np.random.default_rng(3)
    bits = g.integers(0, 2 ** 32, 200000, dtype=np.uint32)
    x = torch.from_numpy(bits.view(np.float32))
    # finite, and large enough that the last part is a normal number
    x = x[torch.isfinite(x) & (x.abs() > 2.0 ** -100) & (x.abs() < 2.0 ** 127)]
    h = x.bfloat16().float()
    m = (x - h).bfloat16().float()
    lo = (x - h - m).bfloat16().float()
    assert torch.equal(h.double() + m.double() + lo.double(), x.double())
    # what the products leave out: ml + lm + ll, below 2^-24 of the product
    assert (m / x).abs().max() <= 2.0 ** -8
    assert (lo / x).abs().max() <= 2.0 ** -17


A = ctypes.c_void_p(4096)   # aligned; never read: every call is refused first
B, C = ctypes.c_void_p(8192), ctypes.c_void_p(16384)  # others, for what is written
ODD = ctypes.c_void_p(4100)
OK = {
    "vae_layer_norm": [A, 1, 8, 64, 1e-6, A, A, A, A, None],
    "vae_layer_norm_backward": [A, A, 1, A, 100000, 64, A, A, A, A, A, A, 1 << 30, None],
    "vae_dropout": [A, 1, 64, 0.1, 1, 2, None, A, A, None],
    "vae_linear": [A, 1, 8, 64, A, A, 64, 1, A, B, C, A, 1 << 30, None],
    "vae_linear_dgrad": [A, 1, 8, 64, A, 64, 1, A, B, A, 1 << 30, None],
    "vae_linear_wgrad": [A, A, 1, 8, 64, 64, B, C, A, 1 << 30, None],
}
EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -3
REFUSALS = [
    ("vae_layer_norm", 0, None, EINVAL), ("vae_layer_norm", 5, None, EINVAL),
    ("vae_layer_norm", 7, None, EINVAL), ("vae_layer_norm", 1, 3, EINVAL),
    ("vae_layer_norm", 1, -1, EINVAL), ("vae_layer_norm", 2, 0, EINVAL),
    ("vae_layer_norm", 2, -5, EINVAL), ("vae_layer_norm", 3, 0, EINVAL),
    ("vae_layer_norm", 3, 66, EUNSUPPORTED), ("vae_layer_norm", 3, 8196, EUNSUPPORTED),
    ("vae_layer_norm", 2, 2 ** 31 - 511, EUNSUPPORTED), ("vae_layer_norm", 0, ODD, EINVAL),
    ("vae_layer_norm", 5, ODD, EINVAL), ("vae_layer_norm", 8, ODD, EINVAL),
    ("vae_layer_norm_backward", 0, None, EINVAL), ("vae_layer_norm_backward", 1, None, EINVAL),
    ("vae_layer_norm_backward", 3, None, EINVAL), ("vae_layer_norm_backward", 6, None, EINVAL),
    ("vae_layer_norm_backward", 8, None, EINVAL), ("vae_layer_norm_backward", 11, None, EINVAL),
    ("vae_layer_norm_backward", 2, 7, EINVAL), ("vae_layer_norm_backward", 4, 0, EINVAL),
    ("vae_layer_norm_backward", 5, 62, EUNSUPPORTED), ("vae_layer_norm_backward", 7, ODD, EINVAL),
    ("vae_layer_norm_backward", 12, 16, EWORKSPACE),
    ("vae_dropout", 0, None, EINVAL), ("vae_dropout", 8, None, EINVAL),
    ("vae_dropout", 1, 3, EINVAL), ("vae_dropout", 2, 0, EINVAL), ("vae_dropout", 2, -8, EINVAL),
    ("vae_dropout", 3, -0.01, EINVAL), ("vae_dropout", 3, 1.01, EINVAL),
    ("vae_dropout", 3, float("nan"), EINVAL), ("vae_dropout", 0, ODD, EINVAL),
    ("vae_dropout", 6, ODD, EINVAL), ("vae_dropout", 7, ODD, EINVAL),
    ("vae_linear", 0, None, EINVAL), ("vae_linear", 4, None, EINVAL),
    ("vae_linear", 9, None, EINVAL), ("vae_linear", 1, 9, EINVAL), ("vae_linear", 7, 3, EINVAL),
    ("vae_linear", 2, 0, EINVAL), ("vae_linear", 3, -8, EINVAL), ("vae_linear", 6, 0, EINVAL),
    ("vae_linear", 3, 60, EUNSUPPORTED), ("vae_linear", 6, 12, EUNSUPPORTED),
    ("vae_linear", 3, 65544, EUNSUPPORTED), ("vae_linear", 2, 2 ** 31 - 511, EUNSUPPORTED),
    ("vae_linear", 5, ODD, EINVAL), ("vae_linear", 8, ODD, EINVAL), ("vae_linear", 10, ODD, EINVAL),
    ("vae_linear_dgrad", 0, None, EINVAL), ("vae_linear_dgrad", 4, None, EINVAL),
    ("vae_linear_dgrad", 7, None, EINVAL), ("vae_linear_dgrad", 8, None, EINVAL),
    ("vae_linear_dgrad", 6, 0, EINVAL), ("vae_linear_dgrad", 6, -1, EINVAL),
    ("vae_linear_dgrad", 3, 4, EUNSUPPORTED), ("vae_linear_dgrad", 5, 4, EUNSUPPORTED),
    ("vae_linear_dgrad", 7, ODD, EINVAL),
    ("vae_linear_wgrad", 0, None, EINVAL), ("vae_linear_wgrad", 1, None, EINVAL),
    ("vae_linear_wgrad", 6, None, EINVAL), ("vae_linear_wgrad", 2, 5, EINVAL),
    ("vae_linear_wgrad", 3, 0, EINVAL), ("vae_linear_wgrad", 4, 4, EUNSUPPORTED),
    ("vae_linear", 9, A, EINVAL), ("vae_linear", 10, A, EINVAL), ("vae_linear", 10, B, EINVAL),
    ("vae_linear_dgrad", 8, A, EINVAL), ("vae_linear_wgrad", 6, A, EINVAL),
    ("vae_linear_wgrad", 7, A, EINVAL), ("vae_linear_wgrad", 7, B, EINVAL),
    ("vae_linear_wgrad", 5, 4, EUNSUPPORTED), ("vae_linear_wgrad", 7, ODD, EINVAL),
]


@pytest.mark.parametrize("fn,at,value,status", REFUSALS)
def test_refused_before_any_launch(lib, fn, at, value, status):
    args = list(OK[fn])
    args[at] = value
    before = lib.vae_kernel_launch_count()
    assert getattr(lib, fn)(*args) == status
    assert lib.vae_kernel_launch_count() == before


@pytest.mark.parametrize("fn,at", [("vae_linear", 11), ("vae_linear_dgrad", 9),
                                   ("vae_linear_wgrad", 8)])
def test_float_products_need_their_workspace(lib, fn, at):
    args = list(OK[fn])
    args[2 if fn == "vae_linear_wgrad" else 1] = 0  # VAE_F32
    rows = 3 if fn == "vae_linear_wgrad" else 2
    args[rows] = 1024  # (a few rows of a linear layer take no workspace)
    short = list(args)
    short[at + 1] = 64
    assert getattr(lib, fn)(*short) == EWORKSPACE
    args[at] = None
    assert getattr(lib, fn)(*args) == EINVAL


def test_workspace_sizes(lib):
    assert lib.vae_linear_workspace_size(1, 1000, 64, 64) == 0
    assert lib.vae_linear_workspace_size(0, 1000, 64, 128) >= 6 * (1000 * 128 + 64 * 128)
    assert lib.vae_linear_dgrad_workspace_size(0, 1000, 64, 128) >= 6 * (1000 * 64 + 64 * 128)
    assert lib.vae_linear_wgrad_workspace_size(0, 1000, 64, 128) >= 6 * 1000 * (64 + 128)
    assert lib.vae_layer_norm_backward_workspace_size(100000, 64) > 0
    assert lib.vae_layer_norm_backward_workspace_size(1000, 64) == 0  # (one launch)
    assert lib.vae_linear_workspace_size(0, 8, 64, 64) == 0
    for bad in ((7, 10, 64, 64), (1, 0, 64, 64), (1, 10, 63, 64), (1, 10, 64, 63)):
        assert lib.vae_linear_workspace_size(*bad) == 0
        assert lib.vae_linear_dgrad_workspace_size(*bad) == 0
        assert lib.vae_linear_wgrad_workspace_size(*bad) == 0
    assert lib.vae_layer_norm_backward_workspace_size(10, 6) == 0


def test_python_checks_refuse_host_tensors(lib):
    import diffusion_vae_decoder_gb300 as vae
    x, w, g = torch.zeros(4, 8), torch.zeros(8, 8), torch.ones(8)
    for call in (lambda: vae.vae_layer_norm(x, g),
                 lambda: vae.vae_layer_norm_backward(x, x, torch.zeros(4, 2), g),
                 lambda: vae.vae_dropout(x, 0.1, seed=1),
                 lambda: vae.vae_linear(x, w),
                 lambda: vae.vae_linear_dgrad(x, w),
                 lambda: vae.vae_linear_wgrad(x, x)):
        with pytest.raises(TypeError):
            call()


class _Devices:
    """Two devices of different SM counts, and a library whose sizes depend on the current
    one's."""

    def __init__(self, monkeypatch, vae):
        self.current, self.asked = 0, []
        devices = self

        class Guard:
            def __init__(self, device):
                self.index = getattr(device, "index", device)

            def __enter__(self):
                self.before, devices.current = devices.current, self.index

            def __exit__(self, *_):
                devices.current = self.before

        class Lib:
            def sizes(self, rows, n):
                return rows * n * (devices.current + 1)
        monkeypatch.setattr(torch.cuda, "device", Guard)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: self.current, raising=False)
        monkeypatch.setattr(torch, "empty", lambda n, **kw: torch.zeros(n, dtype=torch.uint8))
        monkeypatch.setattr(vae, "_lib", Lib())
        vae._ws_bytes.cache_clear()


class _On:
    def __init__(self, index):
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.device.index


def test_workspaces_are_of_the_tensors_device(monkeypatch):
    import diffusion_vae_decoder_gb300 as vae
    devices = _Devices(monkeypatch, vae)
    try:
        for index in (0, 1, 0, 1):
            assert vae._scratch(_On(index), "sizes", 3, 5)[2] == 15 * (index + 1)
            assert vae._workspace(torch.device("cuda", index), "sizes", 7, 5)[2] == 35 * (index + 1)
            assert devices.current == 0
    finally:
        vae._ws_bytes.cache_clear()


@pytest.mark.parametrize("call", ["tokens", "dropout"])
def test_the_library_is_loaded_before_a_call_goes_on(monkeypatch, call):
    """A first call whose library does not load fails, and so does the next one; another
    thread's call meanwhile does not take the library for loaded."""
    import diffusion_vae_decoder_gb300 as vae
    loads = []

    def load(path=None):
        loads.append(dict(vae._DTYPES))
        raise RuntimeError("no library")
    monkeypatch.setattr(vae, "_DTYPES", {})
    monkeypatch.setattr(vae, "load_library", load)
    x = torch.zeros(4, 8)
    for i in range(2):
        with pytest.raises(RuntimeError, match="no library"):
            vae._tokens(x, "x") if call == "tokens" else vae.vae_dropout(x, 0.1, seed=1)
    assert loads == [{}, {}]


# Addresses of arrays that lie apart, and of one that begins inside another: 8 rows of 64
# numbers of 16 bits are 1024 bytes, 64 x 64 weights 8192, a float gradient of them 16384.
P = [ctypes.c_void_p(1 << 20 | i << 16) for i in range(1, 8)]
APART = {
    "vae_layer_norm": [P[0], 1, 8, 64, 1e-6, P[1], P[2], P[3], P[4], None],
    "vae_layer_norm_backward": [P[0], P[1], 1, P[2], 8, 64, P[3], P[4], P[5], P[6], None, None, 0,
                                None],
    "vae_dropout": [P[0], 1, 512, 0.1, 1, 2, None, P[1], P[2], None],
    "vae_linear": [P[0], 1, 8, 64, P[1], None, 64, 1, P[2], P[3], P[4], None, 0, None],
    "vae_linear_dgrad": [P[0], 1, 8, 64, P[1], 64, 1, P[2], P[3], None, 0, None],
    "vae_linear_wgrad": [P[0], P[1], 1, 8, 64, 64, P[2], P[3], P[4], 1 << 30, None],
}


def inside(p, offset):
    return ctypes.c_void_p(p.value + offset)


@pytest.mark.parametrize("fn,at,value", [
    ("vae_layer_norm", 7, inside(P[0], 128)), ("vae_layer_norm", 7, inside(P[0], -1008)),
    ("vae_layer_norm_backward", 8, inside(P[0], 16)), ("vae_layer_norm_backward", 8, inside(P[1], 16)),
    ("vae_layer_norm_backward", 8, inside(P[4], -16)),
    ("vae_dropout", 8, inside(P[0], 1008)), ("vae_dropout", 8, inside(P[1], -16)),
    ("vae_linear", 9, inside(P[0], 128)), ("vae_linear", 9, inside(P[1], 8176)),
    ("vae_linear", 9, inside(P[2], 128)), ("vae_linear", 10, inside(P[3], -128)),
    ("vae_linear", 10, inside(P[2], 16)), ("vae_linear", 10, inside(P[1], 4096)),
    ("vae_linear_dgrad", 8, inside(P[0], 1008)), ("vae_linear_dgrad", 8, inside(P[1], -1008)),
    ("vae_linear_dgrad", 8, inside(P[2], 16)),
    ("vae_linear_wgrad", 6, inside(P[0], 1008)), ("vae_linear_wgrad", 6, inside(P[1], -16368)),
    ("vae_linear_wgrad", 7, inside(P[2], 16368)), ("vae_linear_wgrad", 7, inside(P[0], 16)),
])
def test_outputs_that_begin_inside_another_array_are_refused(lib, fn, at, value):
    """(Before any launch. That arrays next to one another, and outputs that are an input
    as a whole, are taken is the GPU tests' matter.)"""
    args = list(APART[fn])
    args[at] = value
    before = lib.vae_kernel_launch_count()
    assert getattr(lib, fn)(*args) == EINVAL
    assert lib.vae_kernel_launch_count() == before
