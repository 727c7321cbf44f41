"""Failure paths of the linear layers' products, without a fault, a trap or a hang:
copies or accumulators are withheld through a test hook with the wait limit at 2 ms,
so that the kernels' bounded waits run out. The call then reports
VAE_EDEVICE_TIMEOUT, and the next one, on the same memory, is right to the bit."""
import pytest
import torch

import _mlp_ref as R

pytestmark = pytest.mark.gpu
ETIMEOUT = -6


@pytest.fixture(scope="module")
def vae():
    import diffusion_vae_decoder_gb300 as pkg
    pkg.load_library()
    yield pkg
    pkg.vae_debug_inject(0)
    pkg.vae_debug_set_wait_limit(0)
    assert pkg.vae_device_error() == 0


def rand(seed, *shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


# (rows, n, k): small tiles whose reduction a cluster splits, and tiles of pairs of SMs.
# Every block adds up three accumulators of floats at least, and a pair's blocks three
# tiles of 16-bit numbers, so that one is needed again.
SMALL, SMALL_WGRAD = (300, 520, 2048), (4096, 1024, 1152)
LARGE = {"f32": (2500, 2048, 512), "bf16": (8192, 2048, 128), "f16": (8192, 2048, 128)}
LARGE_WGRAD = (8192, 2048, 512)


def make(vae, op, dtype, size):
    """The call that `op` names, with what is drawn for it."""
    t = R.DTYPES[dtype]
    rows, n, k = size
    if op == "wgrad":
        dy, x = rand(1, rows, n, dtype=t), rand(2, rows, k, dtype=t)
        return lambda: torch.cat([v.flatten() for v in vae.vae_linear_wgrad(dy, x)])
    w = rand(3, n, k, dtype=t) * k ** -0.5
    if op == "dgrad":
        # (the reduction runs over n)
        dy, z = rand(4, rows, k, dtype=t), rand(5, rows, n, dtype=t)
        wt = w.t().contiguous()
        return lambda: vae.vae_linear_dgrad(dy, wt, z=z, act=vae.VAE_ACT_GELU)
    x, bias = rand(6, rows, k, dtype=t), rand(7, n, dtype=torch.float32)
    res = rand(8, rows, n, dtype=t) if "residual" in op else None
    keep = "keep" in op

    def call():
        y, z = vae.vae_linear(x, w, bias=bias, act=vae.VAE_ACT_SILU, residual=res, keep=keep)
        return torch.cat([y, z]) if keep else y
    return call


def runs_out(vae, call, bits):
    want = call()
    assert vae.vae_device_error() == 0
    vae.vae_debug_set_wait_limit(2_000_000)
    vae.vae_debug_inject(bits)
    try:
        call()
        code = vae.vae_device_error()
    finally:
        vae.vae_debug_inject(0)
        vae.vae_debug_set_wait_limit(0)
    assert code == ETIMEOUT
    assert torch.equal(call(), want)
    assert vae.vae_device_error() == 0


def large(op, dtype):
    return LARGE_WGRAD if op == "wgrad" else LARGE[dtype]


OPS = ["linear", "linear_residual", "linear_keep", "linear_residual_keep", "dgrad", "wgrad"]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("op", OPS)
def test_copies_of_small_tiles_withheld(vae, op, dtype):
    size = SMALL_WGRAD if op == "wgrad" else SMALL
    runs_out(vae, make(vae, op, dtype, size), vae.INJECT_WITHHOLD_COPY)


@pytest.mark.parametrize("blocks", ["first", "second", "both"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("op", OPS)
def test_copies_of_pairs_withheld(vae, op, dtype, blocks):
    bits = {"first": vae.INJECT_WITHHOLD_COPY, "second": vae.INJECT_WITHHOLD_PAIR_COPY,
            "both": vae.INJECT_WITHHOLD_COPY | vae.INJECT_WITHHOLD_PAIR_COPY}[blocks]
    runs_out(vae, make(vae, op, dtype, large(op, dtype)), bits)


@pytest.mark.parametrize("op,dtype", [(op, "f32") for op in OPS] + [("wgrad", "bf16")])
def test_accumulators_of_small_tiles_withheld(vae, op, dtype):
    size = SMALL_WGRAD if op == "wgrad" else SMALL
    runs_out(vae, make(vae, op, dtype, size), vae.INJECT_WITHHOLD_ACCUMULATOR)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("op", OPS)
def test_accumulators_of_pairs_withheld(vae, op, dtype):
    runs_out(vae, make(vae, op, dtype, large(op, dtype)), vae.INJECT_WITHHOLD_ACCUMULATOR)


def test_unknown_bits_are_refused(vae):
    with pytest.raises(vae.VaeError):
        vae.vae_debug_inject(1 << 20)
