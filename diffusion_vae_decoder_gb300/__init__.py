"""GB300 (sm_103a) FLUX-class AutoencoderKL latent decoder.

A thin ctypes binding over the C ABI in ``include/vae.h`` (``libvae.so``).
Every step of the decoder runs in this library's CUDA kernels; this module only
marshals arguments: it takes torch CUDA tensors, allocates outputs and
workspaces through torch, and passes device pointers plus the current stream.
There is no CPU fallback: if the shared library is missing or a call fails,
an exception is raised.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libvae.so")
HEADER_PATH = os.path.join(os.path.dirname(HERE), "include", "vae.h")

VAE_NCHW = 0
VAE_NHWC = 1
STATUS = {0: "VAE_OK", -1: "VAE_EINVAL", -2: "VAE_EUNSUPPORTED", -3: "VAE_EWORKSPACE",
          -4: "VAE_ECUDA", -5: "VAE_ENOTPREPARED", -6: "VAE_EDEVICE_TIMEOUT", -7: "VAE_ENOMEM"}

_lib = None


class VaeError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS.get(status, status)}")


# ---------------------------------------------------------------- ctypes mirror of vae.h
_P = ctypes.c_void_p


class ConvRef(ctypes.Structure):
    _fields_ = [("weight", _P), ("bias", _P), ("cout", ctypes.c_int), ("cin", ctypes.c_int),
                ("k", ctypes.c_int)]


class NormRef(ctypes.Structure):
    _fields_ = [("weight", _P), ("bias", _P), ("c", ctypes.c_int)]


class ResnetRef(ctypes.Structure):
    _fields_ = [("norm1", NormRef), ("conv1", ConvRef), ("norm2", NormRef), ("conv2", ConvRef),
                ("shortcut", ConvRef)]


class AttnRef(ctypes.Structure):
    _fields_ = [("norm", NormRef), ("q", ConvRef), ("k", ConvRef), ("v", ConvRef),
                ("out", ConvRef)]


class UpRef(ctypes.Structure):
    _fields_ = [("n_resnets", ctypes.c_int), ("resnets", ctypes.POINTER(ResnetRef)),
                ("upsample_conv", ConvRef)]


class ChainArgs(ctypes.Structure):
    _fields_ = [("latent_channels", ctypes.c_int), ("scaling_factor", ctypes.c_float),
                ("shift_factor", ctypes.c_float), ("groups", ctypes.c_int),
                ("eps", ctypes.c_float), ("conv_in", ConvRef), ("mid_res1", ResnetRef),
                ("mid_attn", AttnRef), ("mid_res2", ResnetRef), ("n_ups", ctypes.c_int),
                ("ups", ctypes.POINTER(UpRef)), ("norm_out", NormRef), ("conv_out", ConvRef),
                ("precision", ctypes.c_int)]


PRECISION_AUTO, PRECISION_TF32, PRECISION_SPLIT_TF32 = 0, 1, 2


class CausalDecoderArgs(ctypes.Structure):
    _fields_ = [("latent_channels", ctypes.c_int), ("scaling_factor", ctypes.c_float),
                ("shift_factor", ctypes.c_float), ("groups", ctypes.c_int),
                ("eps", ctypes.c_float), ("conv_in", ConvRef), ("n_mid", ctypes.c_int),
                ("mid", ctypes.POINTER(ResnetRef)), ("n_ups", ctypes.c_int),
                ("ups", ctypes.POINTER(UpRef)), ("norm_out", NormRef), ("conv_out", ConvRef),
                ("precision", ctypes.c_int)]


class ProfRecord(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("kernels", ctypes.c_int), ("flops", ctypes.c_double),
                ("bytes", ctypes.c_double), ("ms", ctypes.c_double)]


PROF_KINDS = {0: "conv3x3", 1: "upsample_conv", 2: "groupnorm", 3: "attention", 4: "layout",
              5: "head", 6: "groupnorm_affine"}


class TracePoint(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("c", ctypes.c_int), ("h", ctypes.c_int),
                ("w", ctypes.c_int), ("input", ctypes.c_int), ("skip", ctypes.c_int),
                ("bytes", ctypes.c_size_t)]


TRACE_KINDS = {0: "latent", 1: "conv", 2: "groupnorm", 3: "resnet", 4: "attention",
               5: "upsample", 6: "rgb"}
INJECT_WITHHOLD_STREAMK_FLAG = 1

_I, _LL, _F, _SZ = ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_size_t
_SIGS = {
    "vae_conv2d_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I, _I, _I]),
    "vae_conv2d": (_I, [_P, _I, _I, _I, _I, _I, _P, _P, _I, _I, _P, _P, _P, _P, _I, _P, _P, _SZ,
                        _P]),
    "vae_conv2d_pack_bytes": (_SZ, [_I, _I, _I, _I]),
    "vae_conv2d_pack": (_I, [_P, _P, _I, _I, _I, _P, _P, _I, _P, _SZ, _P]),
    "vae_conv2d_packed": (_I, [_P, _I, _I, _I, _I, _I, _P, _I, _I, _P, _P, _I, _P, _P, _SZ, _P]),
    "vae_upsample_conv_pack_bytes": (_SZ, [_I, _I]),
    "vae_upsample_conv_pack": (_I, [_P, _P, _I, _I, _P, _SZ, _P]),
    "vae_upsample_conv_packed": (_I, [_P, _I, _I, _I, _I, _I, _P, _I, _P, _P, _SZ, _P]),
    "vae_upsample_conv_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "vae_upsample_conv": (_I, [_P, _I, _I, _I, _I, _I, _P, _P, _I, _P, _P, _SZ, _P]),
    "vae_groupnorm_silu_workspace_size": (_SZ, [_I, _I, _LL, _I, _I]),
    "vae_groupnorm_silu": (_I, [_P, _I, _I, _LL, _I, _I, _F, _P, _P, _I, _P, _P, _SZ, _P]),
    "vae_groupnorm_silu_noalloc": (_I, [_P, _I, _I, _LL, _I, _I, _F, _P, _P, _I, _P, _P]),
    "vae_mid_attn_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "vae_mid_attn": (_I, [_P, _I, _I, _I, _I, _I, _I, _F] + [_P] * 11 + [_P, _SZ, _P]),
    "vae_conv3d_causal_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I, _I]),
    "vae_conv3d_causal": (_I, [_P, _I, _I, _I, _I, _I, _I, _P, _P, _I, _P, _P, _P, _SZ, _P]),
    "vae_causal_stack_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I, _I]),
    "vae_causal_stack": (_I, [_P, _I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(_P),
                              ctypes.POINTER(_P), ctypes.POINTER(_P), ctypes.POINTER(_P), _I, _F,
                              _P, _P, _SZ, _P]),
    "vae_chain_prepare": (_I, [ctypes.POINTER(ChainArgs), ctypes.POINTER(_P), _P]),
    "vae_chain_workspace_size": (_SZ, [_P, _I, _I, _I]),
    "vae_decode_chain": (_I, [_P, _P, _I, _I, _I, _P, _P, _SZ, _P]),
    "vae_chain_destroy": (_I, [_P]),
    "vae_status_string": (ctypes.c_char_p, [_I]),
    "vae_device_error": (_I, [_P, ctypes.POINTER(_I)]),
    "vae_num_sms": (_I, []),
    "vae_chain_profile": (_I, [_P, _I]),
    "vae_chain_profile_read": (_I, [_P, ctypes.POINTER(ProfRecord), _I, ctypes.POINTER(_I)]),
    "vae_kernel_launch_count": (_LL, []),
    "vae_chain_trace_points": (_I, [_P, _I, _I, _I, ctypes.POINTER(TracePoint), _I,
                                    ctypes.POINTER(_I)]),
    "vae_decode_chain_traced": (_I, [_P, _P, _I, _I, _I, _P, _P, _SZ, ctypes.POINTER(_P), _I,
                                     _P]),
    "vae_causal_decoder_prepare": (_I, [ctypes.POINTER(CausalDecoderArgs), ctypes.POINTER(_P),
                                        _P]),
    "vae_causal_decoder_workspace_size": (_SZ, [_P, _I, _I, _I, _I]),
    "vae_decode_causal": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "vae_chain_tiled_workspace_size": (_SZ, [_P, _I, _I, _I, _I, _I, _I]),
    "vae_decode_chain_tiled": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "vae_ckpt_bytes": (_SZ, [_LL, _I]),
    "vae_ckpt_pack": (_I, [_P, _I, _I, _LL, _I, _P, _P, _P]),
    "vae_ckpt_unpack": (_I, [_P, _P, _I, _I, _LL, _I, _P, _P]),
    "vae_groupnorm_silu_ckpt_workspace_size": (_SZ, [_I, _I, _LL, _I, _I]),
    "vae_groupnorm_silu_ckpt": (_I, [_P, _I, _I, _LL, _I, _I, _F, _P, _P, _I] + [_P] * 7 +
                                [_SZ, _P]),
    "vae_groupnorm_silu_backward_workspace_size": (_SZ, [_I, _I, _LL, _I, _I]),
    "vae_groupnorm_silu_backward": (_I, [_P] * 4 + [_I, _I, _LL, _I, _I, _P, _P, _I] + [_P] * 5 +
                                    [_SZ, _P]),
    "vae_conv2d_wgrad_workspace_size": (_SZ, [_I] * 7),
    "vae_conv2d_wgrad": (_I, [_P, _P, _P] + [_I] * 7 + [_P, _P, _P, _SZ, _P]),
    "vae_block_norm": (_I, [_P, _P, _I, _LL, _I, _F] + [_P] * 12),
    "vae_block_norm_backward_workspace_size": (_SZ, [_I, _LL, _I, _I]),
    "vae_block_norm_backward": (_I, [_P] * 7 + [_I, _LL, _I] + [_P] * 11 + [_SZ, _P]),
    "vae_measure_tf32_mma": (_I, [_I, ctypes.POINTER(ctypes.c_double),
                                  ctypes.POINTER(ctypes.c_float), _P]),
    "vae_debug_set_wait_limit": (_I, [ctypes.c_ulonglong]),
    "vae_debug_inject": (_I, [_I]),
    "vae_debug_fail_allocation": (_I, [_I]),
}


def header_symbols() -> list[str]:
    """Names of every entry point include/vae.h declares."""
    with open(HEADER_PATH) as f:
        text = f.read()
    return re.findall(r"^VAE_API\s+[\w\s\*]*?\b(vae_\w+)\s*\(", text, flags=re.M)


def load_library(path: str = LIB_PATH):
    """Load libvae.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build() "
                           "(nvcc, sm_103a); there is no fallback implementation")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(fn, status):
    if status != 0:
        raise VaeError(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, name):
    import torch
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == torch.float32
            and t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous float32 CUDA tensor")
    return t


def _ws(nbytes, device):
    import torch
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _opt(t, name):
    return None if t is None else _need(t, name)


# ---------------------------------------------------------------- single ops
def vae_conv2d(x, weight, bias=None, residual=None, sc_x=None, sc_w=None, sc_b=None,
               layout=VAE_NCHW, out=None, stream=None):
    lib = load_library()
    _need(x, "x"), _need(weight, "weight")
    bias, residual, sc_x, sc_b = (_opt(bias, "bias"), _opt(residual, "residual"),
                                  _opt(sc_x, "sc_x"), _opt(sc_b, "sc_b"))
    if layout == VAE_NCHW:
        n, cin, h, w = x.shape
    else:
        n, h, w, cin = x.shape
    cout, _, k, _ = weight.shape
    sc_cin = 0
    if sc_w is not None:
        sc_w = _need(sc_w.reshape(sc_w.shape[0], -1).contiguous(), "sc_w")
        sc_cin = sc_w.shape[1]
    shape = (n, cout, h, w) if layout == VAE_NCHW else (n, h, w, cout)
    if out is None:
        import torch
        out = torch.empty(shape, dtype=torch.float32, device=x.device)
    ws_bytes = lib.vae_conv2d_workspace_size(n, cin, h, w, layout, cout, k, sc_cin)
    ws = _ws(ws_bytes, x.device)
    _check("vae_conv2d", lib.vae_conv2d(
        _ptr(x), n, cin, h, w, layout, _ptr(weight), _ptr(bias), cout, k, _ptr(residual),
        _ptr(sc_x), _ptr(sc_w), _ptr(sc_b), sc_cin, _ptr(out), _ptr(ws), ws.numel(),
        _stream(stream)))
    return out


class PackedWeights:
    """A conv's weights packed once on the device (vae_conv2d_pack /
    vae_upsample_conv_pack): the byte buffer and the sizes it was made for."""

    def __init__(self, kind, buf, cout, cin, k, sc_cin):
        self.kind, self.buf = kind, buf
        self.cout, self.cin, self.k, self.sc_cin = cout, cin, k, sc_cin


def vae_conv2d_pack(weight, bias=None, sc_w=None, sc_b=None, stream=None):
    import torch
    lib = load_library()
    _need(weight, "weight")
    bias, sc_b = _opt(bias, "bias"), _opt(sc_b, "sc_b")
    cout, cin, k, _ = weight.shape
    sc_cin = 0
    if sc_w is not None:
        sc_w = _need(sc_w.reshape(sc_w.shape[0], -1).contiguous(), "sc_w")
        sc_cin = sc_w.shape[1]
    nbytes = lib.vae_conv2d_pack_bytes(cout, cin, k, sc_cin)
    buf = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=weight.device)
    _check("vae_conv2d_pack", lib.vae_conv2d_pack(
        _ptr(weight), _ptr(bias), cout, cin, k, _ptr(sc_w), _ptr(sc_b), sc_cin, _ptr(buf),
        buf.numel(), _stream(stream)))
    return PackedWeights("conv2d", buf, cout, cin, k, sc_cin)


def vae_conv2d_packed(x, pack, residual=None, sc_x=None, layout=VAE_NCHW, out=None, stream=None):
    lib = load_library()
    _need(x, "x")
    residual, sc_x = _opt(residual, "residual"), _opt(sc_x, "sc_x")
    if pack.kind != "conv2d":
        raise TypeError("pack was not made by vae_conv2d_pack")
    if layout == VAE_NCHW:
        n, cin, h, w = x.shape
    else:
        n, h, w, cin = x.shape
    cout, k = pack.cout, pack.k
    shape = (n, cout, h, w) if layout == VAE_NCHW else (n, h, w, cout)
    if out is None:
        import torch
        out = torch.empty(shape, dtype=torch.float32, device=x.device)
    ws = _ws(lib.vae_conv2d_workspace_size(n, cin, h, w, layout, cout, k, pack.sc_cin), x.device)
    _check("vae_conv2d_packed", lib.vae_conv2d_packed(
        _ptr(x), n, cin, h, w, layout, _ptr(pack.buf), cout, k, _ptr(residual), _ptr(sc_x),
        pack.sc_cin, _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def vae_upsample_conv_pack(weight, bias=None, stream=None):
    import torch
    lib = load_library()
    _need(weight, "weight")
    bias = _opt(bias, "bias")
    cout, cin = weight.shape[0], weight.shape[1]
    nbytes = lib.vae_upsample_conv_pack_bytes(cout, cin)
    buf = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=weight.device)
    _check("vae_upsample_conv_pack", lib.vae_upsample_conv_pack(
        _ptr(weight), _ptr(bias), cout, cin, _ptr(buf), buf.numel(), _stream(stream)))
    return PackedWeights("upsample_conv", buf, cout, cin, 3, 0)


def vae_upsample_conv_packed(x, pack, layout=VAE_NCHW, out=None, stream=None):
    lib = load_library()
    _need(x, "x")
    if pack.kind != "upsample_conv":
        raise TypeError("pack was not made by vae_upsample_conv_pack")
    if layout == VAE_NCHW:
        n, cin, h, w = x.shape
    else:
        n, h, w, cin = x.shape
    cout = pack.cout
    shape = (n, cout, 2 * h, 2 * w) if layout == VAE_NCHW else (n, 2 * h, 2 * w, cout)
    if out is None:
        import torch
        out = torch.empty(shape, dtype=torch.float32, device=x.device)
    ws = _ws(lib.vae_upsample_conv_workspace_size(n, cin, h, w, layout, cout), x.device)
    _check("vae_upsample_conv_packed", lib.vae_upsample_conv_packed(
        _ptr(x), n, cin, h, w, layout, _ptr(pack.buf), cout, _ptr(out), _ptr(ws), ws.numel(),
        _stream(stream)))
    return out


def vae_upsample_conv(x, weight, bias=None, layout=VAE_NCHW, out=None, stream=None):
    lib = load_library()
    _need(x, "x"), _need(weight, "weight")
    bias = _opt(bias, "bias")
    if layout == VAE_NCHW:
        n, cin, h, w = x.shape
    else:
        n, h, w, cin = x.shape
    cout = weight.shape[0]
    shape = (n, cout, 2 * h, 2 * w) if layout == VAE_NCHW else (n, 2 * h, 2 * w, cout)
    if out is None:
        import torch
        out = torch.empty(shape, dtype=torch.float32, device=x.device)
    ws = _ws(lib.vae_upsample_conv_workspace_size(n, cin, h, w, layout, cout), x.device)
    _check("vae_upsample_conv", lib.vae_upsample_conv(
        _ptr(x), n, cin, h, w, layout, _ptr(weight), _ptr(bias), cout, _ptr(out), _ptr(ws),
        ws.numel(), _stream(stream)))
    return out


def vae_groupnorm_silu(x, gamma, beta, groups=32, eps=1e-6, apply_silu=True, layout=VAE_NCHW,
                       out=None, stream=None):
    lib = load_library()
    _need(x, "x"), _need(gamma, "gamma"), _need(beta, "beta")
    n = x.shape[0]
    if layout == VAE_NCHW:
        c = x.shape[1]
        spatial = x.numel() // (n * c)
    else:
        c = x.shape[-1]
        spatial = x.numel() // (n * c)
    if out is None:
        import torch
        out = torch.empty_like(x)
    ws = _ws(lib.vae_groupnorm_silu_workspace_size(n, c, spatial, layout, groups), x.device)
    _check("vae_groupnorm_silu", lib.vae_groupnorm_silu(
        _ptr(x), n, c, spatial, layout, groups, eps, _ptr(gamma), _ptr(beta), int(apply_silu),
        _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def vae_groupnorm_silu_noalloc(x, gamma, beta, groups=32, eps=1e-6, apply_silu=True,
                               layout=VAE_NCHW, out=None, stream=None):
    """GroupNorm(+SiLU) whose scratch is a fixed array inside the library (no
    workspace); for callers that must not allocate device memory."""
    lib = load_library()
    _need(x, "x"), _need(gamma, "gamma"), _need(beta, "beta")
    n = x.shape[0]
    c = x.shape[1] if layout == VAE_NCHW else x.shape[-1]
    spatial = x.numel() // (n * c)
    if out is None:
        import torch
        out = torch.empty_like(x)
    _check("vae_groupnorm_silu_noalloc", lib.vae_groupnorm_silu_noalloc(
        _ptr(x), n, c, spatial, layout, groups, eps, _ptr(gamma), _ptr(beta), int(apply_silu),
        _ptr(out), _stream(stream)))
    return out


def vae_mid_attn(x, p, groups=32, eps=1e-6, layout=VAE_NCHW, out=None, stream=None):
    """``p``: dict with group_norm / to_q / to_k / to_v / to_out -> (weight, bias)."""
    lib = load_library()
    _need(x, "x")
    if layout == VAE_NCHW:
        n, c, h, w = x.shape
    else:
        n, h, w, c = x.shape
    ptrs = []
    for key in ("group_norm", "to_q", "to_k", "to_v", "to_out"):
        wt, b = p[key]
        ptrs += [_ptr(_need(wt, key)), _ptr(_need(b, key))]
    if out is None:
        import torch
        out = torch.empty_like(x)
    ws = _ws(lib.vae_mid_attn_workspace_size(n, c, h, w, layout), x.device)
    _check("vae_mid_attn", lib.vae_mid_attn(
        _ptr(x), n, c, h, w, layout, groups, eps, *ptrs, _ptr(out), _ptr(ws), ws.numel(),
        _stream(stream)))
    return out


def vae_conv3d_causal(x, weight, bias=None, residual=None, layout=VAE_NCHW, out=None,
                      stream=None):
    lib = load_library()
    _need(x, "x"), _need(weight, "weight")
    bias, residual = _opt(bias, "bias"), _opt(residual, "residual")
    if layout == VAE_NCHW:
        n, cin, t, h, w = x.shape
    else:
        n, t, h, w, cin = x.shape
    cout = weight.shape[0]
    shape = (n, cout, t, h, w) if layout == VAE_NCHW else (n, t, h, w, cout)
    if out is None:
        import torch
        out = torch.empty(shape, dtype=torch.float32, device=x.device)
    ws = _ws(lib.vae_conv3d_causal_workspace_size(n, cin, t, h, w, layout, cout), x.device)
    _check("vae_conv3d_causal", lib.vae_conv3d_causal(
        _ptr(x), n, cin, t, h, w, layout, _ptr(weight), _ptr(bias), cout, _ptr(residual),
        _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def vae_kernel_launch_count():
    return load_library().vae_kernel_launch_count()


def vae_causal_stack(x, layers, groups=32, eps=1e-6, layout=VAE_NCHW, out=None, stream=None):
    """``layers``: list of dicts with weight [c,c,3,3,3], bias, gn_weight, gn_bias (CUDA)."""
    lib = load_library()
    _need(x, "x")
    if layout == VAE_NCHW:
        n, c, t, h, w = x.shape
    else:
        n, t, h, w, c = x.shape
    L = len(layers)
    arr = lambda key: (_P * L)(*[_need(d[key], key).data_ptr() for d in layers])  # noqa: E731
    if out is None:
        import torch
        out = torch.empty_like(x)
    ws = _ws(lib.vae_causal_stack_workspace_size(n, c, t, h, w, layout, L), x.device)
    _check("vae_causal_stack", lib.vae_causal_stack(
        _ptr(x), n, c, t, h, w, layout, L, arr("weight"), arr("bias"), arr("gn_weight"),
        arr("gn_bias"), groups, eps, _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return out


# ---------------------------------------------------------------- training operators
# These are called many times a step on tensors whose kernels take a few
# microseconds, so the checks are one short call per tensor. Like the other entry
# points they are outside autograd: results carry no graph, and a training step calls
# the forward and the backward operators itself (or from an autograd.Function).
class Checkpoint:
    """An 8-bit activation checkpoint of ``rows`` pixels or tokens of ``c``
    channels: ``payload`` [rows, cp] (float8_e4m3fn, cp = c rounded up to 32) and
    ``scale`` [rows, cp / 32] (float8_e8m0fnu); a value is payload * scale of its
    block of 32 channels. Made by the operators that keep one, or around the
    bytes of one (payload first, scales at the next multiple of 256 bytes;
    vae_ckpt_bytes long, 16-byte aligned)."""

    __slots__ = ("rows", "c", "_bytes", "_payload", "_scale")

    def __init__(self, buf, rows, c):
        import torch
        if not (isinstance(buf, torch.Tensor) and buf.is_cuda and buf.dtype == torch.uint8
                and buf.is_contiguous()):
            raise TypeError("buf must be a contiguous uint8 CUDA tensor")
        if rows <= 0 or c <= 0 or buf.numel() < self.nbytes(rows, c):
            raise ValueError(f"buf holds no checkpoint of {rows} rows of {c} channels")
        self.rows, self.c = rows, c
        self._bytes, self._payload, self._scale = buf, None, None

    @staticmethod
    def nbytes(rows, c):
        cp = (c + 31) // 32 * 32
        return (rows * cp + 255) // 256 * 256 + rows * (cp // 32)

    @classmethod
    def _make(cls, rows, c, device):
        import torch
        self = cls.__new__(cls)
        self.rows, self.c, self._bytes = rows, c, None
        cp = (c + 31) // 32 * 32
        self._payload = torch.empty((rows, cp), dtype=torch.float8_e4m3fn, device=device)
        self._scale = torch.empty((rows, cp // 32), dtype=torch.float8_e8m0fnu, device=device)
        return self

    def _split(self):
        import torch
        cp = (self.c + 31) // 32 * 32
        at, n = (self.rows * cp + 255) // 256 * 256, self.rows * (cp // 32)
        self._payload = self._bytes[:self.rows * cp].view(torch.float8_e4m3fn).view(self.rows, cp)
        self._scale = self._bytes[at:at + n].view(torch.float8_e8m0fnu).view(self.rows, cp // 32)

    @property
    def payload(self):
        if self._payload is None:
            self._split()
        return self._payload

    @property
    def scale(self):
        if self._scale is None:
            self._split()
        return self._scale

    @property
    def device(self):
        return (self._payload if self._bytes is None else self._bytes).device

    def _addresses(self):
        if self._bytes is None:
            return self._payload.data_ptr(), self._scale.data_ptr()
        at = self._bytes.data_ptr()
        return at, at + (self.rows * ((self.c + 31) // 32 * 32) + 255) // 256 * 256


def _refuse(t, shape, device, name):
    """Why `_at` does not take `t`."""
    _need(t, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    raise ValueError(f"{name} is on {t.device}, not {device}")


def _at(t, shape, device, name):
    """The address of a contiguous float32 tensor of `shape` on `device`."""
    try:
        if (t.dtype is _F32 and t.shape == shape and t.device == device
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, shape, device, name)


def _at_opt(t, shape, device, name):
    return None if t is None else _at(t, shape, device, name)


def _ckpt_at(k, rows, c, device, name):
    """The addresses of a checkpoint's payload and scales."""
    if not isinstance(k, Checkpoint):
        raise TypeError(f"{name} must be a Checkpoint")
    if k.rows != rows or k.c != c:
        raise ValueError(f"{name} holds {k.rows} rows of {k.c} channels, not {rows} of {c}")
    if k.device != device:
        raise ValueError(f"{name} is on {k.device}, not {device}")
    return k._addresses()


_F32 = None  # torch.float32, once torch is loaded


def _first(x, name):
    """(shape, device) of the tensor the others are compared with."""
    import torch
    global _F32
    _F32 = torch.float32
    if not (isinstance(x, torch.Tensor) and x.is_cuda):
        _need(x, name)
    return x.shape, x.device


def _dims(shape, layout):
    """(n, c, spatial) of an activation."""
    if len(shape) < 3:
        raise ValueError("an activation has at least three axes")
    if layout == VAE_NCHW:
        n, c, *rest = shape
    elif layout == VAE_NHWC:
        n, *rest, c = shape
    else:
        raise VaeError("layout", -1)
    spatial = 1
    for v in rest:
        spatial *= v
    return n, c, spatial


def _call(name, device, *args):
    """Calls entry point `name` with `args` and the current stream of `device`."""
    import torch
    fn = getattr(_lib, name)
    index = device.index
    raw = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            status = fn(*args, raw)
    if status != 0:
        raise VaeError(name, status)


def _memory(*values):
    """The tensors that hold `values`: tensors, checkpoints, and tuples and dicts of
    them; other values hold none."""
    todo = list(values)
    while todo:
        v = todo.pop()
        if isinstance(v, (tuple, dict)):
            todo += v.values() if isinstance(v, dict) else v
        elif isinstance(v, Checkpoint):
            todo += (v._payload, v._scale) if v._bytes is None else (v._bytes,)
        elif hasattr(v, "record_stream"):
            yield v


def _on(stream, fn, *args):
    """fn(*args) with `stream` current. The memory it allocates is the stream's, so
    nothing pending on the caller's current stream still uses it; what it returns
    is not reused before that stream's work has passed it, and neither is what it was
    given before `stream` has, so that temporaries may be passed."""
    import torch
    device = next((a.device for a in args if hasattr(a, "device")), stream.device)
    if device != stream.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    here = torch.cuda.current_stream(device)
    if stream != here:
        for t in _memory(*args):
            if t.device == device:  # (fn refuses the others)
                t.record_stream(stream)
    with torch.cuda.stream(stream):
        out = fn(*args)
    if stream != here:
        for t in _memory(out):
            t.record_stream(here)
    return out


@functools.lru_cache(maxsize=4096)
def _ws_bytes(name, *args):
    return getattr(load_library(), name)(*args)


def _workspace(device, name, *args):
    """(tensor, address, bytes) of an operator's workspace; Nones when it takes none."""
    import torch
    nbytes = _ws_bytes(name, *args)
    if not nbytes:
        return None, None, 0
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws, ws.data_ptr(), nbytes


def vae_ckpt_pack(x, layout=VAE_NHWC, stream=None):
    """A Checkpoint of the activation ``x`` (any number of spatial axes)."""
    if stream is not None:
        return _on(stream, vae_ckpt_pack, x, layout)
    load_library()
    shape, dev = _first(x, "x")
    n, c, spatial = _dims(shape, layout)
    at = _at(x, shape, dev, "x")
    k = Checkpoint._make(n * spatial, c, dev)
    _call("vae_ckpt_pack", dev, at, n, c, spatial, layout, *k._addresses())
    return k


def vae_ckpt_unpack(ckpt, shape, layout=VAE_NHWC, stream=None):
    """The float32 activation of ``shape`` (in ``layout``) that ``ckpt`` holds."""
    import torch
    if stream is not None:
        return _on(stream, vae_ckpt_unpack, ckpt, shape, layout)
    load_library()
    if not isinstance(ckpt, Checkpoint):
        raise TypeError("ckpt must be a Checkpoint")
    n, c, spatial = _dims(shape, layout)
    dev = ckpt.device
    pq, ps = _ckpt_at(ckpt, n * spatial, c, dev, "ckpt")
    out = torch.empty(shape, dtype=torch.float32, device=dev)
    _call("vae_ckpt_unpack", dev, pq, ps, n, c, spatial, layout, out.data_ptr())
    return out


def vae_groupnorm_silu_ckpt(x, gamma, beta, groups=32, eps=1e-6, apply_silu=True,
                            layout=VAE_NCHW, out=None, keep_x=True, keep_y=True, stream=None):
    """vae_groupnorm_silu that keeps its backward pass's inputs: returns
    (y, x_ckpt, y_ckpt, stats), a checkpoint None where keep_x / keep_y is
    false, stats [n, groups, 2] (mean, 1 / sqrt(var + eps))."""
    import torch
    if stream is not None:
        return _on(stream, vae_groupnorm_silu_ckpt, x, gamma, beta, groups, eps, apply_silu, layout,
                   out, keep_x, keep_y)
    load_library()
    shape, dev = _first(x, "x")
    n, c, spatial = _dims(shape, layout)
    px = _at(x, shape, dev, "x")
    pg, pb = _at(gamma, (c,), dev, "gamma"), _at(beta, (c,), dev, "beta")
    y = torch.empty_like(x) if out is None else out
    py = y.data_ptr() if out is None else _at(out, shape, dev, "out")
    ws, pw, nw = _workspace(dev, "vae_groupnorm_silu_ckpt_workspace_size", n, c, spatial, layout,
                            groups)
    x_ckpt = y_ckpt = pxq = pxs = pyq = pys = None
    if keep_x:
        x_ckpt = Checkpoint._make(n * spatial, c, dev)
        pxq, pxs = x_ckpt._addresses()
    if keep_y:
        y_ckpt = Checkpoint._make(n * spatial, c, dev)
        pyq, pys = y_ckpt._addresses()
    stats = torch.empty((n, max(groups, 1), 2), dtype=torch.float32, device=dev)
    _call("vae_groupnorm_silu_ckpt", dev, px, n, c, spatial, layout, groups, eps, pg, pb,
          bool(apply_silu), py, pxq, pxs, pyq, pys, stats.data_ptr(), pw, nw)
    return y, x_ckpt, y_ckpt, stats


def vae_groupnorm_silu_backward(dy, x_ckpt, stats, gamma, beta, groups=32, apply_silu=True,
                                layout=VAE_NCHW, dres=None, out=None, stream=None):
    """(dx, dgamma, dbeta) from dy and what vae_groupnorm_silu_ckpt kept; dres, a
    further gradient of x (the resnet skip's), is added to dx."""
    import torch
    if stream is not None:
        return _on(stream, vae_groupnorm_silu_backward, dy, x_ckpt, stats, gamma, beta, groups,
                   apply_silu, layout, dres, out)
    load_library()
    shape, dev = _first(dy, "dy")
    n, c, spatial = _dims(shape, layout)
    pd = _at(dy, shape, dev, "dy")
    pq, pk = _ckpt_at(x_ckpt, n * spatial, c, dev, "x_ckpt")
    ps = _at(stats, (n, groups, 2), dev, "stats")
    pg, pb = _at(gamma, (c,), dev, "gamma"), _at(beta, (c,), dev, "beta")
    pr = _at_opt(dres, shape, dev, "dres")
    dx = torch.empty_like(dy) if out is None else out
    px = dx.data_ptr() if out is None else _at(out, shape, dev, "out")
    ws, pw, nw = _workspace(dev, "vae_groupnorm_silu_backward_workspace_size", n, c, spatial,
                            layout, groups)
    dgamma = torch.empty_like(gamma)
    dbeta = torch.empty_like(beta)
    _call("vae_groupnorm_silu_backward", dev, pd, pq, pk, ps, n, c, spatial, layout, groups, pg,
          pb, bool(apply_silu), pr, px, dgamma.data_ptr(), dbeta.data_ptr(), pw, nw)
    return dx, dgamma, dbeta


def vae_conv2d_wgrad(dy, x_ckpt, k, layout=VAE_NCHW, stream=None):
    """(dw [cout, cin, k, k], dbias [cout]) of vae_conv2d from its output's
    gradient and the checkpoint of its input."""
    import torch
    if stream is not None:
        return _on(stream, vae_conv2d_wgrad, dy, x_ckpt, k, layout)
    load_library()
    shape, dev = _first(dy, "dy")
    if len(shape) != 4:
        raise ValueError("dy must have four axes")
    if layout == VAE_NCHW:
        n, cout, h, w = shape
    else:
        n, h, w, cout = shape
    pd = _at(dy, shape, dev, "dy")
    cin = getattr(x_ckpt, "c", 0)
    pq, pk = _ckpt_at(x_ckpt, n * h * w, cin, dev, "x_ckpt")
    ws, pw, nw = _workspace(dev, "vae_conv2d_wgrad_workspace_size", n, cin, h, w, layout, cout, k)
    dw = torch.empty((cout, cin, k, k), dtype=torch.float32, device=dev)
    dbias = torch.empty(cout, dtype=torch.float32, device=dev)
    _call("vae_conv2d_wgrad", dev, pd, pq, pk, n, cin, h, w, layout, cout, k, dw.data_ptr(),
          dbias.data_ptr(), pw, nw)
    return dw, dbias


def vae_block_norm(u, x, w_post, gate=None, scale=None, w_pre=None, eps=1e-6, keep=True,
                   out_h=None, out_y=None, stream=None):
    """The norms around a transformer block on tokens u, x [n, tokens, c]:
    h = x + gate * scale * w_post * u / rms(u), y = w_pre * h / rms(h). Returns
    (h, y, u_ckpt, h_ckpt, rstd); y and h_ckpt are None without w_pre, and the
    last three None with keep=False (serving)."""
    import torch
    if stream is not None:
        return _on(stream, vae_block_norm, u, x, w_post, gate, scale, w_pre, eps, keep, out_h,
                   out_y)
    load_library()
    shape, dev = _first(u, "u")
    if len(shape) != 3:
        raise ValueError("u must be [n, tokens, c]")
    n, tokens, c = shape
    pu, px = _at(u, shape, dev, "u"), _at(x, shape, dev, "x")
    po, pg = _at(w_post, (c,), dev, "w_post"), _at_opt(gate, (n, c), dev, "gate")
    ps, pp = _at_opt(scale, (c,), dev, "scale"), _at_opt(w_pre, (c,), dev, "w_pre")
    h = torch.empty_like(u) if out_h is None else out_h
    ph = h.data_ptr() if out_h is None else _at(out_h, shape, dev, "out_h")
    y = py = None
    if w_pre is not None:
        y = torch.empty_like(u) if out_y is None else out_y
        py = y.data_ptr() if out_y is None else _at(out_y, shape, dev, "out_y")
    elif out_y is not None:
        raise ValueError("out_y without w_pre")
    u_ckpt = h_ckpt = rstd = puq = pus = phq = phs = pr = None
    if keep:
        u_ckpt = Checkpoint._make(n * tokens, c, dev)
        puq, pus = u_ckpt._addresses()
        rstd = torch.empty((2, n * tokens), dtype=torch.float32, device=dev)
        pr = rstd.data_ptr()
        if w_pre is not None:
            h_ckpt = Checkpoint._make(n * tokens, c, dev)
            phq, phs = h_ckpt._addresses()
    _call("vae_block_norm", dev, pu, px, n, tokens, c, eps, po, pg, ps, pp, ph, py, puq, pus, phq,
          phs, pr)
    return h, y, u_ckpt, h_ckpt, rstd


def vae_block_norm_backward(dy, dh, u_ckpt, h_ckpt, rstd, w_post, gate=None, scale=None,
                            w_pre=None, stream=None):
    """The gradients of vae_block_norm, as a dict: du, dx, dw_post, and dgate,
    dscale, dw_pre (None for an absent input). dy is None without w_pre; dh, the
    gradient that reaches h by the residual stream, may be None."""
    import torch
    if stream is not None:
        return _on(stream, vae_block_norm_backward, dy, dh, u_ckpt, h_ckpt, rstd, w_post, gate,
                   scale, w_pre)
    load_library()
    like, name = (dh, "dh") if dy is None else (dy, "dy")
    if like is None:
        raise ValueError("dy and dh are both None")
    shape, dev = _first(like, name)
    if len(shape) != 3:
        raise ValueError("gradients must be [n, tokens, c]")
    if (dy is None) != (w_pre is None) or (h_ckpt is None) != (w_pre is None):
        raise ValueError("dy and h_ckpt go with w_pre")
    n, tokens, c = shape
    pdy, pdh = _at_opt(dy, shape, dev, "dy"), _at_opt(dh, shape, dev, "dh")
    puq, pus = _ckpt_at(u_ckpt, n * tokens, c, dev, "u_ckpt")
    phq, phs = (None, None) if h_ckpt is None else _ckpt_at(h_ckpt, n * tokens, c, dev, "h_ckpt")
    pr, po = _at(rstd, (2, n * tokens), dev, "rstd"), _at(w_post, (c,), dev, "w_post")
    pg, ps = _at_opt(gate, (n, c), dev, "gate"), _at_opt(scale, (c,), dev, "scale")
    pp = _at_opt(w_pre, (c,), dev, "w_pre")
    ws, pw, nw = _workspace(dev, "vae_block_norm_backward_workspace_size", n, tokens, c,
                            int(gate is not None))
    du, dx, dw_post = torch.empty_like(like), torch.empty_like(like), torch.empty_like(w_post)
    dgate = None if gate is None else torch.empty_like(gate)
    dscale = None if scale is None else torch.empty_like(scale)
    dw_pre = None if w_pre is None else torch.empty_like(w_pre)
    _call("vae_block_norm_backward", dev, pdy, pdh, puq, pus, phq, phs, pr, n, tokens, c, po, pg,
          ps, pp, du.data_ptr(), dx.data_ptr(), dw_post.data_ptr(), _ptr(dgate), _ptr(dscale),
          _ptr(dw_pre), pw, nw)
    return dict(du=du, dx=dx, dw_post=dw_post, dgate=dgate, dscale=dscale, dw_pre=dw_pre)


def vae_measure_tf32_mma(iters, stream=None):
    """(TFLOP/s, ms, flops) of the tensor-pipe TF32 MMA loop (vae_measure_tf32_mma)."""
    flops, ms = ctypes.c_double(0), ctypes.c_float(0)
    _check("vae_measure_tf32_mma", load_library().vae_measure_tf32_mma(
        int(iters), ctypes.byref(flops), ctypes.byref(ms), _stream(stream)))
    return flops.value / (ms.value / 1e3) / 1e12, ms.value, flops.value


def vae_debug_set_wait_limit(ns):
    _check("vae_debug_set_wait_limit", load_library().vae_debug_set_wait_limit(int(ns)))


def vae_debug_inject(bits):
    _check("vae_debug_inject", load_library().vae_debug_inject(int(bits)))


def vae_debug_fail_allocation(nth):
    _check("vae_debug_fail_allocation", load_library().vae_debug_fail_allocation(int(nth)))


def vae_device_error(stream=None):
    lib = load_library()
    code = ctypes.c_int(0)
    _check("vae_device_error", lib.vae_device_error(_stream(stream), ctypes.byref(code)))
    return code.value


# ---------------------------------------------------------------- the chain
def _conv_ref(weights, name, keep):
    w = weights.get(name + ".weight")
    if w is None:
        return ConvRef()
    import numpy as np
    w = np.ascontiguousarray(w, dtype=np.float32)
    b = np.ascontiguousarray(weights[name + ".bias"], dtype=np.float32)
    keep += [w, b]
    return ConvRef(w.ctypes.data, b.ctypes.data, w.shape[0], w.shape[1],
                   w.shape[2] if w.ndim == 4 else 1)


def _norm_ref(weights, name, keep):
    import numpy as np
    g = np.ascontiguousarray(weights[name + ".weight"], dtype=np.float32)
    b = np.ascontiguousarray(weights[name + ".bias"], dtype=np.float32)
    keep += [g, b]
    return NormRef(g.ctypes.data, b.ctypes.data, g.shape[0])


def _resnet_ref(weights, pre, keep):
    return ResnetRef(_norm_ref(weights, pre + ".norm1", keep), _conv_ref(weights, pre + ".conv1", keep),
                     _norm_ref(weights, pre + ".norm2", keep), _conv_ref(weights, pre + ".conv2", keep),
                     _conv_ref(weights, pre + ".conv_shortcut", keep))


class VaeChain:
    """Prepared decoder (vae_chain_prepare / vae_decode_chain / vae_chain_destroy).

    ``weights`` maps diffusers-style names (conv_in.weight, mid.resnets.0...,
    mid.attentions.0.to_q.weight, up_blocks.{i}.resnets.{j}..., ...,
    conv_norm_out.weight, conv_out.weight) to host float32 arrays.
    ``precision``: PRECISION_AUTO (split-TF32 products for decodes with little
    conv work, TF32 otherwise), PRECISION_TF32 or PRECISION_SPLIT_TF32."""

    def __init__(self, weights, n_up_blocks, resnets_per_block=3, latent_channels=16,
                 scaling_factor=0.3611, shift_factor=0.1159, groups=32, eps=1e-6, stream=None,
                 precision=PRECISION_AUTO):
        lib = load_library()
        keep = []
        ups = []
        self._res_arrays = []
        for i in range(n_up_blocks):
            res = (ResnetRef * resnets_per_block)(*[
                _resnet_ref(weights, f"up_blocks.{i}.resnets.{j}", keep)
                for j in range(resnets_per_block)])
            self._res_arrays.append(res)
            ups.append(UpRef(resnets_per_block, res,
                             _conv_ref(weights, f"up_blocks.{i}.upsamplers.0.conv", keep)))
        ups_arr = (UpRef * max(1, n_up_blocks))(*ups)
        a = "mid.attentions.0"
        attn = AttnRef(_norm_ref(weights, a + ".group_norm", keep),
                       *[_conv_ref(weights, f"{a}.{p}", keep)
                         for p in ("to_q", "to_k", "to_v", "to_out")])
        for r in (attn.q, attn.k, attn.v, attn.out):
            r.k = 1
        args = ChainArgs(latent_channels, scaling_factor, shift_factor, groups, eps,
                         _conv_ref(weights, "conv_in", keep),
                         _resnet_ref(weights, "mid.resnets.0", keep), attn,
                         _resnet_ref(weights, "mid.resnets.1", keep), n_up_blocks, ups_arr,
                         _norm_ref(weights, "conv_norm_out", keep),
                         _conv_ref(weights, "conv_out", keep), int(precision))
        h = ctypes.c_void_p()
        _check("vae_chain_prepare", lib.vae_chain_prepare(ctypes.byref(args), ctypes.byref(h),
                                                          _stream(stream)))
        self.handle = h
        self.latent_channels = latent_channels
        self.out_channels = weights["conv_out.weight"].shape[0]
        self.up_factor = 2 ** sum(1 for i in range(n_up_blocks)
                                  if f"up_blocks.{i}.upsamplers.0.conv.weight" in weights)

    def workspace_size(self, n, h, w):
        return load_library().vae_chain_workspace_size(self.handle, n, h, w)

    def decode(self, z, out=None, ws=None, stream=None):
        lib = load_library()
        _need(z, "z")
        n, c, h, w = z.shape
        if out is None:
            import torch
            f = self.up_factor
            out = torch.empty((n, self.out_channels, f * h, f * w), dtype=torch.float32,
                              device=z.device)
        if ws is None:
            ws = _ws(self.workspace_size(n, h, w), z.device)
        _check("vae_decode_chain", lib.vae_decode_chain(
            self.handle, _ptr(z), n, h, w, _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
        return out

    def decode_tiled(self, z, tile=512, min_overlap=64, tiles_per_batch=0, out=None, ws=None,
                     stream=None):
        """vae_decode_chain_tiled: decode in overlapping tiles of ``tile``
        output pixels, cross-faded over their overlaps."""
        lib = load_library()
        _need(z, "z")
        n, c, h, w = z.shape
        if out is None:
            import torch
            f = self.up_factor
            out = torch.empty((n, self.out_channels, f * h, f * w), dtype=torch.float32,
                              device=z.device)
        if ws is None:
            nb = lib.vae_chain_tiled_workspace_size(self.handle, n, h, w, tile, min_overlap,
                                                    tiles_per_batch)
            if nb == 0:
                raise VaeError("vae_chain_tiled_workspace_size", -1)
            ws = _ws(nb, z.device)
        _check("vae_decode_chain_tiled", lib.vae_decode_chain_tiled(
            self.handle, _ptr(z), n, h, w, tile, min_overlap, tiles_per_batch, _ptr(out),
            _ptr(ws), ws.numel(), _stream(stream)))
        return out

    def trace_points(self, n, h, w):
        """The decode's trace points (vae_chain_trace_points) as dicts."""
        lib = load_library()
        cnt = ctypes.c_int(0)
        _check("vae_chain_trace_points", lib.vae_chain_trace_points(
            self.handle, n, h, w, None, 0, ctypes.byref(cnt)))
        arr = (TracePoint * max(1, cnt.value))()
        _check("vae_chain_trace_points", lib.vae_chain_trace_points(
            self.handle, n, h, w, arr, cnt.value, ctypes.byref(cnt)))
        return [dict(kind=TRACE_KINDS[p.kind], c=p.c, h=p.h, w=p.w, input=p.input, skip=p.skip,
                     bytes=p.bytes) for p in arr[:cnt.value]]

    def decode_traced(self, z, trace, out=None, ws=None, stream=None):
        """vae_decode_chain_traced: ``trace`` is a list with one CUDA tensor
        (or None) per trace point, receiving that step's output."""
        lib = load_library()
        _need(z, "z")
        n, c, h, w = z.shape
        if out is None:
            import torch
            f = self.up_factor
            out = torch.empty((n, self.out_channels, f * h, f * w), dtype=torch.float32,
                              device=z.device)
        if ws is None:
            ws = _ws(self.workspace_size(n, h, w), z.device)
        bufs = (_P * max(1, len(trace)))(*[None if t is None else t.data_ptr() for t in trace])
        _check("vae_decode_chain_traced", lib.vae_decode_chain_traced(
            self.handle, _ptr(z), n, h, w, _ptr(out), _ptr(ws), ws.numel(), bufs, len(trace),
            _stream(stream)))
        return out

    def capture_graph(self, z, out, ws):
        """Capture one vae_decode_chain call on fixed buffers into a CUDA graph
        (the chain neither synchronises nor allocates); replay() re-runs the
        whole decode with one launch. Make one eager decode first."""
        import torch
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.decode(z, out=out, ws=ws)
        return g

    def profile(self, enable=True):
        _check("vae_chain_profile", load_library().vae_chain_profile(self.handle, int(enable)))

    def profile_read(self):
        """Per-step records of the profiled decodes (synchronises their events)."""
        lib = load_library()
        cnt = ctypes.c_int(0)
        _check("vae_chain_profile_read", lib.vae_chain_profile_read(self.handle, None, 0,
                                                                    ctypes.byref(cnt)))
        arr = (ProfRecord * max(1, cnt.value))()
        _check("vae_chain_profile_read", lib.vae_chain_profile_read(self.handle, arr, cnt.value,
                                                                    ctypes.byref(cnt)))
        return [dict(kind=PROF_KINDS.get(r.kind, r.kind), kernels=r.kernels, flops=r.flops,
                     bytes=r.bytes, ms=r.ms) for r in arr[:cnt.value]]

    def close(self):
        if getattr(self, "handle", None):
            _check("vae_chain_destroy", load_library().vae_chain_destroy(self.handle))
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class VaeCausalDecoder:
    """Prepared 3-D causal decoder (vae_causal_decoder_prepare /
    vae_decode_causal / vae_chain_destroy). ``weights`` as
    vae_synth.make_causal_decoder_weights names them: conv weights
    [cout, cin, 3, 3, 3], 1x1x1 shortcuts [cout, cin, 1, 1]."""

    def __init__(self, weights, n_up_blocks, n_mid=2, resnets_per_block=2, latent_channels=16,
                 scaling_factor=0.3611, shift_factor=0.1159, groups=32, eps=1e-6, stream=None,
                 precision=PRECISION_AUTO):
        lib = load_library()
        keep = []

        def conv(name):
            r = _conv_ref(weights, name, keep)
            if name + ".weight" in weights and weights[name + ".weight"].ndim == 5:
                r.k = 3
            return r

        def res(pre):
            return ResnetRef(_norm_ref(weights, pre + ".norm1", keep), conv(pre + ".conv1"),
                             _norm_ref(weights, pre + ".norm2", keep), conv(pre + ".conv2"),
                             _conv_ref(weights, pre + ".conv_shortcut", keep))

        mid = (ResnetRef * max(1, n_mid))(*[res(f"mid.resnets.{m}") for m in range(n_mid)])
        ups, self._res_arrays = [], [mid]
        for i in range(n_up_blocks):
            arr = (ResnetRef * resnets_per_block)(*[
                res(f"up_blocks.{i}.resnets.{j}") for j in range(resnets_per_block)])
            self._res_arrays.append(arr)
            ups.append(UpRef(resnets_per_block, arr, conv(f"up_blocks.{i}.upsamplers.0.conv")))
        ups_arr = (UpRef * max(1, n_up_blocks))(*ups)
        args = CausalDecoderArgs(latent_channels, scaling_factor, shift_factor, groups, eps,
                                 conv("conv_in"), n_mid, mid, n_up_blocks, ups_arr,
                                 _norm_ref(weights, "conv_norm_out", keep), conv("conv_out"),
                                 int(precision))
        h = ctypes.c_void_p()
        _check("vae_causal_decoder_prepare", lib.vae_causal_decoder_prepare(
            ctypes.byref(args), ctypes.byref(h), _stream(stream)))
        self.handle = h
        self.out_channels = weights["conv_out.weight"].shape[0]
        self.up_factor = 2 ** sum(1 for i in range(n_up_blocks)
                                  if f"up_blocks.{i}.upsamplers.0.conv.weight" in weights)

    def workspace_size(self, n, t, h, w):
        return load_library().vae_causal_decoder_workspace_size(self.handle, n, t, h, w)

    def decode(self, z, out=None, ws=None, stream=None):
        lib = load_library()
        _need(z, "z")
        n, c, t, h, w = z.shape
        if out is None:
            import torch
            f = self.up_factor
            out = torch.empty((n, self.out_channels, t, f * h, f * w), dtype=torch.float32,
                              device=z.device)
        if ws is None:
            ws = _ws(self.workspace_size(n, t, h, w), z.device)
        _check("vae_decode_causal", lib.vae_decode_causal(
            self.handle, _ptr(z), n, t, h, w, _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
        return out

    def close(self):
        if getattr(self, "handle", None):
            _check("vae_chain_destroy", load_library().vae_chain_destroy(self.handle))
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
