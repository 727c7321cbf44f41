"""Cases for the operators of a transformer block's MLP, forward and backward.

Layer norm ("ln_fwd") with its backward pass ("ln_bwd"), dropout with a residual sum
("dropout"; its backward pass is the same call on the gradient), the matrix product
with bias, activation and residual ("linear"), the gradient of its input through the
activation before it ("dgrad") and of its weights and bias ("wgrad").

Tokens are rows of c channels in float32, bfloat16 or float16; norm weights, biases
and their gradients are float32, as is the gradient of a linear layer's weights.

Dropout's random numbers: element i of the tensor takes 16 bits of a Philox 4x32-10
block (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3",
2011) with the 64-bit seed as its key and offset + i // 8 as its counter: of the
block's four words, word (i % 8) // 2, its low half for even i. It is dropped where
those bits are below T = floor(65536 p + 1/2); what is kept is scaled by
65536 / (65536 - T).
"""
import math

import numpy
import torch

own = False

EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One token in serving: nothing is kept for a backward pass.
        dict(name="ln_fwd_one_token_f32", op="ln_fwd", rows=1, c=512, dtype="f32", keep=False),
        # The tokens of a 1024^2 latent (128 x 128) in training.
        dict(name="ln_fwd_16384x512", op="ln_fwd", rows=16384, c=512, dtype="bf16", keep=True),
        # Odd numbers of tokens and channels, no gradient from the residual stream.
        dict(name="ln_bwd_odd_f32", op="ln_bwd", rows=1221, c=700, dtype="f32", dres=False),
        # A batch of four 512^2 latents through a wider block.
        dict(name="ln_bwd_16384x1024", op="ln_bwd", rows=16384, c=1024, dtype="bf16", dres=True),
        # The tokens of a 256^2 latent: latency counts.
        dict(name="dropout_1024x512_f32", op="dropout", rows=1024, c=512, dtype="f32", p=0.1,
             residual=False),
        # After the second product of a wide block, onto the residual stream.
        dict(name="dropout_16384x2048", op="dropout", rows=16384, c=2048, dtype="bf16", p=0.2,
             residual=True),
        # One token through the first product of an MLP.
        dict(name="linear_one_token", op="linear", rows=1, k=512, n=2048, dtype="bf16",
             act="gelu", bias=True, residual=False, keep=False),
        # The same in training: what the activation's gradient needs is kept.
        dict(name="linear_16384x512_2048", op="linear", rows=16384, k=512, n=2048, dtype="bf16",
             act="gelu", bias=True, residual=False, keep=True),
        # Odd sizes in full precision.
        dict(name="dgrad_odd_f32", op="dgrad", rows=2294, n=264, k=520, dtype="f32", act="silu"),
        # Back through a wide MLP's second product and the activation before it.
        dict(name="dgrad_16384x1024_4096", op="dgrad", rows=16384, n=1024, k=4096, dtype="bf16",
             act="gelu"),
        # A projection's weights on odd-sized crops.
        dict(name="wgrad_odd_f16", op="wgrad", rows=4575, n=256, k=128, dtype="f16"),
        # A wide MLP's first product.
        dict(name="wgrad_16384x1024_4096", op="wgrad", rows=16384, n=4096, k=1024, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "dropout", "linear", "linear", "dgrad", "wgrad"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    if op in ("ln_fwd", "ln_bwd", "dropout"):
        c = 4 * _log_int(rng, 8, 1024) if op != "dropout" else _log_int(rng, 1, 4096)
        most = (16384 * 1024 if op != "dropout" else 16384 * 2048) // (2 if dtype == "f32" else 1)
        case = dict(op=op, rows=_log_int(rng, 1, max(1, most // c)), c=c, dtype=dtype)
        if op == "ln_fwd":
            case["keep"] = rng.random() < 0.7
        elif op == "ln_bwd":
            case["dres"] = rng.random() < 0.6
        else:
            case["p"] = rng.choice([0.1, rng.uniform(0.0, 0.6)])
            case["residual"] = rng.random() < 0.6
        return case
    n, k = 8 * _log_int(rng, 4, 512), 8 * _log_int(rng, 4, 512)
    most = 16384 * 1024 * 4096 // (8 if dtype == "f32" else 1)
    case = dict(op=op, rows=_log_int(rng, 1, max(1, min(most // (n * k), 65536))), n=n, k=k,
                dtype=dtype)
    if op == "linear":
        case.update(act=rng.choice(["none", "silu", "gelu"]), bias=rng.random() < 0.8,
                    residual=rng.random() < 0.4)
        case["keep"] = case["act"] != "none" and rng.random() < 0.6
    elif op == "dgrad":
        case["act"] = rng.choice(["none", "silu", "gelu"])
    return case


def work(case):
    op, rows = case["op"], case["rows"]
    e = 4 if case["dtype"] == "f32" else 2
    if op == "ln_fwd":
        c = case["c"]
        return {"bytes": 2 * e * rows * c + 8 * c + (8 * rows if case["keep"] else 0),
                "flops": 8 * rows * c}
    if op == "ln_bwd":
        c = case["c"]
        return {"bytes": (4 if case["dres"] else 3) * e * rows * c + 8 * rows + 12 * c,
                "flops": 14 * rows * c}
    if op == "dropout":
        count = rows * case["c"]
        return {"bytes": (3 if case["residual"] else 2) * e * count, "flops": 2 * count}
    n, k = case["n"], case["k"]
    if op == "linear":
        cols = 1 + (1 if case["residual"] else 0) + (1 if case["keep"] else 0)
        moved = e * (rows * k + n * k + cols * rows * n) + (4 * n if case["bias"] else 0)
    elif op == "dgrad":
        moved = e * (rows * n + n * k + (1 if case["act"] == "none" else 2) * rows * k)
    else:
        moved = e * rows * (n + k) + 4 * n * (k + 1)
    return {"bytes": moved, "flops": 2 * rows * n * k}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=t):
        v = torch.randn(*shape, generator=g, device="cuda")
        return v.mul_(std).add_(mean).to(dtype)

    op, rows, s = case["op"], case["rows"], dict(case=case)
    f32 = torch.float32
    if op in ("ln_fwd", "ln_bwd"):
        c = case["c"]
        # a residual stream: every channel with its own mean and spread
        x = torch.randn(rows, c, generator=g, device="cuda")
        s["x"] = (x * torch.exp(normal(c, std=0.5, dtype=f32)) + normal(c, std=0.5, dtype=f32)).to(t)
        s["gamma"] = normal(c, std=0.1, mean=1.0, dtype=f32)
        if op == "ln_fwd":
            s["beta"] = normal(c, std=0.1, dtype=f32)
            return s
        x64 = s["x"].double()
        mean = x64.mean(-1)
        rstd = ((x64 - mean.unsqueeze(-1)).square().mean(-1) + EPS).rsqrt()
        s["stats"] = torch.stack([mean, rstd], -1).float()
        s["dy"] = normal(rows, c, std=1e-2)
        s["dres"] = normal(rows, c, std=1e-2) if case["dres"] else None
        return s
    if op == "dropout":
        s["x"] = normal(rows, case["c"])
        s["residual"] = normal(rows, case["c"], std=2.0) if case["residual"] else None
        s["seed"] = (seed * 0x9E3779B97F4A7C15 + 1) % 2 ** 64
        s["offset"] = 2 ** 32 - 100  # one long training run's counters pass 32 bits
        return s
    n, k = case["n"], case["k"]
    if op == "linear":
        s["x"], s["w"] = normal(rows, k), normal(n, k, std=k ** -0.5)
        s["bias"] = normal(n, std=0.1, dtype=f32) if case["bias"] else None
        s["residual"] = normal(rows, n, std=2.0) if case["residual"] else None
    elif op == "dgrad":
        s["dy"], s["w"] = normal(rows, n, std=1e-2), normal(n, k, std=k ** -0.5)
        s["z"] = normal(rows, k) if case["act"] != "none" else None
    else:
        s["dy"], s["x"] = normal(rows, n, std=1e-2), normal(rows, k)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"ln_fwd": _ln_fwd, "ln_bwd": _ln_bwd, "dropout": _dropout, "linear": _linear,
            "dgrad": _dgrad, "wgrad": _wgrad}[s["case"]["op"]](s)


def _run_own(s):
    import diffusion_vae_decoder_gb300 as vae
    case = s["case"]
    op = case["op"]
    if op == "ln_fwd":
        y, stats = vae.vae_layer_norm(s["x"], s["gamma"], s["beta"], eps=EPS, keep=case["keep"])
        return dict(y=y, stats=stats) if case["keep"] else dict(y=y)
    if op == "ln_bwd":
        dx, dgamma, dbeta = vae.vae_layer_norm_backward(s["dy"], s["x"], s["stats"], s["gamma"],
                                                        dres=s["dres"])
        return dict(dx=dx, dgamma=dgamma, dbeta=dbeta)
    if op == "dropout":
        return vae.vae_dropout(s["x"], case["p"], seed=s["seed"], offset=s["offset"],
                               residual=s["residual"])
    if op == "wgrad":
        dw, dbias = vae.vae_linear_wgrad(s["dy"], s["x"])
        return dict(dw=dw, dbias=dbias)
    act = {"none": vae.VAE_ACT_NONE, "silu": vae.VAE_ACT_SILU, "gelu": vae.VAE_ACT_GELU}[case["act"]]
    if op == "dgrad":
        return vae.vae_linear_dgrad(s["dy"], s["w"], z=s["z"], act=act)
    y, z = vae.vae_linear(s["x"], s["w"], bias=s["bias"], act=act, residual=s["residual"],
                          keep=case["keep"])
    return dict(y=y, z=z) if case["keep"] else dict(y=y)


# ------------------------------------------------------------------ plain forms
def _ln_fwd(s):
    x = s["x"].float()
    mean = x.mean(-1, keepdim=True)
    rstd = ((x - mean).square().mean(-1, keepdim=True) + EPS).rsqrt()
    y = ((x - mean) * rstd * s["gamma"] + s["beta"]).to(s["x"].dtype)
    return dict(y=y, stats=torch.cat([mean, rstd], -1)) if s["case"]["keep"] else dict(y=y)


def _ln_bwd(s):
    dy = s["dy"].float()
    mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
    xh = (s["x"].float() - mean) * rstd
    t = dy * s["gamma"]
    dx = rstd * (t - t.mean(-1, keepdim=True) - xh * (t * xh).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dict(dx=dx.to(s["x"].dtype), dgamma=(dy * xh).sum(0), dbeta=dy.sum(0))


def _threshold(p):
    return int(math.floor(65536 * p + 0.5))


def _philox_words(seed, offset, blocks, device):
    """The four words of Philox 4x32-10 for counters offset .. offset + blocks - 1."""
    low = 0xFFFFFFFF

    def product(a, b):  # high and low words of a 32-bit constant times words b
        part = a * (b >> 16) + ((a * (b & 0xFFFF)) >> 16)
        return part >> 16, (a * b) & low

    i = torch.arange(blocks, device=device)
    at = (offset & low) + (i & low)
    c0, c1 = at & low, ((offset >> 32) + (i >> 32) + (at >> 32)) & low
    c2, c3 = torch.zeros_like(i), torch.zeros_like(i)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        h0, l0 = product(0xD2511F53, c0)
        h1, l1 = product(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c0, c1, c2, c3


def _dropout(s):
    x, count, t = s["x"], s["x"].numel(), _threshold(s["case"]["p"])
    words = torch.stack(_philox_words(s["seed"], s["offset"], (count + 7) // 8, x.device), -1)
    bits = torch.stack([words & 0xFFFF, words >> 16], -1).view(-1)[:count].view(x.shape)
    y = torch.where(bits >= t, x.float() * (65536 / (65536 - t)), 0.0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(x.dtype)


def _gate(z, act):
    """(v, v') where the activation is z / (1 + exp(-v))."""
    if act == "silu":
        return z, torch.ones_like(z)
    a = math.sqrt(8 / math.pi)
    return a * (z + 0.044715 * z * z * z), a * (1 + 3 * 0.044715 * z * z)


def _linear(s):
    case, x = s["case"], s["x"]
    z = x.float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"]
    y = z if case["act"] == "none" else z / (1 + torch.exp(-_gate(z, case["act"])[0]))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = y.to(x.dtype)
    return dict(y=y, z=z.to(x.dtype)) if case["keep"] else dict(y=y)


def _dgrad(s):
    dx = s["dy"].float() @ s["w"].float()
    if s["z"] is not None:
        z = s["z"].float()
        v, dv = _gate(z, s["case"]["act"])
        g = 1 / (1 + torch.exp(-v))
        dx = dx * (g * (1 + z * dv * (1 - g)))
    return dx.to(s["dy"].dtype)


def _wgrad(s):
    dy = s["dy"].float()
    return dict(dw=dy.t() @ s["x"].float(), dbias=dy.sum(0))


# ------------------------------------------------------------------ in 64 bits
def _kept_64(seed, offset, count, p):
    """numpy truth values of the elements that dropout keeps."""
    i = numpy.arange(-(-count // 8), dtype=numpy.uint64) + numpy.uint64(offset)
    u = numpy.uint64
    word, half = u(0xFFFFFFFF), u(32)
    ctr = [i & word, i >> half, numpy.zeros_like(i), numpy.zeros_like(i)]
    key = [seed % 2 ** 32, seed // 2 ** 32]
    for _ in range(10):
        a, b = ctr[0] * u(0xD2511F53), ctr[2] * u(0xCD9E8D57)
        ctr = [(b >> half) ^ ctr[1] ^ u(key[0]), b & word, (a >> half) ^ ctr[3] ^ u(key[1]),
               a & word]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    out = numpy.empty((i.size, 8), dtype=numpy.int64)
    for j in range(4):
        out[:, 2 * j] = ctr[j] % u(65536)
        out[:, 2 * j + 1] = ctr[j] // u(65536)
    return out.reshape(-1)[:count] >= int(65536 * p + 0.5)


def exact(case, seed):
    s = {name: v.double() if isinstance(v, torch.Tensor) else v
         for name, v in prepare(case, seed).items()}
    op = case["op"]
    if op == "dropout":
        x = s["x"]
        kept = _kept_64(s["seed"], s["offset"], x.numel(), case["p"])
        kept = torch.from_numpy(kept).to(x.device).view(x.shape)
        y = torch.zeros_like(x) if s["residual"] is None else s["residual"].clone()
        y[kept] += x[kept] / (1 - int(65536 * case["p"] + 0.5) / 65536)
        return y
    if op == "ln_fwd":
        x = s["x"]
        mean = x.sum(1) / case["c"]
        dev = x - mean[:, None]
        rstd = 1 / torch.sqrt((dev * dev).sum(1) / case["c"] + EPS)
        y = s["gamma"] * (dev * rstd[:, None]) + s["beta"]
        return dict(y=y, stats=torch.stack([mean, rstd], 1)) if case["keep"] else dict(y=y)
    if op == "ln_bwd":
        mean, rstd = s["stats"][:, 0, None], s["stats"][:, 1, None]
        xh = (s["x"] - mean) * rstd
        b = s["dy"] * s["gamma"]
        b = b - b.sum(1, keepdim=True) / case["c"] - xh * ((b * xh).sum(1, keepdim=True) / case["c"])
        dx = b * rstd
        if case["dres"]:
            dx = dx + s["dres"]
        return dict(dx=dx, dgamma=torch.einsum("rc,rc->c", s["dy"], xh), dbeta=s["dy"].sum(0))
    if op == "wgrad":
        return dict(dw=torch.einsum("rn,rk->nk", s["dy"], s["x"]), dbias=s["dy"].sum(0))

    def sigmoid_arg(z):
        if case["act"] == "silu":
            return z
        return 2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)

    if op == "dgrad":
        dx = torch.einsum("rn,nk->rk", s["dy"], s["w"])
        if case["act"] != "none":
            z = s["z"]
            g = torch.sigmoid(sigmoid_arg(z))
            slope = 1 if case["act"] == "silu" else 2 * (2 / math.pi) ** 0.5 * (1 + 0.134145 * z ** 2)
            dx = dx * (g + z * slope * g * (1 - g))
        return dx
    z = torch.einsum("rk,nk->rn", s["x"], s["w"])
    if case["bias"]:
        z = z + s["bias"]
    y = z if case["act"] == "none" else z * torch.sigmoid(sigmoid_arg(z))
    if case["residual"]:
        y = y + s["residual"]
    return dict(y=y, z=z) if case["keep"] else dict(y=y)
