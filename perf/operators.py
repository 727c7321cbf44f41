"""Cases for the training operators that work from 8-bit activation checkpoints.

Five operators: GroupNorm(+SiLU) that keeps checkpoints of its input and output
("gn_fwd"), its backward pass from the input's checkpoint ("gn_bwd"), the conv
weight gradient from the conv input's checkpoint ("wgrad"), and the token norm
around a block (norm after it, gate, residual scale, residual sum, norm before
the next block; "bn_fwd") with its backward pass ("bn_bwd").

A checkpoint holds rows (pixels or tokens) of c channels as e4m3 numbers with one
power-of-two scale per 32 channels: payload [rows][cp], cp = c rounded up to 32,
then at the next multiple of 256 bytes the scale exponents [rows][cp / 32], each
stored as exponent + 127.
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # The smallest calls: the tiny decoder's middle block, NCHW, latency only.
        dict(name="gn_fwd_tiny_nchw", op="gn_fwd", n=1, c=128, h=8, w=8, groups=32, silu=True,
             nhwc=False),
        # A middle-block activation of a 512^2 decode.
        dict(name="gn_fwd_512ch_64", op="gn_fwd", n=1, c=512, h=64, w=64, groups=32, silu=True,
             nhwc=True),
        # The last up-block's activation of a 512^2 decode: the bulk of what a step keeps.
        dict(name="gn_fwd_128ch_512", op="gn_fwd", n=1, c=128, h=512, w=512, groups=32, silu=True,
             nhwc=True),
        # A batch of odd-sized crops in the other layout, channels that are no power of two.
        dict(name="gn_bwd_96ch_odd_nchw", op="gn_bwd", n=2, c=96, h=37, w=53, groups=32,
             silu=True, nhwc=False),
        # An up-block's backward pass at 256^2.
        dict(name="gn_bwd_256ch_256", op="gn_bwd", n=1, c=256, h=256, w=256, groups=32, silu=True,
             nhwc=True),
        # The 256^2 decoder's middle convs: many channels, few pixels.
        dict(name="wgrad_3x3_512ch_32", op="wgrad", n=1, cin=512, cout=512, h=32, w=32, k=3,
             nhwc=True),
        # The last up-block's convs at 512^2: few channels, many pixels.
        dict(name="wgrad_3x3_128ch_512", op="wgrad", n=1, cin=128, cout=128, h=512, w=512, k=3,
             nhwc=True),
        # A resnet's 1x1 shortcut on odd-sized crops, NCHW gradients.
        dict(name="wgrad_1x1_odd_nchw", op="wgrad", n=2, cin=256, cout=128, h=61, w=75, k=1,
             nhwc=False),
        # One token of a transformer block in serving: nothing is kept.
        dict(name="bn_fwd_one_token", op="bn_fwd", n=1, tokens=1, c=512, keep=False, gate=True),
        # The tokens of a 1024^2 latent (128 x 128) in training.
        dict(name="bn_fwd_16384x512", op="bn_fwd", n=1, tokens=16384, c=512, keep=True, gate=True),
        # A 256^2 latent's tokens, backward.
        dict(name="bn_bwd_1024x512", op="bn_bwd", n=1, tokens=1024, c=512, gate=True),
        # A batch of wider blocks, backward.
        dict(name="bn_bwd_4x4096x1024", op="bn_bwd", n=4, tokens=4096, c=1024, gate=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gn_fwd", "gn_bwd", "wgrad", "bn_fwd", "bn_bwd"])
    if op in ("gn_fwd", "gn_bwd"):
        groups = rng.choice([8, 32])
        c = groups * rng.choice([4, 8, 12, 16] if groups == 8 else [1, 2, 3, 4, 8, 16])
        most = (128 * 512 * 512 if op == "gn_fwd" else 256 * 256 * 256) // c
        pixels = _log_int(rng, 1, most)
        n = rng.choice([1, 1, 2, 3]) if pixels >= 3 else 1
        side = max(1, pixels // n)
        h = max(1, int(round(math.sqrt(side) * rng.uniform(0.6, 1.4))))
        w = max(1, side // h)
        return dict(op=op, n=n, c=c, h=h, w=w, groups=groups, silu=rng.random() < 0.8,
                    nhwc=rng.random() < 0.6)
    if op == "wgrad":
        k = rng.choice([1, 3, 3])
        cin, cout = (rng.choice([16, 32, 64, 96, 128, 160, 256, 512]) for _ in range(2))
        most = max(1, 128 * 128 * 512 * 512 // max(cin * cout, 128 * max(cin, cout)))
        pixels = _log_int(rng, 1, most)
        n = rng.choice([1, 1, 2, 4]) if pixels >= 4 else 1
        side = max(1, pixels // n)
        h = max(1, int(round(math.sqrt(side) * rng.uniform(0.6, 1.4))))
        w = max(1, side // h)
        return dict(op=op, n=n, cin=cin, cout=cout, h=h, w=w, k=k, nhwc=rng.random() < 0.6)
    c = 4 * _log_int(rng, 8, 1024)
    rows = _log_int(rng, 1, 4 * 4096 * 1024 // c)
    n = rng.choice([1, 1, 2, 4]) if rows >= 4 else 1
    case = dict(op=op, n=n, tokens=max(1, rows // n), c=c, gate=rng.random() < 0.7)
    if op == "bn_fwd":
        case["keep"] = rng.random() < 0.7
    return case


def work(case):
    op = case["op"]
    if op in ("gn_fwd", "gn_bwd"):
        rows, c = case["n"] * case["h"] * case["w"], case["c"]
        cp = (c + 31) // 32 * 32
        kept = rows * (cp + cp // 32)
        stats = 8 * case["n"] * case["groups"]
        if op == "gn_fwd":
            return {"bytes": 8 * rows * c + 2 * kept + stats + 8 * c, "flops": 14 * rows * c}
        return {"bytes": 8 * rows * c + kept + stats + 16 * c, "flops": 24 * rows * c}
    if op == "wgrad":
        rows, cin, cout, k = case["n"] * case["h"] * case["w"], case["cin"], case["cout"], case["k"]
        cp = (cin + 31) // 32 * 32
        return {"bytes": 4 * rows * cout + rows * (cp + cp // 32) + 4 * cout * (cin * k * k + 1),
                "flops": 2 * rows * cin * cout * k * k}
    rows, c, n = case["n"] * case["tokens"], case["c"], case["n"]
    cp = (c + 31) // 32 * 32
    kept = 2 * rows * (cp + cp // 32) + 8 * rows
    small = 4 * c * (3 + (n if case["gate"] else 0))
    if op == "bn_fwd":
        return {"bytes": 16 * rows * c + small + (kept if case["keep"] else 0),
                "flops": 12 * rows * c}
    return {"bytes": 16 * rows * c + kept + 2 * small, "flops": 22 * rows * c}


# ------------------------------------------------------------------ checkpoints
def _ckpt_bytes(rows, c):
    cp = (c + 31) // 32 * 32
    return (rows * cp + 255) // 256 * 256 + rows * (cp // 32)


def _ckpt_parts(buf, rows, c):
    """The payload [rows, cp] and the scale [rows, cp / 32] that a checkpoint's bytes hold."""
    cp = (c + 31) // 32 * 32
    at = (rows * cp + 255) // 256 * 256
    payload = buf[:rows * cp].view(torch.float8_e4m3fn).view(rows, cp)
    scale = buf[at:at + rows * (cp // 32)].view(torch.float8_e8m0fnu).view(rows, cp // 32)
    return payload, scale


def _quantise(v):
    """(payload, scale) of rows v [rows, c]: one power-of-two scale for 32 channels."""
    rows, c = v.shape
    cp = (c + 31) // 32 * 32
    b = torch.nn.functional.pad(v, (0, cp - c)).view(rows, cp // 32, 32)
    amax = b.abs().amax(-1)
    m, ex = torch.frexp(amax)
    e = torch.where(amax > 0, ex - 9 + (m > 0.875), -127).clamp(min=-127)  # 448 = 0.875 * 2^9
    q = torch.ldexp(b, -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.view(rows, cp), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _dequantise(payload, scale, c):
    rows, cp = payload.shape
    v = payload.float().view(rows, cp // 32, 32) * scale.float().unsqueeze(-1)
    return v.view(rows, cp)[:, :c]


def _keep(v):
    """The bytes of rows v's checkpoint."""
    payload, scale = _quantise(v)
    rows, c = v.shape
    buf = torch.zeros(_ckpt_bytes(rows, c), dtype=torch.uint8, device=v.device)
    p, s = _ckpt_parts(buf, rows, c)
    p.view(torch.uint8).copy_(payload.view(torch.uint8))
    s.view(torch.uint8).copy_(scale.view(torch.uint8))
    return buf


# ------------------------------------------------------------------ inputs
def _rows(t, nhwc):
    """[n, pixels, c] view of an activation."""
    if nhwc:
        return t.reshape(t.shape[0], -1, t.shape[-1])
    return t.reshape(t.shape[0], t.shape[1], -1).transpose(1, 2)


def _unrows(r, nhwc, h, w):
    n, _, c = r.shape
    if nhwc:
        return r.reshape(n, h, w, c)
    return r.transpose(1, 2).reshape(n, c, h, w).contiguous()


def _inputs(case, seed, device):
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device=device) * std + mean

    op, n, s = case["op"], case["n"], dict(case=case)
    if op in ("gn_fwd", "gn_bwd", "wgrad"):
        h, w, nhwc = case["h"], case["w"], case["nhwc"]
        c = case["cin"] if op == "wgrad" else case["c"]
        # feature maps: every channel with its own mean and spread
        x = normal(n, h * w, c) * torch.exp(normal(c, std=0.5)) + normal(c, std=0.5)
        if op != "wgrad":
            s["gamma"], s["beta"] = normal(c, std=0.1, mean=1.0), normal(c, std=0.1)
        if op == "gn_fwd":
            s["x"] = _unrows(x, nhwc, h, w)
            return s
        if op == "gn_bwd":
            xg = x.view(n, h * w, case["groups"], -1).double()
            mean = xg.mean((1, 3))
            rstd = (xg.var((1, 3), unbiased=False) + EPS).rsqrt()
            s["stats"] = torch.stack([mean, rstd], -1).float()
        s["x_ckpt"] = _keep(x.reshape(n * h * w, c))
        s["dy"] = _unrows(normal(n, h * w, case["cout"] if op == "wgrad" else c, std=1e-3), nhwc,
                          h, w)
        return s
    tokens, c = case["tokens"], case["c"]
    u = normal(n, tokens, c) * torch.exp(normal(c, std=0.3))
    x = normal(n, tokens, c, std=2.0)
    s["w_post"], s["w_pre"] = normal(c, std=0.1, mean=1.0), normal(c, std=0.1, mean=1.0)
    s["scale"] = normal(c, std=0.05, mean=0.3)
    s["gate"] = normal(n, c, std=0.5) if case["gate"] else None
    if op == "bn_fwd":
        s["u"], s["x"] = u, x
        return s
    u64 = u.double()
    m = (u64.square().mean(-1, keepdim=True) + EPS).rsqrt()
    h = u64 * m * (s["w_post"] * s["scale"])
    if s["gate"] is not None:
        h = h * s["gate"].unsqueeze(1)
    h = h + x
    r = (h.square().mean(-1, keepdim=True) + EPS).rsqrt()
    s["rstd"] = torch.stack([m.reshape(-1), r.reshape(-1)]).float()
    s["u_ckpt"] = _keep(u.reshape(n * tokens, c))
    s["h_ckpt"] = _keep(h.float().reshape(n * tokens, c))
    s["dy"], s["dh"] = normal(n, tokens, c, std=1e-3), normal(n, tokens, c, std=1e-3)
    return s


def prepare(case, seed):
    return _inputs(case, seed, "cuda")


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"gn_fwd": _gn_fwd, "gn_bwd": _gn_bwd, "wgrad": _wgrad, "bn_fwd": _bn_fwd,
            "bn_bwd": _bn_bwd}[s["case"]["op"]](s)


def _run_own(s):
    import diffusion_vae_decoder_gb300 as vae
    case = s["case"]
    op, n = case["op"], case["n"]
    if op == "bn_fwd":
        h, y, u_ckpt, h_ckpt, rstd = vae.vae_block_norm(
            s["u"], s["x"], s["w_post"], gate=s["gate"], scale=s["scale"], w_pre=s["w_pre"],
            eps=EPS, keep=case["keep"])
        out = dict(h=h, y=y)
        if case["keep"]:
            out.update(u_kept=u_ckpt.payload, u_scale=u_ckpt.scale, h_kept=h_ckpt.payload,
                       h_scale=h_ckpt.scale, rstd=rstd)
        return out
    if op == "bn_bwd":
        rows, c = n * case["tokens"], case["c"]
        return vae.vae_block_norm_backward(
            s["dy"], s["dh"], vae.Checkpoint(s["u_ckpt"], rows, c),
            vae.Checkpoint(s["h_ckpt"], rows, c), s["rstd"], s["w_post"], gate=s["gate"],
            scale=s["scale"], w_pre=s["w_pre"])
    layout = vae.VAE_NHWC if case["nhwc"] else vae.VAE_NCHW
    rows = n * case["h"] * case["w"]
    if op == "gn_fwd":
        y, x_ckpt, y_ckpt, stats = vae.vae_groupnorm_silu_ckpt(
            s["x"], s["gamma"], s["beta"], groups=case["groups"], eps=EPS,
            apply_silu=case["silu"], layout=layout)
        return dict(y=y, stats=stats, x_kept=x_ckpt.payload, x_scale=x_ckpt.scale,
                    y_kept=y_ckpt.payload, y_scale=y_ckpt.scale)
    if op == "gn_bwd":
        dx, dgamma, dbeta = vae.vae_groupnorm_silu_backward(
            s["dy"], vae.Checkpoint(s["x_ckpt"], rows, case["c"]), s["stats"], s["gamma"],
            s["beta"], groups=case["groups"], apply_silu=case["silu"], layout=layout)
        return dict(dx=dx, dgamma=dgamma, dbeta=dbeta)
    dw, dbias = vae.vae_conv2d_wgrad(s["dy"], vae.Checkpoint(s["x_ckpt"], rows, case["cin"]),
                                     case["k"], layout=layout)
    return dict(dw=dw, dbias=dbias)


# ------------------------------------------------------------------ plain forms
def _gn_fwd(s):
    case = s["case"]
    n, c, g = case["n"], case["c"], case["groups"]
    x = _rows(s["x"], case["nhwc"])
    xg = x.reshape(n, -1, g, c // g)
    mean = xg.mean((1, 3), keepdim=True)
    rstd = ((xg - mean).square().mean((1, 3), keepdim=True) + EPS).rsqrt()
    z = ((xg - mean) * rstd).reshape(n, -1, c) * s["gamma"] + s["beta"]
    y = z / (1 + torch.exp(-z)) if case["silu"] else z
    x_kept, x_scale = _quantise(x.reshape(-1, c))
    y_kept, y_scale = _quantise(y.reshape(-1, c))
    return dict(y=_unrows(y, case["nhwc"], case["h"], case["w"]),
                stats=torch.stack([mean.reshape(n, g), rstd.reshape(n, g)], -1),
                x_kept=x_kept, x_scale=x_scale, y_kept=y_kept, y_scale=y_scale)


def _gn_bwd(s):
    case = s["case"]
    n, c, g, pixels = case["n"], case["c"], case["groups"], case["h"] * case["w"]
    x = _dequantise(*_ckpt_parts(s["x_ckpt"], n * pixels, c), c).view(n, pixels, g, c // g)
    mean, rstd = (s["stats"][..., i].view(n, 1, g, 1) for i in range(2))
    xh = ((x - mean) * rstd).view(n, pixels, c)
    dz = _rows(s["dy"], case["nhwc"])
    if case["silu"]:
        z = xh * s["gamma"] + s["beta"]
        sg = 1 / (1 + torch.exp(-z))
        dz = dz * (sg * (1 + z * (1 - sg)))
    dbeta, dgamma = dz.sum((0, 1)), (dz * xh).sum((0, 1))
    xh = xh.view(n, pixels, g, c // g)
    dn = (dz * s["gamma"]).reshape(n, pixels, g, c // g)
    dx = rstd * (dn - dn.mean((1, 3), keepdim=True) - xh * (dn * xh).mean((1, 3), keepdim=True))
    return dict(dx=_unrows(dx.view(n, pixels, c), case["nhwc"], case["h"], case["w"]),
                dgamma=dgamma, dbeta=dbeta)


def _wgrad(s):
    case = s["case"]
    n, cin, cout, h, w, k = (case[i] for i in ("n", "cin", "cout", "h", "w", "k"))
    x = _dequantise(*_ckpt_parts(s["x_ckpt"], n * h * w, cin), cin).view(n, h, w, cin)
    dy = _rows(s["dy"], case["nhwc"]).reshape(n * h * w, cout)
    p = k // 2
    taps = torch.nn.functional.pad(x, (0, 0, p, p, p, p)).unfold(1, k, 1).unfold(2, k, 1)
    dw = dy.t() @ taps.reshape(n * h * w, cin * k * k)
    return dict(dw=dw.view(cout, cin, k, k), dbias=dy.sum(0))


def _bn_fwd(s):
    case = s["case"]
    u, x, c = s["u"], s["x"], case["c"]
    m = (u.square().mean(-1, keepdim=True) + EPS).rsqrt()
    f = s["scale"] if s["gate"] is None else (s["scale"] * s["gate"]).unsqueeze(1)
    h = x + f * (u * m * s["w_post"])
    r = (h.square().mean(-1, keepdim=True) + EPS).rsqrt()
    out = dict(h=h, y=h * r * s["w_pre"])
    if case["keep"]:
        u_kept, u_scale = _quantise(u.reshape(-1, c))
        h_kept, h_scale = _quantise(h.reshape(-1, c))
        out.update(u_kept=u_kept, u_scale=u_scale, h_kept=h_kept, h_scale=h_scale,
                   rstd=torch.stack([m.reshape(-1), r.reshape(-1)]))
    return out


def _bn_bwd(s):
    case = s["case"]
    n, tokens, c = case["n"], case["tokens"], case["c"]
    u = _dequantise(*_ckpt_parts(s["u_ckpt"], n * tokens, c), c).view(n, tokens, c)
    h = _dequantise(*_ckpt_parts(s["h_ckpt"], n * tokens, c), c).view(n, tokens, c)
    m, r = (s["rstd"][i].view(n, tokens, 1) for i in range(2))
    uh, hh = u * m, h * r
    dn = s["dy"] * s["w_pre"]
    dx = s["dh"] + r * (dn - hh * (hh * dn).mean(-1, keepdim=True))
    f = s["scale"] if s["gate"] is None else (s["scale"] * s["gate"]).unsqueeze(1)
    dp = dx * f * s["w_post"]
    du = m * (dp - uh * (uh * dp).mean(-1, keepdim=True))
    col = (dx * uh).sum(1)
    gate = 1.0 if s["gate"] is None else s["gate"]
    return dict(du=du, dx=dx, dw_post=(col * s["scale"] * gate).sum(0),
                dgate=None if s["gate"] is None else col * s["scale"] * s["w_post"],
                dscale=(col * s["w_post"] * gate).sum(0), dw_pre=(s["dy"] * hh).sum((0, 1)))


# ------------------------------------------------------------------ in 64 bits
def _e4m3_64(v):
    """v [rows, c] in 64 bits -> the numbers its checkpoint's payload and scales stand for."""
    rows, c = v.shape
    cp = -(-c // 32) * 32
    b = torch.zeros(rows, cp, dtype=torch.float64, device=v.device)
    b[:, :c] = v
    b = b.view(rows, -1, 32)
    top = b.abs().max(-1, keepdim=True).values
    low = torch.full_like(top, 2.0 ** -127)
    scale = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-300) / 448))),
                        low)
    scale = torch.where(448 * scale < top, scale * 2, scale)
    scale = torch.where((top > 0) & (224 * scale >= top), scale / 2, scale)
    scale = torch.maximum(scale, low)
    t = b / scale
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(t / step) * step).view(rows, cp), scale.view(rows, -1)


def _read_64(buf, rows, c):
    cp = -(-c // 32) * 32
    at = -(-rows * cp // 256) * 256
    code = buf[:rows * cp].view(rows, -1, 32).long()
    e, f = (code >> 3) & 15, (code & 7).double()
    v = torch.where(e > 0, (1 + f / 8) * torch.exp2(e.double() - 7), f / 8 * 2.0 ** -6)
    v = torch.where(code > 127, -v, v)
    power = buf[at:at + rows * (cp // 32)].view(rows, -1, 1).double() - 127
    return (v * torch.exp2(power)).view(rows, cp)[:, :c]


def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.dtype == torch.float32 else v
         for k, v in prepare(case, seed).items()}
    op, n = case["op"], case["n"]
    if op in ("bn_fwd", "bn_bwd"):
        rows, c = n * case["tokens"], case["c"]
        each = torch.arange(n, device=s["w_post"].device).repeat_interleave(case["tokens"])
        gate = (torch.ones(n, c, dtype=torch.float64, device=each.device)
                if s["gate"] is None else s["gate"])
        mix = (gate * s["scale"])[each]
        if op == "bn_fwd":
            u, x = s["u"].view(rows, c), s["x"].view(rows, c)
            m = 1 / torch.sqrt((u * u).sum(1, keepdim=True) / c + EPS)
            h = x + mix * s["w_post"] * u * m
            r = 1 / torch.sqrt((h * h).sum(1, keepdim=True) / c + EPS)
            shape = (n, case["tokens"], c)
            out = dict(h=h.view(shape), y=(s["w_pre"] * h * r).view(shape))
            if case["keep"]:
                uk, us = _e4m3_64(u)
                hk, hs = _e4m3_64(h)
                out.update(u_kept=uk, u_scale=us, h_kept=hk, h_scale=hs,
                           rstd=torch.stack([m[:, 0], r[:, 0]]))
            return out
        m, r = s["rstd"][0].view(rows, 1), s["rstd"][1].view(rows, 1)
        uh, hh = _read_64(s["u_ckpt"], rows, c) * m, _read_64(s["h_ckpt"], rows, c) * r
        a = s["dy"].view(rows, c) * s["w_pre"]
        dx = s["dh"].view(rows, c) + r * a - r * hh * (a * hh).sum(1, keepdim=True) / c
        b = dx * mix * s["w_post"]
        du = m * b - m * uh * (b * uh).sum(1, keepdim=True) / c
        per = torch.zeros(n, c, dtype=torch.float64, device=each.device)
        per = torch.stack([(dx * uh)[each == i].sum(0) for i in range(n)])
        return dict(du=du.view(n, -1, c), dx=dx.view(n, -1, c),
                    dw_post=(per * gate).sum(0) * s["scale"],
                    dgate=None if s["gate"] is None else per * (s["scale"] * s["w_post"]),
                    dscale=(per * gate).sum(0) * s["w_post"],
                    dw_pre=(s["dy"].view(rows, c) * hh).sum(0))
    h, w, pixels = case["h"], case["w"], case["h"] * case["w"]
    place = (lambda t: t.view(n, h, w, -1)) if case["nhwc"] else (
        lambda t: t.view(n, h, w, -1).permute(0, 3, 1, 2).contiguous())
    pick = (lambda t: t.reshape(n * pixels, -1)) if case["nhwc"] else (
        lambda t: t.permute(0, 2, 3, 1).reshape(n * pixels, -1))
    if op == "wgrad":
        k, cin = case["k"], case["cin"]
        x = _read_64(s["x_ckpt"], n * pixels, cin).view(n, h, w, cin)
        dy = pick(s["dy"]).view(n, h, w, -1)
        dw = torch.zeros(case["cout"], cin, k, k, dtype=torch.float64, device=x.device)
        for ky in range(k):
            for kx in range(k):
                oy, ox = ky - k // 2, kx - k // 2
                a = dy[:, max(0, -oy):h - max(0, oy), max(0, -ox):w - max(0, ox)]
                b = x[:, max(0, oy):h + min(0, oy), max(0, ox):w + min(0, ox)]
                dw[:, :, ky, kx] = torch.einsum("nhwo,nhwc->oc", a, b)
        return dict(dw=dw, dbias=dy.sum((0, 1, 2)))
    c, g = case["c"], case["groups"]
    if op == "gn_fwd":
        x = pick(s["x"]).view(n, pixels, g, -1)
        mean = x.sum((1, 3)) / (pixels * (c // g))
        var = ((x - mean.view(n, 1, g, 1)) ** 2).sum((1, 3)) / (pixels * (c // g))
        rstd = 1 / torch.sqrt(var + EPS)
        z = ((x - mean.view(n, 1, g, 1)) * rstd.view(n, 1, g, 1)).view(-1, c)
        z = z * s["gamma"] + s["beta"]
        y = z * torch.sigmoid(z) if case["silu"] else z
        xk, xs = _e4m3_64(x.reshape(-1, c))
        yk, ys = _e4m3_64(y)
        return dict(y=place(y), stats=torch.stack([mean, rstd], 2), x_kept=xk, x_scale=xs,
                    y_kept=yk, y_scale=ys)
    x = _read_64(s["x_ckpt"], n * pixels, c).view(n, pixels, g, -1)
    mean, rstd = s["stats"][:, :, 0].view(n, 1, g, 1), s["stats"][:, :, 1].view(n, 1, g, 1)
    xh = (x - mean) * rstd
    gam = s["gamma"].view(1, 1, g, -1)
    dz = pick(s["dy"]).view(n, pixels, g, -1)
    if case["silu"]:
        z = xh * gam + s["beta"].view(1, 1, g, -1)
        sg = torch.sigmoid(z)
        dz = dz * (sg + z * sg * (1 - sg))
    count = pixels * (c // g)
    a = (dz * gam).sum((1, 3), keepdim=True) / count
    b = (dz * gam * xh).sum((1, 3), keepdim=True) / count
    return dict(dx=place((rstd * (dz * gam - a - b * xh)).reshape(-1, c)),
                dgamma=(dz * xh).sum((0, 1)).reshape(c), dbeta=dz.sum((0, 1)).reshape(c))
