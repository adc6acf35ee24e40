"""Cases of the layers kept in BF16 around the quantized convolutions: layer
norm over the channels and the matrix product with bias, activation and
residual, each with its gradients, over [P][C][N] tensors.

P is the number of positions and N the batch, fastest: N = 1 is a sequence of
token rows, P = H·W with N > 1 the channel-batch-first layout of the
convolutions.  `run` computes either the plain form (elementary torch
operations in fp32) or the package's kernels (`own`)."""
import math

import torch

own = False

_T = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # a single token's norm before a projection, at inference: latency
        dict(name="ln_fwd_one_token", op="ln_fwd", P=1, C=1024, N=1, x="bf16", y="bf16", affine=True),
        # a long packed batch of tokens through a wide model's norm
        dict(name="ln_fwd_tokens", op="ln_fwd", P=16384, C=4096, N=1, x="bf16", y="bf16", affine=True),
        # the fp32 output of an 80 x 80 depthwise layer, normalised over its 64 channels for a BF16 layer
        dict(name="ln_fwd_pixels", op="ln_fwd", P=6400, C=64, N=16, x="f32", y="bf16", affine=True),
        # training step of a norm over odd rows: neither the tokens nor the channels fill a vector
        dict(name="ln_bwd_odd_tokens", op="ln_bwd", P=4097, C=1023, N=1, x="bf16", y="bf16", gx="bf16", affine=True),
        # the norm behind a 28 x 28 layer of 128 channels, batch 64: fp32 in, gradients in fp32
        dict(name="ln_bwd_pixels", op="ln_bwd", P=784, C=128, N=64, x="f32", y="f32", gx="f32", affine=True),
        # one decoded token through a square projection: reads the weights once
        dict(name="lin_fwd_one_token", op="lin_fwd", P=1, Cin=4096, Cout=4096, N=1, act="none", bias=True,
             residual=True, z=False, y="bf16"),
        # a packed, ragged batch of tokens through the widening layer of an MLP, pre-activation kept for training
        dict(name="lin_fwd_ragged_tokens", op="lin_fwd", P=8187, Cin=1024, Cout=4096, N=1, act="gelu", bias=True,
             residual=False, z=True, y="bf16"),
        # the projection back to 128 channels of a 40 x 40 block at batch 16, with the block's residual, in fp32
        dict(name="lin_fwd_pixels", op="lin_fwd", P=1600, Cin=512, Cout=128, N=16, act="none", bias=True,
             residual=True, z=False, y="f32"),
        # gradient through the activation and the bias of that widening layer
        dict(name="lin_act_grad_tokens", op="lin_act_grad", P=8187, Cout=4096, N=1, act="gelu", gy="bf16"),
        # the same in the convolutions' layout, from an fp32 gradient of a 20 x 20 layer
        dict(name="lin_act_grad_pixels", op="lin_act_grad", P=400, Cout=512, N=16, act="silu", gy="f32"),
        # input and weight gradients of the narrowing layer of an MLP
        dict(name="lin_grads_tokens", op="lin_grads", P=8192, Cin=4096, Cout=1024, N=1, gx="bf16"),
        # input and weight gradients of a 28 x 28 pointwise layer, batch 64: few weights, a long contraction
        dict(name="lin_grads_pixels", op="lin_grads", P=784, Cin=128, Cout=512, N=64, gx="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "lin_fwd", "lin_fwd", "lin_act_grad", "lin_grads"])
    pixels = rng.random() < 0.4

    def channels(lo, hi):
        c = _log_int(rng, lo, hi)
        return c if rng.random() < 0.3 else max(8, c // 8 * 8)

    if pixels:
        side = _log_int(rng, 7, 80)
        P, N = side * side, rng.choice([4, 8, 12, 16, 16, 20, 32, 64])
    else:
        P, N = _log_int(rng, 1, 16384), 1
    if op in ("ln_fwd", "ln_bwd", "lin_act_grad"):
        C = channels(16, 512) if pixels else channels(64, 8192)
        P = max(1, min(P, (1 << 25) // (C * N)))
    else:
        Cin = channels(16, 512) if pixels else channels(64, 4096)
        C = channels(16, 512) if pixels else channels(64, 4096)
        P = max(1, min(P, (1 << 35) // (C * Cin * N)))
    t = lambda: rng.choice(["f32", "bf16"])  # noqa: E731
    if op == "ln_fwd":
        return dict(op=op, P=P, C=C, N=N, x=t(), y=t(), affine=rng.random() < 0.8)
    if op == "ln_bwd":
        return dict(op=op, P=P, C=C, N=N, x=t(), y=t(), gx=t(), affine=rng.random() < 0.8)
    act = rng.choice(["none", "relu", "gelu", "silu"])
    if op == "lin_fwd":
        return dict(op=op, P=P, Cin=Cin, Cout=C, N=N, act=act, bias=rng.random() < 0.7, residual=rng.random() < 0.5,
                    z=act != "none" and rng.random() < 0.5, y=t())
    if op == "lin_act_grad":
        return dict(op=op, P=P, Cout=C, N=N, act=act if act != "none" else "gelu", gy=t())
    return dict(op=op, P=P, Cin=Cin, Cout=C, N=N, gx=t())


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = case

    def normal(shape, std=1.0, dtype="f32"):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(_T[dtype])

    def acts(shape, dtype):
        # activations: unit noise over a channel-wise offset, some channels ten times the others
        p, ch, n = shape
        scale = torch.where(torch.rand((ch, 1), generator=g, device="cuda") < 0.02, 10.0, 1.0)
        x = torch.randn(shape, generator=g, device="cuda").mul_(scale).add_(normal((ch, 1), 0.5))
        return x.to(_T[dtype])

    s = dict(case)
    if c["op"].startswith("ln"):
        shape = (c["P"], c["C"], c["N"])
        s["x"] = acts(shape, c["x"])
        s["gamma"] = normal(c["C"], 0.2).add_(1.0) if c["affine"] else None
        s["beta"] = normal(c["C"], 0.2) if c["affine"] else None
        s["y_dtype"] = _T[c["y"]]
        if c["op"] == "ln_bwd":
            s["gx_dtype"] = _T[c["gx"]]
            s["gy"] = normal(shape, 1e-2, c["y"])
            # the statistics that the forward pass kept
            xf = s["x"].float()
            s["mean"] = xf.mean(1)
            s["rstd"] = (xf - s["mean"][:, None]).square_().mean(1).add_(1e-5).rsqrt_()
        return s
    if c["op"] != "lin_act_grad":
        s["w"] = normal((c["Cout"], c["Cin"]), math.sqrt(2.0 / c["Cin"]), "bf16")
        s["x"] = acts((c["P"], c["Cin"], c["N"]), "bf16")
    out = (c["P"], c["Cout"], c["N"])
    if c["op"] == "lin_fwd":
        s["y_dtype"] = _T[c["y"]]
        s["bias"] = normal(c["Cout"], 0.1) if c["bias"] else None
        s["residual"] = normal(out, 1.0, c["y"]) if c["residual"] else None
    elif c["op"] == "lin_act_grad":
        s["gy"] = normal(out, 1e-2, c["gy"])
        s["z"] = normal(out, 1.0, "bf16")
    else:
        s["gx_dtype"] = _T[c["gx"]]
        s["gz"] = normal(out, 1e-2, "bf16")
    return s


# ------------------------------------------------------------- plain forms

def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return cdf + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return sig * (1 + z * (1 - sig))
    return torch.ones_like(z)


def _plain(s):
    op = s["op"]
    if op == "ln_fwd":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        xc = x - mean
        rstd = torch.rsqrt((xc * xc).mean(1, keepdim=True) + 1e-5)
        y = xc * rstd
        if s["gamma"] is not None:
            y = y * s["gamma"][:, None] + s["beta"][:, None]
        return {"y": y.to(s["y_dtype"]), "mean": mean.squeeze(1), "rstd": rstd.squeeze(1)}
    if op == "ln_bwd":
        gy = s["gy"].float()
        rstd = s["rstd"][:, None]
        xh = (s["x"].float() - s["mean"][:, None]) * rstd
        ggamma = (gy * xh).sum((0, 2))
        gbeta = gy.sum((0, 2))
        g = gy * s["gamma"][:, None] if s["gamma"] is not None else gy
        gx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        return {"gx": gx.to(s["gx_dtype"]), "ggamma": ggamma, "gbeta": gbeta}
    if op == "lin_fwd":
        w, x = s["w"].float(), s["x"].float()
        z = (x.squeeze(2) @ w.t()).unsqueeze(2) if s["N"] == 1 else torch.matmul(w, x)
        if s["bias"] is not None:
            z = z + s["bias"][:, None]
        y = _act(z, s["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(s["y_dtype"]), "z": z.to(torch.bfloat16) if s["z"] else None}
    if op == "lin_act_grad":
        gz = s["gy"].float() * _act_slope(s["z"].float(), s["act"])
        return {"gz": gz.to(torch.bfloat16), "gbias": gz.sum((0, 2))}
    w, x, gz = s["w"].float(), s["x"].float(), s["gz"].float()
    if s["N"] == 1:
        gx = (gz.squeeze(2) @ w).unsqueeze(2)
        gw = gz.squeeze(2).t() @ x.squeeze(2)
    else:
        gx = torch.matmul(w.t(), gz)
        gw = gz.transpose(0, 1).reshape(s["Cout"], -1) @ x.transpose(0, 1).reshape(s["Cin"], -1).t()
    return {"gx": gx.to(s["gx_dtype"]), "gw": gw}


def run(state):
    if not own:
        return _plain(state)
    import microscaling_quantized_convolution_b200 as mqv
    s = state
    op = s["op"]
    if op == "ln_fwd":
        y, mean, rstd = mqv.ln_fwd(mqv.ln_desc(s["P"], s["C"], s["N"]), s["x"], s["gamma"], s["beta"],
                                   y_dtype=s["y_dtype"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        gx, ggamma, gbeta = mqv.ln_bwd(mqv.ln_desc(s["P"], s["C"], s["N"]), s["gy"], s["x"], s["mean"], s["rstd"],
                                       s["gamma"], gx_dtype=s["gx_dtype"])
        return {"gx": gx, "ggamma": ggamma, "gbeta": gbeta}
    if op == "lin_fwd":
        d = mqv.lin_desc(s["P"], s["Cin"], s["Cout"], s["N"], act=s["act"])
        y, z = mqv.lin_fwd(d, s["w"], s["x"], bias=s["bias"], residual=s["residual"], y_dtype=s["y_dtype"],
                           save_z=s["z"])
        return {"y": y, "z": z}
    if op == "lin_act_grad":
        d = mqv.lin_desc(s["P"], s["Cout"], s["Cout"], s["N"], act=s["act"])
        gz, gbias = mqv.lin_act_grad(d, s["gy"], s["z"])
        return {"gz": gz, "gbias": gbias}
    d = mqv.lin_desc(s["P"], s["Cin"], s["Cout"], s["N"])
    return {"gx": mqv.lin_dgrad(d, s["w"], s["gz"], gx_dtype=s["gx_dtype"]), "gw": mqv.lin_wgrad(d, s["gz"], s["x"])}


def work(case):
    c = case
    size = {"f32": 4, "bf16": 2}
    if c["op"].startswith("ln"):
        n, cols, ch = c["P"] * c["C"] * c["N"], c["P"] * c["N"], c["C"]
        if c["op"] == "ln_fwd":
            return {"bytes": n * (size[c["x"]] + size[c["y"]]) + 8 * cols + (8 * ch if c["affine"] else 0),
                    "flops": 8 * n}
        return {"bytes": n * (size[c["x"]] + size[c["y"]] + size[c["gx"]]) + 8 * cols + (12 if c["affine"] else 8) * ch,
                "flops": 16 * n}
    out = c["P"] * c["Cout"] * c["N"]
    if c["op"] == "lin_act_grad":
        return {"bytes": out * (size[c["gy"]] + 4) + 4 * c["Cout"], "flops": 12 * out}
    w, x = c["Cout"] * c["Cin"], c["P"] * c["Cin"] * c["N"]
    product = 2 * w * c["P"] * c["N"]
    if c["op"] == "lin_fwd":
        b = 2 * (w + x) + out * (size[c["y"]] * (2 if c["residual"] else 1) + (2 if c["z"] else 0))
        return {"bytes": b + (4 * c["Cout"] if c["bias"] else 0), "flops": product}
    return {"bytes": 2 * (w + x + out) + size[c["gx"]] * x + 4 * w, "flops": 2 * product}


# ------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    op = case["op"]
    if op == "ln_fwd":
        var, mean = torch.var_mean(d["x"], dim=1, correction=0)
        rstd = (var + 1e-5) ** -0.5
        y = torch.einsum("pcn,pn->pcn", d["x"] - mean.unsqueeze(1), rstd)
        if case["affine"]:
            y = torch.einsum("pcn,c->pcn", y, d["gamma"]) + d["beta"].view(1, -1, 1)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        C = case["C"]
        xh = torch.einsum("pcn,pn->pcn", d["x"] - d["mean"].unsqueeze(1), d["rstd"])
        gamma = d["gamma"] if case["affine"] else torch.ones(C, dtype=torch.float64, device="cuda")
        a = torch.einsum("pcn,c->pn", d["gy"], gamma) / C
        b = torch.einsum("pcn,pcn,c->pn", d["gy"], xh, gamma) / C
        gx = torch.einsum("pcn,c->pcn", d["gy"], gamma) - a.unsqueeze(1) - torch.einsum("pcn,pn->pcn", xh, b)
        return {"gx": torch.einsum("pcn,pn->pcn", gx, d["rstd"]), "ggamma": torch.einsum("pcn,pcn->c", d["gy"], xh),
                "gbeta": torch.einsum("pcn->c", d["gy"])}
    if op == "lin_fwd":
        z = torch.einsum("oi,pin->pon", d["w"], d["x"])
        if case["bias"]:
            z += d["bias"].view(1, -1, 1)
        if case["act"] == "relu":
            y = z.clamp(min=0)
        elif case["act"] == "gelu":
            y = z * torch.special.ndtr(z)
        elif case["act"] == "silu":
            y = z * torch.special.expit(z)
        else:
            y = z.clone()
        if case["residual"]:
            y += d["residual"]
        return {"y": y, "z": z if case["z"] else None}
    if op == "lin_act_grad":
        z = d["z"]
        if case["act"] == "relu":
            slope = torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
        elif case["act"] == "gelu":
            slope = torch.special.ndtr(z) + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
        elif case["act"] == "silu":
            p = torch.special.expit(z)
            slope = p + z * p * torch.special.expit(-z)
        else:
            slope = torch.ones_like(z)
        gz = d["gy"] * slope
        return {"gz": gz, "gbias": torch.einsum("pcn->c", gz)}
    return {"gx": torch.einsum("oi,pon->pin", d["w"], d["gz"]), "gw": torch.einsum("pon,pin->oi", d["gz"], d["x"])}
