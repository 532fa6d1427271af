"""Measured cases of the operators around a differential-attention layer in a transformer block.

Three operators, each with its backward pass: the product with bias, activation and residual
(``linear``), the gated feed-forward product act(x Wg^T) * (x Wu^T) (``gated``), and the norms after
and before a block with its gate and residual scale (``norm``).  ``run`` computes a case in its plain
form, or, where ``own`` is true, by the framework's entry points.
"""

import math

import torch

own = False

EPS = 1e-5
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def listed():
    return [
        # the output projection of one decoded token onto its residual stream
        dict(name="linear-token", op="linear", M=1, N=2048, K=2048, act="none", bias=False, residual=True, out="bf16",
             train=False, strided=False),
        # the widening product of a feed-forward block over a padded batch of two long sequences, kept for training
        dict(name="linear-train-gelu", op="linear", M=8002, N=8192, K=2048, act="gelu", bias=True, residual=False,
             out="bf16", train=True, strided=False),
        # the gradients of a small layer's product, the weights' in 32 bits
        dict(name="linear-grad-small", op="linear_grad", M=1000, N=1304, K=1000, act="none", bias=True, dw="f32"),
        # the gradients of the widening product of four 2048-token sequences
        dict(name="linear-grad-gelu", op="linear_grad", M=8192, N=8192, K=2048, act="gelu", bias=True, dw="bf16"),
        # the feed-forward block of a decode step of 48 sequences
        dict(name="gated-decode", op="gated", M=48, D=2048, F=5464, act="silu", train=False),
        # the feed-forward block of a padded batch of two long sequences, kept for training
        dict(name="gated-train", op="gated", M=8002, D=4096, F=10928, act="silu", train=True),
        # the gradients of a narrow block over one short sequence
        dict(name="gated-grad-small", op="gated_grad", M=777, D=1024, F=2736, act="gelu_tanh"),
        # the gradients of a block over four 2048-token sequences
        dict(name="gated-grad", op="gated_grad", M=8192, D=2048, F=5464, act="silu"),
        # the norm between two halves of a block in a decode step of 16 sequences
        dict(name="norm-decode", op="norm", B=16, n=1, D=2048, types="bf16", post=False, gate="none", scale=1.0),
        # norms after and before, gated by the sequence, on a 32-bit residual stream
        dict(name="norm-prefill", op="norm", B=2, n=4001, D=4096, types="mixed", post=True, gate="sequence", scale=0.5),
        # the gradients of a small model's norms in 32 bits, gated by the token
        dict(name="norm-grad-small", op="norm_grad", B=3, n=333, D=1000, types="f32", post=True, gate="token", scale=1.0),
        # the gradients of four 4096-token sequences, gated by the channel
        dict(name="norm-grad", op="norm_grad", B=4, n=4096, D=2048, types="bf16", post=True, gate="channel", scale=0.7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    return 8 * _log(rng, lo // 8, hi // 8)


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "gated", "gated", "gated_grad", "norm", "norm_grad"])
    if op.startswith("norm"):
        D = _width(rng, 64, 8192) if rng.random() < 0.7 else _log(rng, 33, 4099)
        rows = max(1, min(_log(rng, 1, 16384), (16384 * 2048) // D))
        B = max(1, min(rows, _log(rng, 1, 16)))
        return dict(op=op, B=B, n=max(1, rows // B), D=D, types=rng.choice(["bf16", "mixed", "f32"]),
                    post=rng.random() < 0.6, gate=rng.choice(["none", "channel", "sequence", "token"]),
                    scale=rng.choice([1.0, 0.5, 0.1]))
    M = _log(rng, 1, 128) if rng.random() < 0.5 else _log(rng, 128, 8192)
    if op.startswith("gated"):
        D, F = _width(rng, 64, 4096), _width(rng, 64, 10928)
        return dict(op=op, M=M, D=D, F=F, act=rng.choice(ACTS), **({} if op == "gated_grad" else
                                                                  {"train": rng.random() < 0.5}))
    N, K = _width(rng, 64, 8192), _width(rng, 64, 8192)
    act, bias = rng.choice(ACTS), rng.random() < 0.6
    if op == "linear_grad":
        # (behind an activation the products' operand is rounded: their gradients are asked for in its type)
        return dict(op=op, M=M, N=N, K=K, act=act, bias=bias, dw=rng.choice(["bf16", "f32"]) if act == "none" else "bf16")
    return dict(op=op, M=M, N=N, K=K, act=act, bias=bias, residual=rng.random() < 0.5,
                out=rng.choice(["bf16", "bf16", "f32"]), train=act != "none" and rng.random() < 0.4,
                strided=rng.random() < 0.3)


# ----------------------------------------------------------------------------- inputs
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    def bf(*shape, std=1.0):
        return randn(*shape, std=std).to(torch.bfloat16)

    s = {"case": c}
    if c["op"].startswith("norm"):
        B, n, D = c["B"], c["n"], c["D"]
        dt = _TYPES["f32" if c["types"] == "f32" else "bf16"]
        st = _TYPES["bf16" if c["types"] == "bf16" else "f32"]
        rows = torch.exp(0.5 * randn(B, n, 1))  # tokens of different sizes
        s["x"] = (randn(B, n, D) * rows).to(dt)
        s["residual"] = (3.0 * randn(B, n, D) * rows).to(st)
        shape = {"none": None, "channel": (D,), "sequence": (B, D), "token": (B, n, D)}[c["gate"]]
        s["gate"] = None if shape is None else 1.0 + 0.3 * randn(*shape)
        s["gamma_post"] = 1.0 + 0.1 * randn(D) if c["post"] else None
        s["gamma"] = 1.0 + 0.1 * randn(D)
        if c["op"] == "norm_grad":
            s["dy"], s["ds"] = randn(B, n, D).to(dt), (0.5 * randn(B, n, D)).to(st)
            s["s"] = _norm_sum(s)[0].to(st)
        return s
    if c["op"].startswith("gated"):
        M, D, F = c["M"], c["D"], c["F"]
        s["x"] = bf(M, D)
        s["w"] = bf(2 * F, D, std=D ** -0.5)
        if c["op"] == "gated_grad":
            s["gu"], s["dh"] = bf(M, 2 * F), bf(M, F)
        return s
    M, N, K = c["M"], c["N"], c["K"]
    wide = bf(M, 2 * K if c.get("strided") else K)
    s["a"] = wide[:, K:] if c.get("strided") else wide  # (a slice of a token's wider row)
    s["w"] = bf(N, K, std=K ** -0.5)
    s["bias"] = randn(N, std=0.5) if c["bias"] else None
    if c["op"] == "linear_grad":
        s["dy"] = bf(M, N)
        s["pre"] = bf(M, N) if c["act"] != "none" else None
    else:
        s["residual"] = (2.0 * randn(M, N)).to(_TYPES[c["out"]]) if c["residual"] else None
    return s


# ----------------------------------------------------------------------------- plain forms
_C0, _C1 = math.sqrt(2 / math.pi), 0.044715


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(_C0 * (z + _C1 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _slope(z, act):
    """The derivative of the activation."""
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(_C0 * (z + _C1 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * _C0 * (1 + 3 * _C1 * z * z)
    if act == "silu":
        w = 1 / (1 + torch.exp(-z))
        return w * (1 + z * (1 - w))
    return torch.ones_like(z)


def _plain_linear(s):
    c = s["case"]
    z = s["a"].float() @ s["w"].float().T
    if s["bias"] is not None:
        z = z + s["bias"]
    out = _act(z, c["act"])
    if s["residual"] is not None:
        out = out + s["residual"].float()
    r = {"out": out.to(_TYPES[c["out"]])}
    if c["train"]:
        r["pre"] = z.to(torch.bfloat16)
    return r


def _plain_linear_grad(s):
    c = s["case"]
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _slope(s["pre"].float(), c["act"])
    r = {"da": (dz @ s["w"].float()).to(torch.bfloat16), "dw": (dz.T @ s["a"].float()).to(_TYPES[c["dw"]])}
    if c["bias"]:
        r["dbias"] = dz.sum(0)
    return r


def _plain_gated(s):
    c = s["case"]
    gu = s["x"].float() @ s["w"].float().T
    g, u = gu[:, :c["F"]], gu[:, c["F"]:]
    r = {"h": (_act(g, c["act"]) * u).to(torch.bfloat16)}
    if c["train"]:
        r["gu"] = gu.to(torch.bfloat16)
    return r


def _plain_gated_grad(s):
    c = s["case"]
    g, u, dh = s["gu"][:, :c["F"]].float(), s["gu"][:, c["F"]:].float(), s["dh"].float()
    dgu = torch.cat([dh * u * _slope(g, c["act"]), dh * _act(g, c["act"])], 1)
    return {"dx": (dgu @ s["w"].float()).to(torch.bfloat16), "dw": (dgu.T @ s["x"].float()).to(torch.bfloat16)}


def _normed(x):
    """x over the root of its rows' mean square, and one over that root."""
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r, r


def _gate(s):
    g = s["gate"]
    return None if g is None else g[:, None] if g.dim() == 2 else g


def _norm_sum(s):
    """The residual stream behind the block, and what was gated."""
    c, p, g = s["case"], s["x"].float(), _gate(s)
    if c["post"]:
        p = _normed(p)[0] * s["gamma_post"]
    t = p if g is None else g * p
    return s["residual"].float() + c["scale"] * t, p


def _plain_norm(s):
    y = _norm_sum(s)[0]
    return {"s": y.to(s["residual"].dtype), "y": (_normed(y)[0] * s["gamma"]).to(s["x"].dtype)}


def _over_rows(x, like):
    """x [B, n, D] summed over the rows that share a row of `like`."""
    return x.sum((0, 1)) if like.dim() == 1 else x.sum(1) if like.dim() == 2 else x


def _plain_norm_grad(s):
    c, g = s["case"], _gate(s)
    dy = s["dy"].float()
    n, r = _normed(s["s"].float())
    dn = dy * s["gamma"]
    t = s["ds"].float() + r * (dn - n * (dn * n).mean(-1, keepdim=True))
    out = {"dresidual": t.to(s["s"].dtype), "dgamma": (dy * n).sum((0, 1))}
    x = s["x"].float()
    dp = c["scale"] * (t if g is None else t * g)
    if c["post"]:
        n, r = _normed(x)
        dn = dp * s["gamma_post"]
        out["dgamma_post"] = (dp * n).sum((0, 1))
        if g is not None:
            out["dgate"] = _over_rows(c["scale"] * t * n * s["gamma_post"], s["gate"])
        out["dx"] = (r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(s["x"].dtype)
        return out
    if g is not None:
        out["dgate"] = _over_rows(c["scale"] * t * x, s["gate"])
    out["dx"] = dp.to(s["x"].dtype)
    return out


# ----------------------------------------------------------------------------- the framework's calls
def _own(s):
    from differential_attention_03_gb300 import binding as da
    c = s["case"]
    op = c["op"]
    if op == "linear":
        a = dict(bias=s["bias"], act=c["act"], residual=s["residual"], dtype=_TYPES[c["out"]])
        if c["train"]:
            out, pre = da.linear_train(s["a"], s["w"], **a)
            return {"out": out, "pre": pre}
        return {"out": da.linear(s["a"], s["w"], **a)}
    if op == "linear_grad":
        return da.linear_backward(s["a"], s["w"], s["dy"], pre=s["pre"], act=c["act"], bias=c["bias"],
                                  dw_dtype=_TYPES[c["dw"]])
    if op == "gated":
        if c["train"]:
            h, gu = da.gated_linear_train(s["x"], s["w"], act=c["act"])
            return {"h": h, "gu": gu}
        return {"h": da.gated_linear(s["x"], s["w"], act=c["act"])}
    if op == "gated_grad":
        return da.gated_linear_backward(s["x"], s["w"], s["gu"], s["dh"], act=c["act"], dw_dtype=torch.bfloat16)
    a = dict(gate=s["gate"], scale=c["scale"], gamma_post=s["gamma_post"], gamma=s["gamma"], eps=EPS)
    if op == "norm":
        y, stream = da.residual_norm(s["x"], s["residual"], **a)
        return {"s": stream, "y": y}
    return da.residual_norm_backward(s["x"], s["s"], s["dy"], s["ds"], **a)


def run(state):
    if own:
        return _own(state)
    return {"linear": _plain_linear, "linear_grad": _plain_linear_grad, "gated": _plain_gated,
            "gated_grad": _plain_gated_grad, "norm": _plain_norm, "norm_grad": _plain_norm_grad}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"].startswith("norm"):
        v = c["B"] * c["n"] * c["D"]
        e = 4 if c["types"] == "f32" else 2
        t = 2 if c["types"] == "bf16" else 4
        gate = 4 * c["D"] * {"none": 0, "channel": 1, "sequence": c["B"], "token": c["B"] * c["n"]}[c["gate"]]
        if c["op"] == "norm":
            return {"bytes": 2.0 * v * (e + t) + gate + 8 * c["D"], "flops": 10.0 * v}
        return {"bytes": v * (3.0 * e + 3.0 * t) + 2 * gate + 16 * c["D"], "flops": 25.0 * v}
    if c["op"].startswith("gated"):
        M, D, F = c["M"], c["D"], c["F"]
        if c["op"] == "gated":
            return {"bytes": 2.0 * (M * D + 2 * F * D + M * F * (3 if c["train"] else 1)), "flops": 4.0 * M * D * F}
        return {"bytes": 2.0 * (2 * M * D + 4 * F * D + 3 * M * F), "flops": 8.0 * M * D * F}
    M, N, K = c["M"], c["N"], c["K"]
    if c["op"] == "linear":
        e = 4 if c["out"] == "f32" else 2
        each = e * (2 if c["residual"] else 1) + (2 if c["train"] else 0)
        return {"bytes": 2.0 * (M * K + N * K) + M * N * each + (4 * N if c["bias"] else 0), "flops": 2.0 * M * N * K}
    return {"bytes": 2.0 * (2 * M * K + N * K + M * N * (1 if c["act"] == "none" else 2)) +
            N * K * (4 if c["dw"] == "f32" else 2) + (4 * N if c["bias"] else 0), "flops": 4.0 * M * N * K}


# ----------------------------------------------------------------------------- 64 bits
def _bend(z, act):
    """The activation in 64 bits, by other identities than the plain form's."""
    if act == "relu":
        return (z + z.abs()) / 2
    if act == "gelu":
        return z * torch.special.erfc(-z / math.sqrt(2.0)) / 2
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * (1 + torch.tanh(z / 2)) / 2
    return z


def _rms(x, gamma):
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    return y * gamma


def _pull(outs, leaves, cots):
    """The gradients of the leaves from those of the outputs."""
    return torch.autograd.grad(outs, leaves, cots)


def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    op = c["op"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if op == "linear":
        z = torch.einsum("mk,nk->mn", d["a"], d["w"]) + (d["bias"] if "bias" in d else 0.0)
        r = {"out": _bend(z, c["act"]) + (d["residual"] if "residual" in d else 0.0)}
        return dict(r, pre=z) if c["train"] else r
    if op == "gated":
        g, u = (torch.einsum("md,fd->mf", d["x"], w) for w in d["w"].chunk(2))
        r = {"h": u * _bend(g, c["act"])}
        return dict(r, gu=torch.cat([g, u], 1)) if c["train"] else r
    with torch.enable_grad():
        if op == "linear_grad":
            dz = d["dy"]
            if c["act"] == "relu":
                dz = torch.where(d["pre"] > 0, dz, torch.zeros_like(dz))  # (at zero the slope is zero)
            elif c["act"] != "none":
                z = d["pre"].requires_grad_()
                dz, = _pull(_bend(z, c["act"]), z, dz)
            r = {"da": torch.einsum("mn,nk->mk", dz, d["w"]), "dw": torch.einsum("mn,mk->nk", dz, d["a"])}
            return dict(r, dbias=torch.ones_like(dz[:, 0]) @ dz) if c["bias"] else r
        if op == "gated_grad":
            g, u = (t.clone().requires_grad_() for t in d["gu"].chunk(2, 1))
            if c["act"] == "relu":
                dg, du = torch.where(g > 0, d["dh"] * u, torch.zeros_like(u)), d["dh"] * _bend(g, "relu")
                dg, du = dg.detach(), du.detach()
            else:
                dg, du = _pull(u * _bend(g, c["act"]), (g, u), d["dh"])
            wg, wu = d["w"].chunk(2)
            return {"dx": dg @ wg + du @ wu, "dw": torch.cat([torch.einsum("mf,md->fd", t, d["x"]) for t in (dg, du)])}

        def stream(x, residual, gate, gp):
            p = _rms(x, gp) if gp is not None else x
            if gate is not None:
                p = p * (gate.unsqueeze(1) if gate.dim() == 2 else gate)
            return residual + c["scale"] * p
        if op == "norm":
            t = stream(d["x"], d["residual"], d.get("gate"), d.get("gamma_post"))
            return {"s": t, "y": _rms(t, d["gamma"])}
        t, ga = d["s"].requires_grad_(), d["gamma"].requires_grad_()
        dt, dga = _pull(_rms(t, ga), (t, ga), d["dy"])
        dt = dt + d["ds"]
        names = ["x"] + [k for k in ("gate", "gamma_post") if k in d]
        for k in names:
            d[k].requires_grad_()
        got = _pull(stream(d["x"], d["residual"], d.get("gate"), d.get("gamma_post")), [d[k] for k in names], dt)
        return dict({"d" + k: v for k, v in zip(names, got)}, dresidual=dt, dgamma=dga)
