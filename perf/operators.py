"""Measured cases of the serving operators around a differential-attention key/value cache.

Four operators: rotary positions (and their backward pass), the cache append (rotary, quantisation
and the write in one pass), attention of a tree of drafted tokens over the cache (one token is a
tree of one node), and the move of an accepted path to the front of its drafts.  DIFF V1 has two
query/key maps of width d and values of width 2d with the per-head norm; DIFF V2 has pairs of
query heads over a shared key head.  ``run`` computes a case in its plain form, or, where ``own``
is true, by the framework's entry points.
"""

import math

import numpy as np
import torch

own = False

LAM, LAM_INIT, EPS = 0.4, 0.55, 1e-5


def listed():
    return [
        # the queries and keys of a prefill of four 2048-token sequences, both maps
        dict(name="rope-prefill-v1-d64", op="rope", kind="v1", dtype="bf16", B=4, T=2048, H=16, Hq=16, d=64, rot=64,
             inter=False, scaling="none", factor=1.0, far=0, inverse=False),
        # a few drafted tokens far into long documents; half of each head rotated, in interleaved pairs
        dict(name="rope-drafts-v2-far", op="rope", kind="v2", dtype="bf16", B=8, T=5, H=16, Hq=32, d=128, rot=64,
             inter=True, scaling="yarn", factor=16.0, far=1000000, inverse=False),
        # the gradients of rotated queries and keys in a training step (fp32, as the backward pass gives them)
        dict(name="rope-gradient-v1-d128", op="rope", kind="v1", dtype="f32", B=2, T=4096, H=12, Hq=12, d=128, rot=128,
             inter=False, scaling="ntk", factor=4.0, far=0, inverse=True),
        # one decode step's new token of 16 sequences, queries rotated in the same pass
        dict(name="append-token-v1-fp8", op="append", kind="v1", fmt="fp8", B=16, T=1, H=16, Hq=16, d=64, n=1024,
             rot=64, inter=False, scaling="none", factor=1.0, far=0, ragged=False),
        # a padded prefill written to the cache in 8 bits
        dict(name="append-prefill-v2-fp8", op="append", kind="v2", fmt="fp8", B=2, T=4001, H=16, Hq=32, d=128, n=4100,
             rot=128, inter=False, scaling="linear", factor=4.0, far=0, ragged=True),
        # a decode step without drafts over long 8-bit caches
        dict(name="tree-token-v1-fp8", op="tree", kind="v1", fmt="fp8", B=8, T=1, H=16, Hq=16, d=64, n=32768,
             ragged=False),
        # five drafts over one short conversation: the call's latency
        dict(name="tree-short-v1-bf16", op="tree", kind="v1", fmt="bf16", B=1, T=5, H=8, Hq=8, d=64, n=512,
             ragged=False),
        # sixteen drafts a sequence over caches of different lengths
        dict(name="tree-drafts-v1-bf16", op="tree", kind="v1", fmt="bf16", B=4, T=16, H=12, Hq=12, d=128, n=8192,
             ragged=True),
        # eight drafts a sequence, grouped heads
        dict(name="tree-drafts-v2-bf16", op="tree", kind="v2", fmt="bf16", B=8, T=8, H=16, Hq=32, d=128, n=8192,
             ragged=True),
        # a full tree of drafts over one long document in 8 bits
        dict(name="tree-long-v1-fp8", op="tree", kind="v1", fmt="fp8", B=1, T=64, H=12, Hq=12, d=128, n=65536,
             ragged=False),
        # accepted paths of a small batch
        dict(name="keep-v1-bf16", op="keep", kind="v1", fmt="bf16", B=8, T=16, H=12, Hq=12, d=128, n=512, ragged=True),
        # accepted paths of a large batch with full trees
        dict(name="keep-v2-fp8", op="keep", kind="v2", fmt="fp8", B=256, T=64, H=16, Hq=32, d=128, n=256, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "tree", "tree", "keep"])
    kind = rng.choice(["v1", "v2"])
    d = rng.choice([64, 128]) if kind == "v1" else 128
    H = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    Hq = H if kind == "v1" else H * rng.choice([2, 4])
    if op == "tree":
        T = rng.randint(1, 64)
        n = _log(rng, 100, 30000)
        B = max(1, min(_log(rng, 1, 32), (8 * 16 * 32768 * 64) // (n * Hq * d * (1 + T // 8))))
        return dict(op=op, kind=kind, fmt=rng.choice(["bf16", "fp8k", "fp8"]), B=B, T=T, H=H, Hq=Hq, d=d,
                    n=n + T, ragged=rng.random() < 0.7)
    if op == "keep":
        T = rng.randint(2, 64)
        return dict(op=op, kind=kind, fmt=rng.choice(["bf16", "fp8k", "fp8"]), B=_log(rng, 1, 128), T=T, H=H, Hq=Hq,
                    d=d, n=T + rng.randint(1, 128), ragged=True)
    T = _log(rng, 1, 4001)
    B = max(1, min(_log(rng, 1, 32), (2 * 4001 * 16) // (T * H)))
    rot = 2 * rng.randint(1, d // 2) if rng.random() < 0.3 else rng.choice([d // 2, d])
    c = dict(op=op, kind=kind, B=B, T=T, H=H, Hq=Hq, d=d, rot=rot, inter=rng.random() < 0.5,
             scaling=rng.choice(["none", "linear", "ntk", "yarn"]) if rot > 2 else "none",
             factor=float(rng.choice([2, 4, 8, 16])), far=rng.choice([0, 0, 5000, 1000000]))
    if op == "rope":
        c.update(dtype=rng.choice(["bf16", "f32"]), inverse=rng.random() < 0.5)
    else:
        c.update(fmt=rng.choice(["bf16", "fp8k", "fp8"]), n=T + rng.randint(0, 200), ragged=rng.random() < 0.5)
    return c


# ----------------------------------------------------------------------------- inputs
def _tree(rs, T, nt):
    """Ancestor masks of a draft tree over nt of T nodes: a main chain first, its side branches behind it.
    Returns (mask uint64 [T], main chain's length, parents)."""
    D = max(1, (nt + 1) // 2)
    parent = list(range(-1, D - 1))
    for j in range(D, T):
        parent.append(int(rs.randint(0, D)) if j == D or rs.rand() < 0.5 else j - 1)
    mask = np.zeros(T, np.uint64)
    for j in range(T):
        mask[j] = np.uint64(1) << np.uint64(j)
        if parent[j] >= 0:
            mask[j] |= mask[parent[j]]
    return mask, D, parent


def _quantise(x):
    """Rows of x in e4m3 with one scale each, laid out [B, heads, n]."""
    scale = x.abs().amax(-1) / 448.0
    codes = (x / scale.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes, scale.transpose(1, 2).contiguous()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rs = np.random.RandomState(int(seed) % (1 << 31))
    B, T, H, Hq, d, v1 = c["B"], c["T"], c["H"], c["Hq"], c["d"], c["kind"] == "v1"
    dv = 2 * d if v1 else d

    def randn(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    def bf(*shape, std=1.0):
        return randn(*shape, std=std).to(torch.bfloat16)

    s = {"case": c}
    if c["op"] in ("rope", "append"):
        pos = np.arange(T)[None, :] + (rs.randint(0, c["far"], (B, 1)) if c["far"] else 0)
    if c["op"] == "rope":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s["pos"] = torch.tensor(np.broadcast_to(pos, (B, T)).copy(), dtype=torch.int32, device="cuda")
        s["x"] = [randn(B, T, h, d).to(dt) for h in ((H, H, H, H) if v1 else (Hq, H))]
        return s
    n = c["n"]
    ntok = np.full(B, T)
    if c["ragged"]:
        ntok = rs.randint((T + 1) // 2, T + 1, B)
    if c["op"] == "tree":
        lens = rs.randint((n - T) // 2, n - T + 1, B) if c["ragged"] else np.full(B, n - T)
    elif c["op"] == "append":
        lens = rs.randint(0, n - T + 1, B)
        if c["far"]:
            s["pos"] = torch.tensor(np.broadcast_to(pos, (B, T)).copy(), dtype=torch.int32, device="cuda")
        else:
            s["pos"] = None
    else:
        lens = rs.randint(0, n - T + 1, B)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["ntok"] = torch.tensor(ntok, dtype=torch.int32, device="cuda")
    trees = [_tree(rs, T, int(ntok[b])) for b in range(B)] if c["op"] != "append" else []
    if c["op"] == "tree":
        s["mask"] = torch.tensor(np.stack([t[0] for t in trees]).astype(np.int64), device="cuda")
        s["lam"] = torch.tensor([LAM], device="cuda")
        s["gamma"] = 0.9 + 0.2 * torch.rand(dv, generator=g, device="cuda")
        s["logits"] = randn(B, T, max(1, Hq // 2))
        s["q"] = [bf(B, T, Hq, d) for _ in range(2 if v1 else 1)]
    if c["op"] == "keep":
        path, nkeep = np.zeros((B, T), np.int32), np.zeros(B, np.int32)
        for b, (_, D, parent) in enumerate(trees):
            node = int(rs.randint(0, ntok[b]))  # the deepest accepted node, and its ancestors
            way = []
            while node >= 0:
                way.append(node)
                node = parent[node]
            nkeep[b] = min(len(way), D)  # (what lies behind the main chain is not overwritten)
            path[b, :len(way)] = way[::-1]
        s["path"], s["nkeep"] = torch.tensor(path, device="cuda"), torch.tensor(nkeep, device="cuda")
    if c["op"] == "append":
        s["new"] = [bf(B, T, H, d, std=1.0 + 0.5 * m) for m in range(2 if v1 else 1)] + [bf(B, T, H, dv)]
        s["q"] = [bf(B, T, Hq, d) for _ in range(2 if v1 else 1)]
    # the cache as earlier steps left it
    keys = [randn(B, n, H, d) for _ in range(2 if v1 else 1)]
    val = randn(B, n, H, dv) * torch.exp(0.3 * randn(B, n, H, 1))
    s["k_scale"] = [0.0125 * (1 + m) for m in range(len(keys))]
    if c["fmt"] == "bf16":
        s["k"], s["v"] = [k.to(torch.bfloat16) for k in keys], val.to(torch.bfloat16)
    elif c["fmt"] == "fp8k":
        s["k"] = [(k / f).clamp(-448, 448).to(torch.float8_e4m3fn) for k, f in zip(keys, s["k_scale"])]
        s["v"] = val.to(torch.bfloat16)
    else:
        both = [_quantise(k) for k in keys]
        s["k"], s["ks"] = [x[0] for x in both], [x[1] for x in both]
        s["v"], s["vs"] = _quantise(val)
    return s


# ----------------------------------------------------------------------------- plain forms
def _frequencies(c):
    """Rotary frequencies of a case in 64 bits and the factor on the rotated values."""
    r, base, f = c["rot"], 10000.0, c["factor"]
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    if c["scaling"] == "ntk":
        base = base * f ** (r / (r - 2))
    th = base ** (-2.0 * i / r)
    if c["scaling"] == "linear":
        th = th / f
    if c["scaling"] != "yarn":
        return th, 1.0
    low = max(0, math.floor(r * math.log(4096 / (2 * math.pi * 32.0)) / (2 * math.log(base))))
    high = min(r - 1, math.ceil(r * math.log(4096 / (2 * math.pi * 1.0)) / (2 * math.log(base))))
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return th * (1 - ramp) + th / f * ramp, 0.1 * math.log(f) + 1.0


def _rotate(x, pos, c, inverse=False):
    """x [B, T, heads, d] rotated in 32 bits (angles in 64)."""
    r = c["rot"]
    th, m = _frequencies(c)
    a = pos.double()[:, :, None, None] * th
    co, si = (torch.cos(a) * m).float(), (torch.sin(a) * (-m if inverse else m)).float()
    y = x.float().clone()
    if c["inter"]:
        x0, x1 = y[..., 0:r:2].clone(), y[..., 1:r:2].clone()
        y[..., 0:r:2], y[..., 1:r:2] = x0 * co - x1 * si, x1 * co + x0 * si
    else:
        x0, x1 = y[..., :r // 2].clone(), y[..., r // 2:r].clone()
        y[..., :r // 2], y[..., r // 2:r] = x0 * co - x1 * si, x1 * co + x0 * si
    return y


def _plain_append(s):
    c, v1 = s["case"], s["case"]["kind"] == "v1"
    B, T = c["B"], c["T"]
    t = torch.arange(T, device="cuda")
    at = s["lens"].long()[:, None] + t  # cache rows
    pos = s["pos"] if s["pos"] is not None else at
    live = t < s["ntok"][:, None]
    b, tt = live.nonzero(as_tuple=True)
    rows = at[b, tt]
    keys = [_rotate(k, pos, c) for k in s["new"][:-1]]
    queries = [torch.where(live[:, :, None, None], _rotate(q, pos, c).to(torch.bfloat16), torch.zeros_like(q))
               for q in s["q"]]
    for j, x in enumerate(keys + [s["new"][-1].float()]):
        val = j == len(keys)
        cache = s["v"] if val else s["k"][j]
        x = x[b, tt]
        if c["fmt"] == "bf16" or (val and c["fmt"] == "fp8k"):
            cache[b, rows] = x.to(torch.bfloat16)
            continue
        if c["fmt"] == "fp8k":
            codes = x * (1.0 / s["k_scale"][j])
        else:
            scales = s["vs"] if val else s["ks"][j]
            amax = x.abs().amax(-1)
            codes = x * torch.where(amax > 0, 448.0 / amax, torch.zeros_like(amax)).unsqueeze(-1)
            scales[b, :, rows] = amax / 448.0
        cache.view(torch.uint8)[b, rows] = codes.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return _written(s, queries)


def _written(s, queries):
    out = {"q": queries, "k": s["k"], "v": s["v"]}
    if s["case"]["fmt"] == "fp8":
        out["ks"], out["vs"] = s["ks"], s["vs"]
    return out


def _values(x, scale):
    """A cache tensor's values [B, heads, n, width] in 32 bits; scale a number, [B, heads, n] or None."""
    x = x.float().transpose(1, 2)
    if scale is None:
        return x
    return x * (scale if isinstance(scale, float) else scale.unsqueeze(-1))


def _visible(s, n):
    """[B, T, n]: which cache rows each drafted token sees."""
    j = torch.arange(n, device="cuda")
    T = s["case"]["T"]
    L = s["lens"].long()[:, None, None]
    node = j - L
    bit = (s["mask"][:, :, None] >> node.clamp(0, T - 1)) & 1
    return (node < 0) | ((node < s["ntok"][:, None, None]) & (node >= 0) & (bit == 1))


def _softmax_rows(x, seen):
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, torch.ones_like(total))


def _plain_tree(s):
    c, v1 = s["case"], s["case"]["kind"] == "v1"
    B, T, H, Hq, d = c["B"], c["T"], c["H"], c["Hq"], c["d"]
    fp8, fp8k = c["fmt"] == "fp8", c["fmt"] == "fp8k"
    seen = _visible(s, c["n"])[:, None]  # [B, 1, T, n]
    v = _values(s["v"], s["vs"] if fp8 else None)
    maps = []
    for m in range(2):
        j = m if v1 else 0
        k = _values(s["k"][j], s["ks"][j] if fp8 else s["k_scale"][j] if fp8k else None)
        if v1:
            q = s["q"][m].float().transpose(1, 2)  # [B, H, T, d]
            p = _softmax_rows(q @ k.transpose(2, 3) * (1 / math.sqrt(d)), seen)
            maps.append(p @ v)
        else:
            G = Hq // H // 2  # pairs a key head
            q = s["q"][0].float()[:, :, m::2].reshape(B, T, H, G, d).permute(0, 2, 3, 1, 4)
            x = (q.reshape(B, H, G * T, d) @ k.transpose(2, 3)).view(B, H, G, T, -1) * (1 / math.sqrt(d))
            p = _softmax_rows(x, seen[:, :, None])
            maps.append((p.view(B, H, G * T, -1) @ v).view(B, H, G, T, d).reshape(B, H * G, T, d))
        del k, p
    live = (torch.arange(T, device="cuda") < s["ntok"][:, None])[:, :, None, None]
    if v1:
        o = maps[0] - s["lam"] * maps[1]
        o = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS) * s["gamma"] * (1 - LAM_INIT)
        o = o.transpose(1, 2)
    else:
        o = maps[0].transpose(1, 2) - maps[1].transpose(1, 2) / (1 + torch.exp(-s["logits"])).unsqueeze(-1)
    return torch.where(live, o, torch.zeros_like(o)).to(torch.bfloat16)


def _plain_keep(s):
    c = s["case"]
    A = s["path"].shape[1]
    a = torch.arange(A, device="cuda")
    b, i = (a < s["nkeep"][:, None]).nonzero(as_tuple=True)
    dst = s["lens"].long()[b] + i
    src = s["lens"].long()[b] + s["path"].long()[b, i]
    for x in s["k"] + [s["v"]]:
        x = x.view(torch.uint8) if x.dtype != torch.bfloat16 else x
        x[b, dst] = x[b, src]
    if c["fmt"] == "fp8":
        for x in s["ks"] + [s["vs"]]:
            x[b, :, dst] = x[b, :, src]
    return dict(_written(s, []), lens=s["lens"] + s["nkeep"])


# ----------------------------------------------------------------------------- the framework's calls
def _spec(da, c):
    return da.rope_spec(c["rot"], interleaved=c["inter"], scaling=c["scaling"], factor=c["factor"],
                        original_context=4096)


def _cache(da, s):
    c, k = s["case"], s["k"]
    two = c["kind"] == "v1"
    a = dict(k1=k[0], k2=k[1] if two else None, v=s["v"])
    if c["fmt"] == "fp8k":
        a.update(k1_scale=s["k_scale"][0], k2_scale=s["k_scale"][1] if two else 1.0)
    if c["fmt"] == "fp8":
        a.update(k1_scales=s["ks"][0], k2_scales=s["ks"][1] if two else None, v_scales=s["vs"])
    return da.KVCache(c["fmt"], **a)


def _own(s):
    from differential_attention_03_gb300 import binding as da
    c, v1 = s["case"], s["case"]["kind"] == "v1"
    if c["op"] == "rope":
        return da.rope(s["x"], _spec(da, c), positions=s["pos"], inverse=c["inverse"])
    cache = _cache(da, s)
    if c["op"] == "append":
        a = dict(rope=_spec(da, c), positions=s["pos"], lens=s["lens"], ntok=s["ntok"])
        if v1:
            q = da.cache_append(cache, *s["new"], q1=s["q"][0], q2=s["q"][1], **a)
        else:
            q = [da.v2_cache_append(cache, *s["new"], q=s["q"][0], **a)]
        return _written(s, list(q))
    if c["op"] == "tree":
        a = dict(lens=s["lens"], ntok=s["ntok"], mask=s["mask"])
        if v1:
            return da.tree_decode(s["q"][0], s["q"][1], cache, s["lam"], LAM_INIT, gamma=s["gamma"], eps=EPS, **a)
        return da.v2_tree_decode(s["q"][0], cache, s["logits"], **a)
    lens = da.cache_keep(cache, s["lens"], s["path"], s["nkeep"])
    return dict(_written(s, []), lens=lens)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "rope":
        c = state["case"]
        return [_rotate(x, state["pos"], c, c["inverse"]).to(x.dtype) for x in state["x"]]
    return {"append": _plain_append, "tree": _plain_tree, "keep": _plain_keep}[op](state)


# ----------------------------------------------------------------------------- work
def work(case):
    c = case
    B, T, H, Hq, d, v1 = c["B"], c["T"], c["H"], c["Hq"], c["d"], c["kind"] == "v1"
    dv, maps = (2 * d, 2) if v1 else (d, 1)
    if c["op"] == "rope":
        e = 2 if c["dtype"] == "bf16" else 4
        values = B * T * d * (4 * H if v1 else Hq + H)
        return {"bytes": 2.0 * values * e + 4 * B * T, "flops": 3.0 * values}
    share = 0.75 if c["ragged"] else 1.0  # what padding and lengths leave, on average
    kb, vb = (1 if c["fmt"] != "bf16" else 2), (1 if c["fmt"] == "fp8" else 2)
    row = H * (maps * d * kb + dv * vb + (4 * (maps + 1) if c["fmt"] == "fp8" else 0))  # bytes of a token in the cache
    if c["op"] == "append":
        tokens = B * T * share
        fresh = H * (maps * d + dv) * 2 + 2 * maps * Hq * d * 2
        return {"bytes": tokens * (row + fresh), "flops": tokens * (H * (maps * d * 5 + dv * 2) + maps * Hq * d * 3.0)}
    if c["op"] == "keep":
        return {"bytes": 2.0 * B * max(1, T // 4) * share * row, "flops": 0.0}
    keys = B * (c["n"] * share)
    qs = maps * Hq * d if v1 else Hq * d
    return {"bytes": keys * row + B * T * share * (qs + (Hq * dv if v1 else Hq // 2 * d)) * 2,
            "flops": keys * T * share * (Hq * (2 * d + 2 * dv) * (2 if v1 else 1))}


# ----------------------------------------------------------------------------- 64 bits
def _turned(x, pos, c, inverse):
    """The rotation as a product of complex numbers, in 64 bits."""
    r = c["rot"]
    i = np.arange(r // 2, dtype=np.float64)
    base = 10000.0 * (c["factor"] ** (r / (r - 2)) if c["scaling"] == "ntk" else 1.0)
    th = np.exp(-2.0 * i / r * np.log(base))
    m = 1.0
    if c["scaling"] == "linear":
        th = th / c["factor"]
    elif c["scaling"] == "yarn":
        def turn(beta):  # the pair that makes `beta` turns over the original context
            return r * np.log(4096 / (beta * 2 * np.pi)) / (2 * np.log(base))
        low, high = max(0, np.floor(turn(32.0))), min(r - 1, np.ceil(turn(1.0)))
        w = np.clip((i - low) / max(high - low, 0.001), 0, 1)
        th, m = th * (1 - w + w / c["factor"]), 0.1 * np.log(c["factor"]) + 1.0
    th = torch.tensor(th, device=x.device)
    a = (pos.double().unsqueeze(-1) * th).unsqueeze(2)
    z = torch.polar(torch.full_like(a, m), -a if inverse else a)
    y = x.double().clone()
    if c["inter"]:
        w = torch.view_as_complex(y[..., :r].reshape(*y.shape[:-1], r // 2, 2).contiguous()) * z
        y[..., :r] = torch.view_as_real(w).flatten(-2)
    else:
        w = torch.complex(y[..., :r // 2], y[..., r // 2:r]) * z
        y[..., :r] = torch.cat([w.real, w.imag], -1)
    return y


def _e4m3(x):
    """Nearest e4m3 values (ties to even) of x in 64 bits."""
    x = x.clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    v1 = c["kind"] == "v1"
    B, T, H, Hq, d = c["B"], c["T"], c["H"], c["Hq"], c["d"]
    if c["op"] == "rope":
        return [_turned(x, s["pos"], c, c["inverse"]) for x in s["x"]]
    lens, ntok = s["lens"].tolist(), s["ntok"].tolist()
    if c["op"] == "tree":
        out = torch.zeros(B, T, Hq if v1 else Hq // 2, 2 * d if v1 else d, dtype=torch.float64, device="cuda")
        mask = s["mask"].cpu().numpy().astype(np.uint64)
        for b in range(B):
            L, nt = lens[b], ntok[b]
            end = L + nt
            bits = (mask[b, :nt, None] >> np.arange(nt, dtype=np.uint64)) & np.uint64(1)
            hide = torch.tensor(np.where(bits == 1, 0.0, -np.inf), device="cuda")
            for h in range(H):
                def rows(x, scales):
                    y = x[b, :end, h].double()
                    return y if scales is None else y * scales[b, h, :end].double()[:, None]
                v = rows(s["v"], s["vs"] if c["fmt"] == "fp8" else None)
                def attend(q, j):
                    k = rows(s["k"][j], s["ks"][j] if c["fmt"] == "fp8" else None)
                    if c["fmt"] == "fp8k":
                        k = k * s["k_scale"][j]
                    x = q[b, :nt].double() @ k.T / math.sqrt(d)
                    x[:, L:] += hide
                    return torch.softmax(x, -1) @ v
                if v1:
                    o = attend(s["q"][0][:, :, h], 0) - LAM * attend(s["q"][1][:, :, h], 1)
                    o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS)
                    out[b, :nt, h] = (1 - LAM_INIT) * s["gamma"].double() * o
                else:
                    for g in range(h * Hq // H // 2, (h + 1) * Hq // H // 2):
                        w = torch.sigmoid(s["logits"][b, :nt, g].double())[:, None]
                        out[b, :nt, g] = attend(s["q"][0][:, :, 2 * g], 0) - w * attend(s["q"][0][:, :, 2 * g + 1], 0)
        return out
    if c["op"] == "keep":
        path, nkeep = s["path"].tolist(), s["nkeep"].tolist()
        for b in range(B):
            L = lens[b]
            for i in range(nkeep[b]):
                for x in s["k"] + [s["v"]]:
                    y = x.view(torch.uint8) if x.dtype != torch.bfloat16 else x
                    y[b, L + i] = y[b, L + path[b][i]].clone()
                if c["fmt"] == "fp8":
                    for x in s["ks"] + [s["vs"]]:
                        x[b, :, L + i] = x[b, :, L + path[b][i]].clone()
        r = _written(s, [])
        r = {k: [x.double() for x in v] if isinstance(v, list) else v.double() for k, v in r.items()}
        return dict(r, lens=s["lens"] + s["nkeep"])
    pos = s["pos"] if s["pos"] is not None else s["lens"][:, None] + torch.arange(T, device="cuda")
    q = [_turned(x, pos, c, False) for x in s["q"]]
    fresh = [_turned(x, pos, c, False) for x in s["new"][:-1]] + [s["new"][-1].double()]
    r = _written(s, q)
    r = {k: [x.double() for x in v] if isinstance(v, list) else v.double() for k, v in r.items()}
    caches = r["k"] + [r["v"]]
    scales = r["ks"] + [r["vs"]] if c["fmt"] == "fp8" else []
    for b in range(B):
        L, nt = lens[b], ntok[b]
        for x in r["q"]:
            x[b, nt:] = 0
        for j, x in enumerate(fresh):
            x = x[b, :nt]
            if c["fmt"] == "fp8":
                f = x.abs().amax(-1, keepdim=True) / 448
                caches[j][b, L:L + nt] = _e4m3(x / f)
                scales[j][b, :, L:L + nt] = f[..., 0].T
            elif c["fmt"] == "fp8k" and j + 1 < len(fresh):
                caches[j][b, L:L + nt] = _e4m3(x / s["k_scale"][j])
            else:
                caches[j][b, L:L + nt] = x
    return r
