"""The operators between the state-space layer and the tokens of a language model, as they are measured.

  group_norm   grouped normalisation with an activation, channels last (the output norm of a block), forward and backward
  xent         softmax cross entropy of a head over a large vocabulary from the hidden states, forward and backward
  w4           products with 4-bit weights and group scales (projections and the head while serving)

`own` false: elementary torch operations in 32 bits, rounded once at the end.  `own` true: the library's calls.
"""
import math

import torch

own = False

IGNORE = -100
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # The output norm of one decode step: 128 sequences, 64 heads of 64 channels, gated.  Latency counts.
        {"name": "norm_decode_128", "op": "group_norm", "scope": "token", "batch": 128, "seqlen": 1, "groups": 64, "cg": 64, "act": "gate", "io": "bf16", "train": False},
        # The same norm in a training step over 8 x 2048 tokens: y, and every gradient.
        {"name": "norm_train_16k", "op": "group_norm", "scope": "token", "batch": 16384, "seqlen": 1, "groups": 64, "cg": 64, "act": "gate", "io": "bf16", "train": True},
        # Normalising over whole sequences (a bidirectional encoder), SiLU after the norm, training.
        {"name": "norm_seq_8x2048", "op": "group_norm", "scope": "sequence", "batch": 8, "seqlen": 2048, "groups": 32, "cg": 64, "act": "silu", "io": "bf16", "train": True},
        # Odd sizes in fp32: rows that are not a multiple of 16 bytes, few groups, a sequence of 1001 positions.
        {"name": "norm_seq_odd_f32", "op": "group_norm", "scope": "sequence", "batch": 3, "seqlen": 1001, "groups": 6, "cg": 85, "act": "silu", "io": "f32", "train": True},
        # A small head (byte- or character-level vocabulary), few tokens: launches and latency count.
        {"name": "xent_small", "op": "xent", "tokens": 77, "vocab": 1003, "width": 256, "ignored": 0.2, "train": True},
        # Loss alone, as evaluation computes it, half of the tokens being a prompt that is not scored.
        {"name": "xent_eval_4k", "op": "xent", "tokens": 4096, "vocab": 32768, "width": 1024, "ignored": 0.5, "train": False},
        # One short micro-batch of a block of width 2048: loss and gradients.
        {"name": "xent_train_2k", "op": "xent", "tokens": 2048, "vocab": 32000, "width": 2048, "ignored": 0.1, "train": True},
        # A full training batch of 8 x 2048 tokens over an odd vocabulary.
        {"name": "xent_train_16k", "op": "xent", "tokens": 16384, "vocab": 50257, "width": 2048, "ignored": 0.05, "train": True},
        # One token through a block projection (2048 -> 4096): the smallest serving call.
        {"name": "w4_one_token", "op": "w4", "tokens": 1, "rows": 4096, "width": 2048, "group": 128, "zeros": False, "out": "bf16"},
        # One token through the head, logits in fp32 for the sampler, small groups with zero points.
        {"name": "w4_head_one_token", "op": "w4", "tokens": 1, "rows": 50257, "width": 2048, "group": 32, "zeros": True, "out": "f32"},
        # A few sequences of a small server.
        {"name": "w4_head_11", "op": "w4", "tokens": 11, "rows": 50257, "width": 2048, "group": 64, "zeros": True, "out": "f32"},
        # The decode batch of 128 through the block's wide projection.
        {"name": "w4_decode_128", "op": "w4", "tokens": 128, "rows": 8192, "width": 4096, "group": 128, "zeros": True, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["group_norm", "xent", "w4"])
    if op == "group_norm":
        scope = rng.choice(["token", "sequence"])
        groups, cg = _log(rng, 1, 64), _log(rng, 5, 300)
        most = 30_000_000 // (groups * cg)  # elements of x
        if scope == "token":
            batch, seqlen = _log(rng, 1, min(16384, most)), 1
        else:
            seqlen = _log(rng, 2, min(8192, most))
            batch = _log(rng, 1, max(1, min(64, most // seqlen)))
        return {"op": op, "scope": scope, "batch": batch, "seqlen": seqlen, "groups": groups, "cg": cg, "act": rng.choice(["none", "silu", "gate"]), "io": rng.choice(["bf16", "bf16", "f32"]),
                "train": rng.random() < 0.6}
    if op == "xent":
        width = 8 * _log(rng, 8, 512)
        vocab = _log(rng, 100, 130000)
        tokens = _log(rng, 1, max(2, min(16384, 1_500_000_000_000 // (vocab * width), 800_000_000 // vocab)))
        return {"op": op, "tokens": tokens, "vocab": vocab, "width": width, "ignored": rng.choice([0.0, 0.1, 0.5]), "train": rng.random() < 0.7}
    group = rng.choice([32, 64, 128])
    width = group * _log(rng, 1, 8192 // group)
    rows = _log(rng, 1, 60000)
    tokens = rng.choice([1, 1, _log(rng, 2, 32), _log(rng, 17, 512)])
    return {"op": op, "tokens": tokens, "rows": rows, "width": width, "group": group, "zeros": rng.random() < 0.5, "out": rng.choice(["bf16", "f32"])}


def _normal(g, shape, std=1.0, mean=0.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(std).add_(mean)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": dict(case)}
    if case["op"] == "group_norm":
        dt, C = DTYPES[case["io"]], case["groups"] * case["cg"]
        shape = (case["batch"], C) if case["scope"] == "token" else (case["batch"], case["seqlen"], C)
        s["x"] = _normal(g, shape, 1.5, 0.3).to(dt)
        s["w"], s["b"] = _normal(g, (C,), 0.2, 1.0), _normal(g, (C,), 0.2)
        s["z"] = _normal(g, shape).to(dt) if case["act"] == "gate" else None
        s["dy"] = _normal(g, shape, 0.1).to(dt) if case["train"] else None
    elif case["op"] == "xent":
        M, V, K = case["tokens"], case["vocab"], case["width"]
        s["h"] = _normal(g, (M, K)).to(torch.bfloat16)
        s["W"] = torch.empty((V, K), device="cuda", dtype=torch.bfloat16)
        s["W"].normal_(0.0, 2.0 / math.sqrt(K), generator=g)
        t = torch.randint(0, V, (M,), generator=g, device="cuda")
        off = torch.rand((M,), generator=g, device="cuda") < case["ignored"]
        s["targets"] = torch.where(off, torch.full_like(t, IGNORE), t)
        # the mean over the tokens that are scored
        s["dloss"] = torch.ones((M,), device="cuda") / (~off).sum().clamp(min=1) if case["train"] else None
    else:
        M, N, K, G = case["tokens"], case["rows"], case["width"], case["group"]
        s["A"] = _normal(g, (M, K)).to(torch.bfloat16)
        s["codes"] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)  # two codes a byte, the even column low
        s["scales"] = ((torch.rand((N, K // G), generator=g, device="cuda") + 0.5) / (4.6 * math.sqrt(K))).to(torch.bfloat16)
        s["zeros"] = torch.randint(4, 12, (N, K // G), generator=g, device="cuda", dtype=torch.uint8) if case["zeros"] else None
    return s


# ---- the library's calls -------------------------------------------------------

def _run_own(s):
    from selective_state_space_exp_b200 import m3

    c = s["case"]
    if c["op"] == "group_norm":
        kw = {"weight": s["w"], "bias": s["b"], "z": s["z"], "act": c["act"], "eps": EPS, "scope": c["scope"]}
        y, mean, rstd = m3.m3_group_norm_fwd(s["x"], c["groups"], **kw)
        if not c["train"]:
            return {"y": y}
        kw.pop("eps")
        d = m3.m3_group_norm_bwd(s["x"], c["groups"], mean, rstd, s["dy"], **kw)
        return {"y": y, "dx": d["x"], "dw": d["weight"], "db": d["bias"], **({"dz": d["z"]} if s["z"] is not None else {})}
    if c["op"] == "xent":
        loss, lse = m3.m3_linear_xent_fwd(s["h"], s["W"], s["targets"], ignore_index=IGNORE)
        if not c["train"]:
            return {"loss": loss, "lse": lse}
        dh, dW = m3.m3_linear_xent_bwd(s["h"], s["W"], s["targets"], lse, s["dloss"], ignore_index=IGNORE)
        return {"loss": loss, "lse": lse, "dh": dh, "dW": dW}
    return {"out": m3.m3_linear_w4(s["A"], s["codes"], s["scales"], s["zeros"], out_dtype=DTYPES[c["out"]])}


# ---- the plain forms -------------------------------------------------------------

def _plain_norm(s):
    c, dt = s["case"], s["x"].dtype
    B, L, G = c["batch"], c["seqlen"], c["groups"]
    x = s["x"].float().view(B, L, G, c["cg"])
    w, b = s["w"].view(G, -1), s["b"].view(G, -1)
    n = L * c["cg"]
    mean = x.sum((1, 3), keepdim=True) / n
    xc = x - mean
    rstd = 1.0 / torch.sqrt((xc * xc).sum((1, 3), keepdim=True) / n + EPS)
    xhat = xc * rstd
    u = xhat * w + b
    z = s["z"].float().view_as(u) if s["z"] is not None else None
    if c["act"] == "silu":
        sg = 1.0 / (1.0 + torch.exp(-u))
        y = u * sg
    elif c["act"] == "gate":
        sg = 1.0 / (1.0 + torch.exp(-z))
        y = u * z * sg
    else:
        y = u
    out = {"y": y.to(dt).view_as(s["x"])}
    if not c["train"]:
        return out
    dy = s["dy"].float().view_as(u)
    if c["act"] == "silu":
        du = dy * sg * (1.0 + u * (1.0 - sg))
    elif c["act"] == "gate":
        du = dy * z * sg
        out["dz"] = (dy * u * sg * (1.0 + z * (1.0 - sg))).to(dt).view_as(s["x"])
    else:
        du = dy
    out["dw"], out["db"] = (du * xhat).sum((0, 1)).reshape(-1), du.sum((0, 1)).reshape(-1)
    a = du * w
    c1, c2 = a.sum((1, 3), keepdim=True) / n, (a * xhat).sum((1, 3), keepdim=True) / n
    out["dx"] = (rstd * (a - c1 - xhat * c2)).to(dt).view_as(s["x"])
    return out


def _plain_xent(s):
    h, W, t = s["h"].float(), s["W"].float(), s["targets"]
    on = t != IGNORE
    at = torch.where(on, t, torch.zeros_like(t))[:, None]
    logits = h @ W.T
    top = logits.max(1, keepdim=True).values
    lse = top + torch.log(torch.exp(logits - top).sum(1, keepdim=True))
    loss = torch.where(on[:, None], lse - logits.gather(1, at), torch.zeros_like(lse))[:, 0]
    if not s["case"]["train"]:
        return {"loss": loss, "lse": lse[:, 0]}
    scale = torch.where(on, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
    d = logits.sub_(lse).exp_()
    d.scatter_add_(1, at, torch.full_like(lse, -1.0))
    d.mul_(scale)
    return {"loss": loss, "lse": lse[:, 0], "dh": (d @ W).to(torch.bfloat16), "dW": (d.T @ h).to(torch.bfloat16)}


def _plain_w4(s):
    c = s["case"]
    q = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).float().view(c["rows"], -1, c["group"])
    q = q - (s["zeros"].float()[..., None] if s["zeros"] is not None else 8.0)
    w = (q * s["scales"].float()[..., None]).view(c["rows"], c["width"])
    return {"out": (s["A"].float() @ w.T).to(DTYPES[c["out"]])}


def run(state):
    if own:
        return _run_own(state)
    return {"group_norm": _plain_norm, "xent": _plain_xent, "w4": _plain_w4}[state["case"]["op"]](state)


# ---- what a pass cannot do without -------------------------------------------------

def work(case):
    if case["op"] == "group_norm":
        C = case["groups"] * case["cg"]
        n = case["batch"] * case["seqlen"] * C
        e = 2 if case["io"] == "bf16" else 4
        gate = case["act"] == "gate"
        reads, writes = 1 + gate, 1
        if case["train"]:
            reads, writes = reads + 1, writes + 1 + gate
        return {"bytes": n * e * (reads + writes) + C * (16 if case["train"] else 8), "flops": n * (40 if case["train"] else 15)}
    if case["op"] == "xent":
        M, V, K = case["tokens"], case["vocab"], case["width"]
        once = 2 * (M * K + V * K)
        return {"bytes": once * (2 if case["train"] else 1) + M * (20 if case["train"] else 16), "flops": (6 if case["train"] else 2) * M * V * K}
    M, N, K = case["tokens"], case["rows"], case["width"]
    groups = N * (K // case["group"])
    return {"bytes": N * K // 2 + groups * (3 if case["zeros"] else 2) + 2 * M * K + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * M * N * K}


# ---- the definitions in 64 bits ------------------------------------------------------

def _exact_norm(case, s):
    C, G, cg = case["groups"] * case["cg"], case["groups"], case["cg"]
    x = s["x"].double().reshape(case["batch"], -1, G, cg).permute(0, 2, 1, 3)  # sample, group, position, channel
    shape = x.shape
    w, b = (s[k].double().reshape(1, G, 1, cg) for k in ("w", "b"))
    flat = x.reshape(shape[0], G, -1)
    mu = flat.mean(-1)[..., None, None]
    inv = (flat.var(-1, unbiased=False)[..., None, None] + EPS).rsqrt()
    back = lambda t: t.permute(0, 2, 1, 3).reshape(s["x"].shape)  # noqa: E731
    xn = (x - mu) * inv
    u = xn * w + b
    silu = lambda t: t * torch.sigmoid(t)  # noqa: E731
    dsilu = lambda t: torch.sigmoid(t) + t * torch.sigmoid(t) * torch.sigmoid(-t)  # noqa: E731
    z = s["z"].double().reshape(case["batch"], -1, G, cg).permute(0, 2, 1, 3) if s["z"] is not None else None
    y = {"none": lambda: u, "silu": lambda: silu(u), "gate": lambda: u * silu(z)}[case["act"]]()
    out = {"y": back(y)}
    if case["train"]:
        dy = s["dy"].double().reshape(case["batch"], -1, G, cg).permute(0, 2, 1, 3)
        du = {"none": lambda: dy, "silu": lambda: dy * dsilu(u), "gate": lambda: dy * silu(z)}[case["act"]]()
        if z is not None:
            out["dz"] = back(dy * u * dsilu(z))
        out["dw"] = torch.einsum("bgpc,bgpc->gc", du, xn).reshape(C)
        out["db"] = torch.einsum("bgpc->gc", du).reshape(C)
        dn = du * w
        m1, m2 = (t.reshape(shape[0], G, -1).mean(-1)[..., None, None] for t in (dn, dn * xn))
        out["dx"] = back(inv * (dn - m1 - xn * m2))
    return out


def _exact_xent(case, s):
    W = s["W"].double()
    keep = s["targets"] != IGNORE
    loss, lse, dh = [], [], []
    dW = torch.zeros_like(W) if case["train"] else None
    step = max(1, 200_000_000 // case["vocab"])  # tokens at a time
    for i in range(0, case["tokens"], step):
        h, t, k = s["h"][i:i + step].double(), s["targets"][i:i + step], keep[i:i + step]
        logits = torch.mm(h, W.t())
        z = torch.logsumexp(logits, 1)
        lse.append(z)
        rows = torch.nonzero(k)[:, 0]
        part = torch.zeros_like(z)
        part[rows] = z[rows] - logits[rows, t[rows]]
        loss.append(part)
        if case["train"]:
            p = torch.exp(logits - z[:, None])
            p[rows, t[rows]] -= 1.0
            p *= (s["dloss"][i:i + step].double() * k)[:, None]
            dh.append(torch.mm(p, W))
            dW += torch.mm(p.t(), h)
    out = {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    return {**out, "dh": torch.cat(dh), "dW": dW} if case["train"] else out


def _exact_w4(case, s):
    G = case["group"]
    out = torch.zeros((case["tokens"], case["rows"]), dtype=torch.float64, device="cuda")
    for g in range(case["width"] // G):  # one group of columns at a time
        byte = s["codes"][:, g * G // 2:(g + 1) * G // 2]
        zero = s["zeros"][:, g, None].double() if s["zeros"] is not None else 8.0
        a = s["A"][:, g * G:(g + 1) * G].double()
        dot = a[:, 0::2] @ (torch.remainder(byte.int(), 16).double() - zero).t() + a[:, 1::2] @ (torch.div(byte.int(), 16, rounding_mode="floor").double() - zero).t()
        out += dot * s["scales"][:, g].double()
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    return {"group_norm": _exact_norm, "xent": _exact_xent, "w4": _exact_w4}[case["op"]](case, s)
