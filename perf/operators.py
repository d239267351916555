"""Cases of the state space block's operators: layer norm, the short causal
convolution and the selective scan, each with its gradients, and the two
one-token steps.

Widths and lengths are those of the repository's workloads (``synth.py``):
model width H*d = 192 (ViT-T), 768 (ViT-B and the 2496-px images), 1024
(BERT-large) and 512 (the 4096-token task), the block's inner width twice
that, L = 197, 4096 and 24337.  ``run`` computes a case in plain torch
operations in 32 bits, or, where ``own`` is true, through
``bidirectional_masked_linear_gb300.ssm``.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_EPS = 1e-5


# ------------------------------------------------------------------- cases

def _norm(**kw):
    return {"op": "norm", "dtype": "bf16", "train": False, "bias": True, **kw}


def _conv(**kw):
    return {"op": "conv", "dtype": "bf16", "train": False, "K": 4, "act": "silu", "ragged": False, "state": False,
            "reverse": False, "view": False, **kw}


def _scan(**kw):
    return {"op": "scan", "dtype": "bf16", "train": False, "N": 16, "G": 1, "R": 0, "gate": True, "ragged": False,
            "state": False, "reverse": False, **kw}


def listed():
    return [
        # one image's tokens through one norm of the smallest model: a launch's latency
        _norm(name="norm_one_image", rows=197, C=192),
        # a training step of a ViT-B block's norm
        _norm(name="norm_train_vit", rows=64 * 197, C=768, train=True),
        # the same on two 2496-px images, in 32 bits
        _norm(name="norm_train_hires", rows=2 * 24337, C=768, train=True, dtype="fp32"),
        # one token of 64 sequences while serving
        {"op": "conv_step", "name": "conv_step", "dtype": "bf16", "B": 64, "D": 2048, "K": 4, "act": "silu"},
        # ragged prompts of up to 4096 tokens, with the states that decoding goes on from
        _conv(name="conv_prompts", B=16, L=4096, D=1024, ragged=True, state=True),
        # a training step of a ViT-B block's convolution, on one half of the in-projection
        _conv(name="conv_train_vit", B=64, L=197, D=1536, train=True, view=True),
        # one token of one sequence: latency
        {"op": "scan_step", "name": "scan_step_one", "dtype": "bf16", "B": 1, "D": 384, "N": 16, "G": 1, "gate": True},
        # one token of 256 sequences: the states' traffic
        {"op": "scan_step", "name": "scan_step_batch", "dtype": "bf16", "B": 256, "D": 2048, "N": 16, "G": 1,
         "gate": True},
        # two 2496-px images: few rows, a long axis
        _scan(name="scan_hires", B=2, L=24337, D=1536, R=96),
        # ragged prompts that go on from states and leave states
        _scan(name="scan_prompts", B=16, L=4096, D=1024, R=64, ragged=True, state=True),
        # a training step of a ViT-B block's scan
        _scan(name="scan_train_vit", B=64, L=197, D=1536, R=96, train=True),
        # odd sizes, a wide state, two groups, right to left, from a state, in 32 bits
        _scan(name="scan_train_odd", B=3, L=1021, D=330, N=64, G=2, R=21, train=True, dtype="fp32", state=True,
              reverse=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("norm", "norm", "conv", "conv", "conv_step", "scan", "scan", "scan", "scan_step"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    coin = lambda: rng.random() < 0.5  # noqa: E731
    if op == "norm":
        C = rng.choice((rng.choice((192, 512, 768, 1024, 2048)), _log_int(rng, 48, 8192)))
        train = coin()
        rows = _log_int(rng, 1, max(1, min(100000, (2 * 24337 * 768) // C)))
        return _norm(rows=rows, C=C, train=train, dtype=dtype, bias=rng.random() < 0.8)
    if op == "conv_step":
        return {"op": op, "dtype": dtype, "B": _log_int(rng, 1, 256), "D": _log_int(rng, 64, 2048),
                "K": rng.choice((2, 3, 4)), "act": rng.choice(("silu", "none"))}
    D = rng.choice((rng.choice((384, 1024, 1536, 2048)), _log_int(rng, 32, 2048)))
    if op == "conv":
        train = coin()
        most = 16 * 4096 * 1024 // (2 if train else 1)
        L = _log_int(rng, 1, 24337)
        B = _log_int(rng, 1, max(1, min(64, most // (L * D))))
        return _conv(B=B, L=L, D=D, K=rng.choice((2, 3, 4)), act=rng.choice(("silu", "silu", "none")), dtype=dtype,
                     train=train, ragged=coin(), state=coin(), reverse=coin(), view=coin())
    N = rng.choice((8, 16, 16, 32, 64))
    G = rng.choice((1, 1, 2, 3))
    D = max(G, D // G * G)
    if op == "scan_step":
        return {"op": op, "dtype": dtype, "B": _log_int(rng, 1, 256), "D": D, "N": N, "G": G, "gate": coin()}
    train = coin()
    most = 64 * 197 * 1536 * 16 if train else 2 * 24337 * 1536 * 16
    L = max(1, min(_log_int(rng, 1, 24337), most // (D * N)))
    B = _log_int(rng, 1, max(1, min(64, most // (L * D * N))))
    return _scan(B=B, L=L, D=D, N=N, G=G, R=rng.choice((0, D // 16 // 8 * 8, D // 16)), dtype=dtype, train=train,
                 gate=rng.random() < 0.8, ragged=coin(), state=coin(), reverse=coin())


# ------------------------------------------------------------------ inputs

def _lengths(c):
    """The lengths of a ragged batch: evenly spread from one token to all L."""
    B, L = c["B"], c["L"]
    if not c["ragged"]:
        return [L] * B
    return [1 + (L - 1) * i // max(1, B - 1) for i in range(B)] if B > 1 else [(L + 1) // 2]


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    T = _DTYPES[c["dtype"]]
    f32 = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    uni = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    s = {"case": dict(c)}
    if c["op"] == "norm":
        rows, C = c["rows"], c["C"]
        s["x"] = (0.5 + 2.0 * f32(rows, C)).to(T)
        s["weight"], s["bias"] = 1 + 0.1 * f32(C), 0.1 * f32(C) if c["bias"] else None
        if c["train"]:
            s["dy"] = f32(rows, C).to(T)
        return s
    D = c["D"]
    if c["op"] == "conv_step":
        s["x"], s["state"] = f32(c["B"], D).to(T), f32(c["B"], c["K"] - 1, D).to(T)
        s["weight"], s["bias"] = 0.5 * f32(D, c["K"]), 0.1 * f32(D)
        return s
    if c["op"] in ("conv", "scan"):
        B, L = c["B"], c["L"]
        s["lengths"] = None
        if c["ragged"]:
            order = torch.randperm(B, generator=g, device="cuda")
            s["lengths"] = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")[order].contiguous()
    if c["op"] == "conv":
        # in a model x is one half of the in-projection's output
        s["x"] = f32(B, L, 2 * D).to(T)[..., :D] if c["view"] else f32(B, L, D).to(T)
        s["weight"], s["bias"] = 0.5 * f32(D, c["K"]), 0.1 * f32(D)
        s["state"] = f32(B, c["K"] - 1, D).to(T) if c["state"] else None
        if c["train"]:
            s["dy"] = f32(B, L, D).to(T)
        return s
    N, G = c["N"], c["G"]
    s["A"] = -(torch.arange(1, N + 1, device="cuda") * torch.exp(0.1 * f32(D, N)))
    s["Dskip"] = 1 + 0.1 * f32(D)
    step = torch.exp(math.log(1e-3) + (math.log(1e-1) - math.log(1e-3)) * uni(D))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus of it is the step
    if c["op"] == "scan_step":
        B = c["B"]
        s["h"] = 0.3 * f32(B, D, N)
        s["u"], s["dt"] = f32(B, D).to(T), (0.5 * f32(B, D)).to(T)
        s["z"] = f32(B, D).to(T) if c["gate"] else None
        s["Bm"], s["Cm"] = f32(B, G, N).to(T), f32(B, G, N).to(T)
        return s
    # in a model u is the convolution's output, z one half of the in-projection's, and B and C lie behind the
    # low-rank step size in one projection's output
    s["u"], s["dt"] = f32(B, L, D).to(T), (0.5 * f32(B, L, D)).to(T)
    s["z"] = f32(B, L, 2 * D).to(T)[..., D:] if c["gate"] else None
    R = c["R"]
    xp = f32(B, L, R + 2 * G * N).to(T)
    s["Bm"] = xp[..., R:R + G * N].unflatten(2, (G, N))
    s["Cm"] = xp[..., R + G * N:].unflatten(2, (G, N))
    s["h0"] = 0.3 * f32(B, D, N) if c["state"] else None
    if c["train"]:
        s["dout"] = f32(B, L, D).to(T)
    return s


# ------------------------------------------------------------- plain forms

def _plain_norm(s, c):
    x, w, T = s["x"].float(), s["weight"], s["x"].dtype
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    rstd = 1 / torch.sqrt((xc * xc).mean(-1, keepdim=True) + _EPS)
    xh = xc * rstd
    y = xh * w if s["bias"] is None else xh * w + s["bias"]
    if not c["train"]:
        return {"y": y.to(T)}
    dy = s["dy"].float()
    gy = dy * w
    dx = rstd * (gy - gy.mean(-1, keepdim=True) - xh * (gy * xh).mean(-1, keepdim=True))
    return {"y": y.to(T), "dx": dx.to(T), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0) if c["bias"] else None}


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _plain_conv_step(s, c):
    win = torch.cat((s["state"].float(), s["x"].float().unsqueeze(1)), 1)  # [B, K, D], the new token last
    p = (win * s["weight"].t()).sum(1) + s["bias"]
    y = p * _sigmoid(p) if c["act"] == "silu" else p
    s["state"].copy_(win[:, 1:])
    return {"y": y.to(s["x"].dtype), "state": s["state"]}


def _order(s, c):
    """(token at each processing index [B, L], which of them there are): a sequence's own tokens first, from its
    last one where it runs in reverse."""
    L = c["L"]
    i = torch.arange(L, device="cuda")
    n = torch.full((c["B"], 1), L, device="cuda") if s["lengths"] is None else s["lengths"].long().unsqueeze(1)
    valid = i < n
    at = torch.where(valid, n - 1 - i, i) if c["reverse"] else i.expand(c["B"], L)
    return at, valid


def _take(x, at):
    return x[torch.arange(x.shape[0], device=x.device).unsqueeze(1), at]


def _plain_conv(s, c):
    T, K, B, D = s["x"].dtype, c["K"], c["B"], c["D"]
    plain = s["lengths"] is None and not c["reverse"]
    x = s["x"].float()
    if not plain:
        at, valid = _order(s, c)
        keep = valid.unsqueeze(-1)
        x = torch.where(keep, _take(x, at), 0.0)
    first = torch.zeros(B, K - 1, D, device="cuda") if s["state"] is None else s["state"].float()
    xp = torch.cat((first, x), 1)
    win = xp.unfold(1, K, 1)  # [B, L, D, K]
    p = (win * s["weight"]).sum(-1) + s["bias"]
    sg = _sigmoid(p) if c["act"] == "silu" else None
    y = p if sg is None else p * sg
    y = y if plain else _take(torch.where(keep, y, 0.0), at)
    out = {"y": y.to(T)}
    if c["state"]:
        n = torch.full((B,), c["L"], device="cuda") if s["lengths"] is None else s["lengths"].long()
        out["state"] = _take(xp, n.unsqueeze(1) + torch.arange(K - 1, device="cuda")).to(T)
    if not c["train"]:
        return out
    dp = s["dy"].float()
    dp = dp if plain else torch.where(keep, _take(dp, at), 0.0)
    dp = dp if sg is None else dp * sg * (1 + p * (1 - sg))
    pad = torch.zeros(B, K - 1, D, device="cuda")
    dxp = (torch.cat((pad, dp, pad), 1).unfold(1, K, 1) * s["weight"].flip(1)).sum(-1)  # [B, K - 1 + L, D]
    dx = dxp[:, K - 1:]
    out["dx"] = (dx if plain else _take(torch.where(keep, dx, 0.0), at)).to(T)
    out["dweight"] = (win * dp.unsqueeze(-1)).sum((0, 1))
    out["dbias"] = dp.sum((0, 1))
    if c["state"]:
        out["dstate"] = dxp[:, :K - 1].to(T)
    return out


def _silu(x):
    return x * _sigmoid(x)


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _plain_scan_step(s, c):
    G, N, D = c["G"], c["N"], c["D"]
    u, dt = s["u"].float(), _softplus(s["dt"].float() + s["dt_bias"])
    Bm = s["Bm"].float().repeat_interleave(D // G, 1)
    Cm = s["Cm"].float().repeat_interleave(D // G, 1)
    h = torch.exp(dt.unsqueeze(-1) * s["A"]) * s["h"] + (dt * u).unsqueeze(-1) * Bm
    y = (h * Cm).sum(-1) + s["Dskip"] * u
    y = y if s["z"] is None else y * _silu(s["z"].float())
    s["h"].copy_(h)
    return {"out": y.to(s["u"].dtype), "h": s["h"]}


def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 by doubling, in log2(L) rounds; takes a and b as its own."""
    r, L = 1, a.shape[1]
    while r < L:
        b[:, r:] += a[:, r:] * b[:, :-r]
        a[:, r:] = a[:, r:] * a[:, :-r]
        r *= 2
    return b


def _plain_scan(s, c):
    T, B, L, D, N, G = s["u"].dtype, c["B"], c["L"], c["D"], c["N"], c["G"]
    plain = s["lengths"] is None and not c["reverse"]
    at, valid = (None, None) if plain else _order(s, c)
    keep = None if plain else valid.unsqueeze(-1)
    take = lambda x: x if plain else torch.where(keep, _take(x, at), 0.0)  # noqa: E731
    back = lambda x: x if plain else _take(torch.where(keep, x, 0.0), at)  # noqa: E731
    u, raw = take(s["u"].float()), take(s["dt"].float()) + s["dt_bias"]
    dt = _softplus(raw) if plain else torch.where(keep, _softplus(raw), 0.0)
    heads = lambda x: x.unflatten(2, (G, D // G))  # noqa: E731
    Bm = take(s["Bm"].float().flatten(2)).unflatten(2, (G, 1, N))  # [B, L, G, 1, N] against [B, L, G, D/G, N]
    Cm = take(s["Cm"].float().flatten(2)).unflatten(2, (G, 1, N))
    A = s["A"].view(G, D // G, N)
    a = torch.exp(heads(dt).unsqueeze(-1) * A)
    b = heads(dt * u).unsqueeze(-1) * Bm
    h0 = None if s["h0"] is None else s["h0"].view(B, G, D // G, N)
    if h0 is not None:
        b[:, 0] += a[:, 0] * h0
    keep_a = a.clone() if c["train"] else None
    h = _recur(a, b)
    del a
    y = (h * Cm).sum(-1).flatten(2) + s["Dskip"] * u
    if s["z"] is None:
        z = sz = None
        out = y
    else:
        z = take(s["z"].float())
        sz = _sigmoid(z)
        out = y * z * sz
    res = {"out": back(out).to(T)}
    if c["state"]:
        res["h"] = h[:, -1].reshape(B, D, N).clone()
    if not c["train"]:
        return res
    a = keep_a
    dout = take(s["dout"].float())
    dy = dout if z is None else dout * z * sz
    g = (heads(dy).unsqueeze(-1) * Cm).flip(1)
    later = torch.cat((torch.zeros_like(a[:, :1]), a.flip(1)[:, :-1]), 1)
    g = _recur(later, g).flip(1)
    del later
    first = torch.zeros(B, 1, G, D // G, N, device="cuda") if h0 is None else h0.unsqueeze(1)
    q = g * a * torch.cat((first, h[:, :-1]), 1)
    gB = (g * Bm).sum(-1).flatten(2)
    ddt = (q * A).sum(-1).flatten(2) + gB * u
    ddt = ddt * _sigmoid(raw) if plain else torch.where(keep, ddt * _sigmoid(raw), 0.0)
    res["du"] = back(s["Dskip"] * dy + dt * gB).to(T)
    res["ddt"] = back(ddt).to(T)
    res["dA"] = (q * heads(dt).unsqueeze(-1)).sum((0, 1)).view(D, N)
    dB = (g * heads(dt * u).unsqueeze(-1)).sum(3).flatten(2)
    dC = (h * heads(dy).unsqueeze(-1)).sum(3).flatten(2)
    res["dB"], res["dC"] = back(dB).unflatten(2, (G, N)).to(T), back(dC).unflatten(2, (G, N)).to(T)
    res["dDskip"] = (dy * u).sum((0, 1))
    res["ddt_bias"] = ddt.sum((0, 1))
    if z is not None:
        res["dz"] = back(dout * y * sz * (1 + z * (1 - sz))).to(T)
    if h0 is not None:
        res["dh0"] = (a[:, 0] * g[:, 0]).reshape(B, D, N)
    return res


# ------------------------------------------------------ the framework's own

def _own_norm(s, c):
    from bidirectional_masked_linear_gb300 import ssm
    if not c["train"]:
        return {"y": ssm.layernorm_fwd(s["x"], s["weight"], s["bias"], eps=_EPS)}
    y, mean, rstd = ssm.layernorm_fwd(s["x"], s["weight"], s["bias"], eps=_EPS, save_stats=True)
    dx, dw, db = ssm.layernorm_bwd(s["dy"], s["x"], s["weight"], mean, rstd, bias=c["bias"])
    return {"y": y, "dx": dx, "dweight": dw, "dbias": db}


def _own_conv_step(s, c):
    from bidirectional_masked_linear_gb300 import ssm
    y = ssm.conv_step(s["x"], s["state"], s["weight"], s["bias"], activation=c["act"])
    return {"y": y, "state": s["state"]}


def _own_conv(s, c):
    from bidirectional_masked_linear_gb300 import ssm
    kw = dict(activation=c["act"], state=s["state"], lengths=s["lengths"], reverse=c["reverse"])
    out = {}
    if c["state"]:
        out["y"], out["state"] = ssm.conv_fwd(s["x"], s["weight"], s["bias"], return_state=True, **kw)
    else:
        out["y"] = ssm.conv_fwd(s["x"], s["weight"], s["bias"], **kw)
    if c["train"]:
        g = ssm.conv_bwd(s["dy"], s["x"], s["weight"], s["bias"], **kw)
        out.update(dx=g.dx, dweight=g.dweight, dbias=g.dbias)
        if c["state"]:
            out["dstate"] = g.dstate
    return out


def _own_scan_step(s, c):
    from bidirectional_masked_linear_gb300 import ssm
    y = ssm.scan_step(s["h"], s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], Dskip=s["Dskip"], z=s["z"],
                      dt_bias=s["dt_bias"], dt_softplus=True)
    return {"out": y, "h": s["h"]}


def _own_scan(s, c):
    from bidirectional_masked_linear_gb300 import ssm
    ins = (s["u"], s["dt"], s["A"], s["Bm"], s["Cm"])
    kw = dict(Dskip=s["Dskip"], z=s["z"], dt_bias=s["dt_bias"], dt_softplus=True, h0=s["h0"], lengths=s["lengths"],
              reverse=c["reverse"])
    f = ssm.scan_fwd(*ins, return_state=c["state"], save_states=c["train"], **kw)
    res = {"out": f.out}
    if c["state"]:
        res["h"] = f.h
    if c["train"]:
        g = ssm.scan_bwd(s["dout"], *ins, states=f.states, **kw)
        res.update(du=g.du, ddt=g.ddt, dA=g.dA, dB=g.dB, dC=g.dC, dDskip=g.dDskip, ddt_bias=g.ddt_bias)
        if s["z"] is not None:
            res["dz"] = g.dz
        if s["h0"] is not None:
            res["dh0"] = g.dh0
    return res


_PLAIN = {"norm": _plain_norm, "conv": _plain_conv, "conv_step": _plain_conv_step, "scan": _plain_scan,
          "scan_step": _plain_scan_step}
_OWN = {"norm": _own_norm, "conv": _own_conv, "conv_step": _own_conv_step, "scan": _own_scan,
        "scan_step": _own_scan_step}


def run(state):
    c = state["case"]
    out = (_OWN if own else _PLAIN)[c["op"]](state, c)
    return {k: v for k, v in out.items() if v is not None}


# -------------------------------------------------------------------- work

def work(case):
    """Inputs once, outputs once; exponentials count as one operation."""
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"] == "norm":
        n = c["rows"] * c["C"]
        return {"bytes": n * e * (5 if c["train"] else 2) + 4 * c["C"] * (5 if c["train"] else 2),
                "flops": n * (8 + (14 if c["train"] else 0))}
    D = c["D"]
    if c["op"] == "conv_step":
        return {"bytes": c["B"] * D * e * 2 * c["K"] + 4 * D * (c["K"] + 1), "flops": c["B"] * D * (2 * c["K"] + 4)}
    if c["op"] == "scan_step":
        n = c["B"] * D
        return {"bytes": n * (8 * c["N"] + e * (4 if c["gate"] else 3)) + 4 * D * (c["N"] + 2)
                + 2 * c["B"] * c["G"] * c["N"] * e, "flops": n * (6 * c["N"] + 12)}
    full, some = c["B"] * c["L"], sum(_lengths(c))
    if c["op"] == "conv":
        by = D * e * (some + full) + (2 * c["B"] * (c["K"] - 1) * D * e if c["state"] else 0) + 4 * D * (c["K"] + 1)
        fl = some * D * (2 * c["K"] + 4)
        if c["train"]:
            by += D * e * (2 * some + full) + 8 * D * (c["K"] + 1)
            fl += some * D * (6 * c["K"] + 10)
        return {"bytes": by, "flops": fl}
    N, z = c["N"], 1 if c["gate"] else 0
    bc = 2 * c["G"] * N * e * some
    par = 4 * D * (N + 2)
    st = 8 * c["B"] * D * N if c["state"] else 0
    by, fl = D * e * ((2 + z) * some + full) + bc + par + st, some * D * (6 * N + 12)
    if c["train"]:  # the gradients read the inputs again
        by += D * e * ((3 + z) * some + (2 + z) * full) + bc + 2 * c["G"] * N * e * full + 2 * par + st
        fl += some * D * (12 * N + 25)
    return {"bytes": by, "flops": fl}


# ----------------------------------------------------------- in 64 bits

def _exact_norm(s, c):
    import numpy as np
    x, w = s["x"].double().cpu().numpy(), s["weight"].double().cpu().numpy()
    C = x.shape[1]
    mu = np.sum(x, axis=1) / C
    var = np.sum((x - mu[:, None]) ** 2, axis=1) / C
    inv = 1.0 / np.sqrt(var + _EPS)
    n = (x - mu[:, None]) * inv[:, None]
    y = n * w[None]
    if s["bias"] is not None:
        y = y + s["bias"].double().cpu().numpy()
    out = {"y": y}
    if c["train"]:
        dy = s["dy"].double().cpu().numpy()
        d = dy * w
        # the derivative of n_i in x_j is inv (delta_ij - 1/C - n_i n_j / C)
        out["dx"] = inv[:, None] * (d - d.sum(1, keepdims=True) / C - n * (d * n).sum(1, keepdims=True) / C)
        out["dweight"] = np.einsum("rc,rc->c", dy, n)
        if c["bias"]:
            out["dbias"] = dy.sum(0)
    return out


def _exact_conv(s, c):
    """Token by token from the definition; one tap and one token of every sequence at a time."""
    B, D, K = c["B"], c["D"], c["K"]
    step = c["op"] == "conv_step"
    x = s["x"].double().unsqueeze(1) if step else s["x"].double()
    L = x.shape[1]
    n = [L] * B if step or s["lengths"] is None else [int(v) for v in s["lengths"].tolist()]
    rev = not step and c["reverse"]
    w, bias = s["weight"].double(), s["bias"].double()
    st = s["state"]
    y = torch.zeros(B, L, D, dtype=torch.float64, device=x.device)
    final = torch.zeros(B, K - 1, D, dtype=torch.float64, device=x.device)
    train = not step and c["train"]
    dx, dst = torch.zeros_like(y), torch.zeros_like(final)
    dw, db = torch.zeros_like(w), torch.zeros_like(bias)
    for b in range(B):
        m = n[b]
        seq = x[b, :m].flip(0) if rev else x[b, :m]
        before = torch.zeros(K - 1, D, dtype=torch.float64, device=x.device) if st is None else st[b].double()
        line = torch.cat((before, seq))  # line[i + K - 1] is the token processed i-th
        pre = bias.expand(m, D).clone()
        for k in range(K):
            pre = pre + w[:, k] * line[k:k + m]
        val = pre / (1 + torch.exp(-pre)) if c["act"] == "silu" else pre
        y[b, :m] = val.flip(0) if rev else val
        final[b] = line[m:m + K - 1]
        if train:
            d = s["dy"][b, :m].double()
            d = d.flip(0) if rev else d
            if c["act"] == "silu":
                sg = 1 / (1 + torch.exp(-pre))
                d = d * (sg + pre * sg * (1 - sg))
            dline = torch.zeros_like(line)
            for k in range(K):
                dline[k:k + m] += w[:, k] * d
                dw[:, k] += (line[k:k + m] * d).sum(0)
            db += d.sum(0)
            dst[b] = dline[:K - 1]
            dx[b, :m] = dline[K - 1:].flip(0) if rev else dline[K - 1:]
    if step:
        return {"y": y[:, 0], "state": final}
    out = {"y": y}
    if c["state"]:
        out["state"] = final
    if train:
        out.update(dx=dx, dweight=dw, dbias=db)
        if c["state"]:
            out["dstate"] = dst
    return out


def _exact_scan(s, c):
    """The recurrence one token after the other, all sequences at once."""
    step = c["op"] == "scan_step"
    row = (lambda k: s[k].double().unsqueeze(1)) if step else (lambda k: s[k].double())
    u, raw, Bm, Cm = row("u"), row("dt") + s["dt_bias"].double(), row("Bm"), row("Cm")
    B, L, D = u.shape
    N, G = c["N"], c["G"]
    A, skip = s["A"].double(), s["Dskip"].double()
    z = None if s["z"] is None else row("z")
    n = torch.full((B,), L, device=u.device) if step or s["lengths"] is None else s["lengths"]
    rev, train = not step and c["reverse"], not step and c["train"]
    dev = u.device
    start = s["h"] if step else s["h0"]
    h = torch.zeros(B, D, N, dtype=torch.float64, device=dev) if start is None else start.double().clone()
    of = torch.arange(D, device=dev) // (D // G)
    y = torch.zeros(B, L, D, dtype=torch.float64, device=dev)
    hs = torch.zeros(L + 1 if train else 0, B, D, N, dtype=torch.float64, device=dev)
    walk = list(range(L - 1, -1, -1) if rev else range(L))
    delta = torch.log(1 + torch.exp(-raw.abs())) + torch.where(raw > 0, raw, torch.zeros_like(raw))
    for i, t in enumerate(walk):
        there = (n > t).view(B, 1, 1)
        if train:
            hs[i] = h
        d = delta[:, t].unsqueeze(-1)
        new = torch.exp(d * A) * h + d * u[:, t].unsqueeze(-1) * Bm[:, t][:, of]
        h = torch.where(there, new, h)
        y[:, t] = torch.where(there[..., 0], (new * Cm[:, t][:, of]).sum(-1) + skip * u[:, t], torch.zeros_like(u[:, t]))
    gate = None if z is None else z / (1 + torch.exp(-z))
    there = (torch.arange(L, device=dev) < n.view(B, 1)).unsqueeze(-1)
    zero = torch.zeros((), dtype=torch.float64, device=dev)
    out = torch.where(there, y if z is None else y * gate, zero)
    if step:
        return {"out": out[:, 0], "h": h}
    res = {"out": out}
    if c["state"]:
        res["h"] = h
    if not train:
        return res
    hs[L] = h
    do = torch.where(there, s["dout"].double(), zero)
    dy = do if z is None else do * gate
    du, dd = torch.zeros_like(u), torch.zeros_like(u)
    dA = torch.zeros_like(A)
    dB, dC = torch.zeros_like(Bm), torch.zeros_like(Cm)
    lam = torch.zeros(B, D, N, dtype=torch.float64, device=dev)  # the gradient of the state after the token
    for i in range(L - 1, -1, -1):
        t = walk[i]
        ok = there[:, t].unsqueeze(-1)
        d, x = delta[:, t].unsqueeze(-1), u[:, t].unsqueeze(-1)
        bt, ct = Bm[:, t][:, of], Cm[:, t][:, of]
        mine = lam + ct * dy[:, t].unsqueeze(-1)
        dC[:, t] += torch.where(ok, hs[i + 1] * dy[:, t].unsqueeze(-1), zero).unflatten(1, (G, D // G)).sum(2)
        e = torch.exp(d * A)
        dB[:, t] += torch.where(ok, mine * d * x, zero).unflatten(1, (G, D // G)).sum(2)
        de = mine * hs[i] * e
        dA += torch.where(ok, de * d, zero).sum(0)
        dd[:, t] = torch.where(ok[..., 0], (de * A + mine * x * bt).sum(-1), zero)
        du[:, t] = torch.where(ok[..., 0], (mine * d * bt).sum(-1) + skip * dy[:, t], zero)
        lam = torch.where(ok, mine * e, lam)
    dd = dd / (1 + torch.exp(-raw))
    res.update(du=du, ddt=dd, dA=dA, dB=dB, dC=dC, dDskip=torch.where(there, dy * u, zero).sum((0, 1)),
               ddt_bias=dd.sum((0, 1)))
    if z is not None:
        sg = 1 / (1 + torch.exp(-z))
        res["dz"] = torch.where(there, do * y * (sg + z * sg * (1 - sg)), zero)
    if s["h0"] is not None:
        res["dh0"] = lam
    return res


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "conv": _exact_conv, "conv_step": _exact_conv, "scan": _exact_scan,
            "scan_step": _exact_scan}[case["op"]](s, case)
