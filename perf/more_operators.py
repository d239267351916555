"""Cases of the delta rule's operators: the norms of queries and keys for each
head with the position rotation, the gated delta rule over chunks, both with
their gradients, and the delta rule's one-token step.

Lengths, head counts and widths are those of the repository's workloads
(``synth.py``): 197 tokens of 3 or 12 heads, 512 of 16, 4096 of 8 and 24337 of
12, heads of 64; heads of 128 and query heads that several value heads share
are generic.  ``run`` computes a case in plain torch operations in 32 bits, or,
where ``own`` is true, through ``bidirectional_masked_linear_gb300.delta``.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_EPS = 1e-6
_CHUNK = 64


# ------------------------------------------------------------------- cases

def _qknorm(**kw):
    return {"op": "qknorm", "dtype": "bf16", "train": False, "norm": "l2", "weight": False, "rot": 0,
            "interleaved": False, "far": False, **kw}


def _delta(**kw):
    return {"op": "delta", "dtype": "bf16", "train": False, "ragged": False, "state": False, "reverse": False, **kw}


def listed():
    return [
        # one token of 64 sequences that are at different places: latency
        _qknorm(name="qknorm_step", B=64, L=1, Hq=16, Hk=16, d=64, norm="rms", weight=True, rot=64, far=True),
        # a training step of a BERT-large block's queries and keys
        _qknorm(name="qknorm_train_bert", B=32, L=512, Hq=16, Hk=16, d=64, norm="rms", weight=True, rot=64, train=True),
        # two 2496-px images' queries and keys ahead of the delta rule
        _qknorm(name="qknorm_hires", B=2, L=24337, Hq=12, Hk=12, d=64),
        # odd sizes, adjacent pairs, part of a head rotated, in 32 bits
        _qknorm(name="qknorm_train_odd", B=5, L=1021, Hq=6, Hk=2, d=72, norm="rms", weight=True, rot=48,
                interleaved=True, far=True, train=True, dtype="fp32"),
        # one token of one sequence: latency
        {"op": "delta_step", "name": "delta_step_one", "dtype": "bf16", "B": 1, "Hk": 12, "Hv": 12, "dk": 64, "dv": 64},
        # one token of 256 sequences: the states' traffic
        {"op": "delta_step", "name": "delta_step_batch", "dtype": "bf16", "B": 256, "Hk": 8, "Hv": 16, "dk": 128,
         "dv": 128},
        # one image through the smallest model: a short chain
        _delta(name="delta_one_image", B=1, L=197, Hk=3, Hv=3, dk=64, dv=64),
        # a training step of a ViT-B block
        _delta(name="delta_train_vit", B=64, L=197, Hk=12, Hv=12, dk=64, dv=64, train=True),
        # a training step on texts of 4096 tokens
        _delta(name="delta_train_text", B=16, L=4096, Hk=8, Hv=8, dk=64, dv=64, train=True),
        # two 2496-px images: few heads, a long chain
        _delta(name="delta_hires", B=2, L=24337, Hk=12, Hv=12, dk=64, dv=64),
        # ragged prompts that go on from states and leave states, wide heads, two value heads a query head
        _delta(name="delta_prompts", B=16, L=4096, Hk=4, Hv=8, dk=128, dv=128, ragged=True, state=True),
        # odd sizes, three value heads a query head, right to left, from a state, in 32 bits
        _delta(name="delta_train_odd", B=3, L=1021, Hk=2, Hv=6, dk=40, dv=72, train=True, dtype="fp32", state=True,
               reverse=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("qknorm", "qknorm", "delta", "delta", "delta", "delta", "delta_step"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    coin = lambda: rng.random() < 0.5  # noqa: E731
    Hk, group = _log_int(rng, 1, 16), rng.choice((1, 1, 2, 3))
    if op == "qknorm":
        d = rng.choice((64, 64, 128, 8 * rng.randint(2, 32)))
        L = _log_int(rng, 1, 24337)
        most = 2 * 24337 * 24 * 64 // (2 if dtype == "fp32" else 1)
        heads = (1 + group) * Hk
        B = _log_int(rng, 1, max(1, min(64, most // (L * heads * d))))
        L = max(1, min(L, most // (heads * d)))
        return _qknorm(B=B, L=L, Hq=group * Hk, Hk=Hk, d=d, norm=rng.choice(("l2", "rms")), weight=coin(),
                       rot=rng.choice((0, d, 8 * rng.randint(1, d // 8))), interleaved=coin(), far=coin(),
                       train=coin(), dtype=dtype)
    dk, dv = (rng.choice((64, 64, 128, 8 * rng.randint(2, 16))) for _ in range(2))
    if op == "delta_step":
        return {"op": op, "dtype": dtype, "B": _log_int(rng, 1, 256 // group), "Hk": Hk, "Hv": group * Hk, "dk": dk,
                "dv": dv}
    train = coin()
    per = group * Hk * dk * dv
    most = (16 * 4096 * 8 * 64 * 64 if train else 2 * 24337 * 12 * 64 * 64) // (4 if dtype == "fp32" else 1)
    L = max(1, min(_log_int(rng, 1, 24337), most // per))
    B = _log_int(rng, 1, max(1, min(64, most // (L * per))))
    return _delta(B=B, L=L, Hk=Hk, Hv=group * Hk, dk=dk, dv=dv, dtype=dtype, train=train, ragged=coin(), state=coin(),
                  reverse=coin())


# ------------------------------------------------------------------ inputs

def _lengths(c):
    """The lengths of a ragged batch: evenly spread from one token to all L."""
    B, L = c["B"], c["L"]
    if not c["ragged"]:
        return [L] * B
    return [1 + (L - 1) * i // max(1, B - 1) for i in range(B)] if B > 1 else [(L + 1) // 2]


def _frequencies(rot):
    return torch.tensor([10000.0 ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float32, device="cuda")


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    T = _DTYPES[c["dtype"]]
    f32 = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    uni = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    s = {"case": dict(c)}
    B = c["B"]
    if c["op"] == "qknorm":
        L, Hq, Hk, d, rot = c["L"], c["Hq"], c["Hk"], c["d"], c["rot"]
        # in a model queries and keys are slices of one projection's output
        qk = (1.5 * f32(B, L, (Hq + Hk) * d)).to(T)
        s["q"] = qk[..., :Hq * d].unflatten(2, (Hq, d))
        s["k"] = qk[..., Hq * d:].unflatten(2, (Hk, d))
        s["wq"] = 1 + 0.1 * f32(d) if c["weight"] else None
        s["wk"] = 1 + 0.1 * f32(d) if c["weight"] else None
        s["freqs"] = _frequencies(rot) if rot else None
        s["positions"] = None
        if rot and c["far"]:  # sequences that go on from where they are, up to a million tokens in
            start = (1e6 * uni(B, 1)).to(torch.int32)
            s["positions"] = (start + torch.arange(L, dtype=torch.int32, device="cuda")).contiguous()
        if c["train"]:
            s["dqo"], s["dko"] = f32(B, L, Hq, d).to(T), f32(B, L, Hk, d).to(T)
        return s
    step = c["op"] == "delta_step"
    at = (B,) if step else (B, c["L"])
    Hk, Hv, dk, dv = c["Hk"], c["Hv"], c["dk"], c["dv"]
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    s["q"], s["k"] = unit(f32(*at, Hk, dk)).to(T), unit(f32(*at, Hk, dk)).to(T)
    logsig = lambda x: -torch.log1p(torch.exp(-x))  # noqa: E731
    decay, beta = logsig(3 + f32(*at, Hv)).to(T), torch.sigmoid(f32(*at, Hv)).to(T)
    if step:
        s["v"], s["g"], s["beta"] = f32(B, Hv, dv).to(T), decay, beta
        s["h"] = 0.3 * f32(B, Hv, dk, dv)
        return s
    # in a model the values are a slice of a convolution's output
    L = c["L"]
    s["v"] = f32(B, L, Hv * dv + Hk * dk).to(T)[..., Hk * dk:].unflatten(2, (Hv, dv))
    s["g"], s["beta"] = decay, beta
    s["lengths"] = None
    if c["ragged"]:
        order = torch.randperm(B, generator=g, device="cuda")
        s["lengths"] = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")[order].contiguous()
    s["h0"] = 0.3 * f32(B, Hv, dk, dv) if c["state"] else None
    if c["train"]:
        s["dout"] = f32(B, L, Hv, dv).to(T)
    return s


# ------------------------------------------------------------- plain forms

def _angles(s, c):
    """cos and sin of position times frequency, [B or 1, L, 1, rot / 2]; the angle in 64 bits."""
    p = torch.arange(c["L"], device="cuda").unsqueeze(0) if s["positions"] is None else s["positions"]
    a = p.double().unsqueeze(-1) * s["freqs"].double()
    return torch.cos(a).float().unsqueeze(2), torch.sin(a).float().unsqueeze(2)


def _rotate(x, cos, sin, c):
    rot = c["rot"]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_qknorm(s, c):
    T, d = s["q"].dtype, c["d"]
    n = 1 if c["norm"] == "l2" else d
    cos, sin = _angles(s, c) if c["rot"] else (None, None)
    out = {}
    for name, w in (("q", s["wq"]), ("k", s["wk"])):
        x = s[name].float()
        r = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / n + _EPS)
        xh = x * r
        y = xh if w is None else xh * w
        out[name + "o"] = (_rotate(y, cos, sin, c) if c["rot"] else y).to(T)
        if c["train"]:
            dy = s["d" + name + "o"].float()
            dy = _rotate(dy, cos, -sin, c) if c["rot"] else dy
            g = dy if w is None else dy * w
            out["d" + name] = (r * (g - xh * ((g * xh).sum(-1, keepdim=True) / n))).to(T)
            out["dw" + name] = None if w is None else (dy * xh).sum((0, 1, 2))
    return out


def _plain_delta_step(s, c):
    group = c["Hv"] // c["Hk"]
    q, k = (s[x].float().repeat_interleave(group, 1) for x in ("q", "k"))
    h = torch.exp(s["g"].float())[..., None, None] * s["h"]
    u = s["beta"].float().unsqueeze(-1) * (s["v"].float() - (h * k.unsqueeze(-1)).sum(2))
    h = h + k.unsqueeze(-1) * u.unsqueeze(2)
    out = (h * q.unsqueeze(-1)).sum(2) * c["dk"] ** -0.5
    s["h"].copy_(h)
    return {"out": out.to(s["v"].dtype), "h": s["h"]}


def _order(s, c):
    """(token at each processing index [B, L], which of them there are): a sequence's own tokens first, from its
    last one where it runs in reverse."""
    L = c["L"]
    i = torch.arange(L, device="cuda")
    n = torch.full((c["B"], 1), L, device="cuda") if s["lengths"] is None else s["lengths"].long().unsqueeze(1)
    valid = i < n
    at = torch.where(valid, n - 1 - i, i) if c["reverse"] else i.expand(c["B"], L)
    return at, valid


def _chunks(x, pad):
    """[B, L, H, ...] to [B, H, chunks, 64, ...], padded with zeros."""
    x = torch.cat((x, x.new_zeros(x.shape[0], pad, *x.shape[2:])), 1) if pad else x
    return x.transpose(1, 2).unflatten(2, (-1, _CHUNK))


def _chunkwise(q, k, v, g, beta, h0, c):
    """(out, state) of the rule on [B, L, H, .] in chunks of 64.  Within a chunk, with G the decays' sums, the
    corrected values R solve  R_i = v_i - e^G_i S^T k_i - sum_{j < i} e^(G_i - G_j) (k_i . k_j) beta_j R_j."""
    B, L, Hk, dk = q.shape
    H, dv, group = v.shape[2], v.shape[3], v.shape[2] // Hk
    pad = -L % _CHUNK
    q, k, v, g, beta = (_chunks(x, pad) for x in (q, k, v, g, beta))
    q, k = (x.repeat_interleave(group, 1) for x in (q * dk ** -0.5, k))
    G = torch.cumsum(g.double(), -1)
    lower = torch.ones(_CHUNK, _CHUNK, dtype=torch.bool, device=q.device).tril()
    D = torch.exp((G.unsqueeze(-1) - G.unsqueeze(-2)).masked_fill(~lower, -math.inf)).float()
    grown, left = torch.exp(G).float().unsqueeze(-1), torch.exp(G[..., -1:] - G).float()
    last = grown[..., -1:, :]
    eye = torch.eye(_CHUNK, device=q.device)
    M = (k @ k.transpose(-1, -2)) * (D - eye) * beta.unsqueeze(-2)
    inv = torch.linalg.solve_triangular(eye + M, eye, upper=False, unitriangular=True)
    P = (q @ k.transpose(-1, -2)) * D * beta.unsqueeze(-2)
    kin, qin, kout = k * grown, q * grown, (k * (left * beta).unsqueeze(-1)).transpose(-1, -2)
    own_part = inv @ v
    kin = inv @ kin
    S = torch.zeros(B, H, dk, dv, device=q.device) if h0 is None else h0
    outs = []
    for j in range(q.shape[2]):
        R = own_part[:, :, j] - kin[:, :, j] @ S
        outs.append(qin[:, :, j] @ S + P[:, :, j] @ R)
        S = last[:, :, j] * S + kout[:, :, j] @ R
    return torch.cat(outs, 2).transpose(1, 2)[:, :L], S


def _plain_delta(s, c):
    T = s["q"].dtype
    names = ("q", "k", "v", "g", "beta")
    ins = [s[x].float().detach() for x in names]
    h0 = s["h0"]
    leaves = [x.requires_grad_(c["train"]) if x is not s[n] else x.clone().requires_grad_(c["train"])
              for n, x in zip(names, ins)]
    if h0 is not None and c["train"]:
        h0 = h0.clone().requires_grad_()
    straight = s["lengths"] is None and not c["reverse"]
    with torch.set_grad_enabled(c["train"]):
        walked, row = leaves, None
        if not straight:
            at, valid = _order(s, c)
            row = torch.arange(c["B"], device="cuda").unsqueeze(1)
            walked = [torch.where(valid.view(*valid.shape, *[1] * (x.dim() - 2)), x[row, at], 0.0) for x in leaves]
        y, h = _chunkwise(*walked, h0, c)
        if not straight:
            y = torch.where(valid[..., None, None], y, 0.0)[row, at]
    out = {"out": y.detach().to(T)}
    if c["state"]:
        out["h"] = h.detach()
    if c["train"]:
        wrt = leaves + ([h0] if h0 is not None else [])
        grads = torch.autograd.grad(y, wrt, s["dout"].float())
        out.update({"d" + n: x.to(T) for n, x in zip(names, grads)})
        if h0 is not None:
            out["dh0"] = grads[-1]
    return out


# ------------------------------------------------------ the framework's own

def _own_qknorm(s, c):
    from bidirectional_masked_linear_gb300 import delta
    kw = dict(q_weight=s["wq"], k_weight=s["wk"], norm=c["norm"], eps=_EPS, freqs=s["freqs"],
              positions=s["positions"], interleaved=c["interleaved"])
    out = {}
    out["qo"], out["ko"] = delta.qknorm_fwd(s["q"], s["k"], **kw)
    if c["train"]:
        g = delta.qknorm_bwd(s["dqo"], s["dko"], s["q"], s["k"], **kw)
        out.update(dq=g.dq, dk=g.dk, dwq=g.dq_weight, dwk=g.dk_weight)
    return out


def _own_delta_step(s, c):
    from bidirectional_masked_linear_gb300 import delta
    return {"out": delta.delta_step(s["h"], s["q"], s["k"], s["v"], s["g"], s["beta"]), "h": s["h"]}


def _own_delta(s, c):
    from bidirectional_masked_linear_gb300 import delta
    ins = (s["q"], s["k"], s["v"], s["g"], s["beta"])
    kw = dict(h0=s["h0"], lengths=s["lengths"], reverse=c["reverse"])
    f = delta.delta_fwd(*ins, return_state=c["state"], save=c["train"], **kw)
    out = {"out": f.out}
    if c["state"]:
        out["h"] = f.h
    if c["train"]:
        g = delta.delta_bwd(s["dout"], *ins, saved=f.saved, **kw)
        out.update(dq=g.dq, dk=g.dk, dv=g.dv, dg=g.dg, dbeta=g.dbeta)
        if s["h0"] is not None:
            out["dh0"] = g.dh0
    return out


_PLAIN = {"qknorm": _plain_qknorm, "delta": _plain_delta, "delta_step": _plain_delta_step}
_OWN = {"qknorm": _own_qknorm, "delta": _own_delta, "delta_step": _own_delta_step}


def run(state):
    c = state["case"]
    out = (_OWN if own else _PLAIN)[c["op"]](state, c)
    return {k: v for k, v in out.items() if v is not None}


# -------------------------------------------------------------------- work

def work(case):
    """Inputs once, outputs once; the delta rule's products are those of the recurrence, token by token."""
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"] == "qknorm":
        n = c["B"] * c["L"] * (c["Hq"] + c["Hk"]) * c["d"]
        return {"bytes": n * e * (5 if c["train"] else 2) + (4 * c["B"] * c["L"] if c["far"] and c["rot"] else 0),
                "flops": n * (7 + (15 if c["train"] else 0))}
    Hk, Hv, dk, dv = c["Hk"], c["Hv"], c["dk"], c["dv"]
    token = 2 * Hk * dk + 2 * Hv * dv + 2 * Hv
    state, product = 4 * c["B"] * Hv * dk * dv, 2 * Hv * dk * dv
    if c["op"] == "delta_step":
        return {"bytes": c["B"] * e * token + 2 * state, "flops": 3 * c["B"] * product}
    full, some = c["B"] * c["L"], sum(_lengths(c))
    by = e * (some * (token - Hv * dv) + full * Hv * dv) + (2 * state if c["state"] else 0)
    fl = 3 * some * product
    if c["train"]:  # the gradients read the inputs and their own again and write as much
        by += e * (some * token + full * (token - Hv * dv)) + (2 * state if c["state"] else 0)
        fl += 8 * some * product
    return {"bytes": by, "flops": fl}


# ----------------------------------------------------------- in 64 bits

def _exact_qknorm(s, c):
    import numpy as np
    d, rot, L = c["d"], c["rot"], c["L"]
    if rot:
        pos = np.arange(L)[None] if s["positions"] is None else s["positions"].cpu().numpy()
        z = np.exp(1j * pos[:, :, None, None] * s["freqs"].double().cpu().numpy())  # a pair as a complex number
        first, second = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if c["interleaved"] else \
            (np.arange(rot // 2), np.arange(rot // 2, rot))

    def turn(x, by):
        x = x.copy()
        pair = (x[..., first] + 1j * x[..., second]) * by
        x[..., first], x[..., second] = pair.real, pair.imag
        return x

    res = {}
    for name, weight in (("q", s["wq"]), ("k", s["wk"])):
        x = s[name].double().cpu().numpy()
        w = np.ones(d) if weight is None else weight.double().cpu().numpy()
        size = np.einsum("blhd,blhd->blh", x, x) / (d if c["norm"] == "rms" else 1)
        scale = (size + _EPS) ** -0.5
        y = x * scale[..., None] * w
        res[name + "o"] = turn(y, z) if rot else y
        if not c["train"]:
            continue
        dy = s["d" + name + "o"].double().cpu().numpy()
        dy = turn(dy, np.conj(z)) if rot else dy
        # the derivative of scale in x_j is -scale^3 x_j / n
        along = np.einsum("blhd,blhd->blh", dy * w, x) * scale ** 3 / (d if c["norm"] == "rms" else 1)
        res["d" + name] = scale[..., None] * dy * w - along[..., None] * x
        if weight is not None:
            res["dw" + name] = np.einsum("blhd,blhd,blh->d", dy, x, scale)
    return res


def _exact_delta(s, c):
    """The recurrence one token after the other, all sequences and heads at once."""
    step, train = c["op"] == "delta_step", c.get("train", False)
    row = (lambda n: s[n].double().unsqueeze(1)) if step else (lambda n: s[n].double())
    q, k, v, g, beta = (row(n) for n in ("q", "k", "v", "g", "beta"))
    B, L, Hv, dv = v.shape
    Hk, dk = q.shape[2:]
    of = torch.arange(Hv, device=v.device) // (Hv // Hk)
    scale = 1 / math.sqrt(dk)
    n = torch.full((B,), L, device=v.device) if step or s["lengths"] is None else s["lengths"].long()
    ids = torch.arange(B, device=v.device)
    start = s["h"] if step else s["h0"]
    S = torch.zeros(B, Hv, dk, dv, dtype=torch.float64, device=v.device) if start is None else start.double().clone()
    out = torch.zeros_like(v)
    kept = torch.empty(L if train else 0, *S.shape, dtype=torch.float64, device=v.device)

    def token(i):
        there = i < n
        t = torch.where(there, n - 1 - i, i) if not step and c["reverse"] else torch.full_like(n, i)
        return there, t, q[ids, t][:, of], k[ids, t][:, of], v[ids, t], torch.exp(g[ids, t]), beta[ids, t]

    for i in range(L):
        there, t, qi, ki, vi, a, b = token(i)
        if train:
            kept[i] = S
        old = a[..., None, None] * S
        miss = vi - torch.einsum("bhkv,bhk->bhv", old, ki)
        new = old + torch.einsum("bhk,bhv->bhkv", ki, b.unsqueeze(-1) * miss)
        ok = there.view(B, 1, 1, 1)
        S = torch.where(ok, new, S)
        o = scale * torch.einsum("bhkv,bhk->bhv", S, qi)
        out[ids, t] = torch.where(ok[..., 0], o, torch.zeros_like(o))
    if step:
        return {"out": out[:, 0], "h": S}
    res = {"out": out}
    if c["state"]:
        res["h"] = S
    if not train:
        return res
    dq, dk_, dvv, dg, db = (torch.zeros_like(x) for x in (q, k, v, g, beta))
    later = torch.zeros_like(S)
    for i in range(L - 1, -1, -1):
        there, t, qi, ki, vi, a, b = token(i)
        ok = there.view(B, 1, 1, 1)
        before = kept[i]
        old = a[..., None, None] * before
        miss = vi - torch.einsum("bhkv,bhk->bhv", old, ki)
        u = b.unsqueeze(-1) * miss
        now = old + torch.einsum("bhk,bhv->bhkv", ki, u)
        do = scale * s["dout"][ids, t].double()
        G = later + torch.einsum("bhk,bhv->bhkv", qi, do)
        du = torch.einsum("bhkv,bhk->bhv", G, ki)
        dmiss = b.unsqueeze(-1) * du
        dki = torch.einsum("bhkv,bhv->bhk", G, u) - torch.einsum("bhkv,bhv->bhk", old, dmiss)
        dold = G - torch.einsum("bhk,bhv->bhkv", ki, dmiss)
        dqi = torch.einsum("bhkv,bhv->bhk", now, do)
        put = lambda to, x: to.index_put_((ids, t), torch.where(there.view(B, *[1] * (x.dim() - 1)), x,  # noqa: E731
                                                                torch.zeros_like(x)))
        put(dq, dqi.unflatten(1, (Hk, -1)).sum(2))
        put(dk_, dki.unflatten(1, (Hk, -1)).sum(2))
        put(dvv, dmiss)
        put(db, (du * miss).sum(-1))
        put(dg, (dold * old).sum((-1, -2)))
        later = torch.where(ok, a[..., None, None] * dold, later)
    res.update(dq=dq, dk=dk_, dv=dvv, dg=dg, dbeta=db)
    if s["h0"] is not None:
        res["dh0"] = later
    return res


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_qknorm if case["op"] == "qknorm" else _exact_delta)(s, case)
