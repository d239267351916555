"""The delta rule's operators in 64 bits, token by token from their formulas,
with a bound beside each result of what the kernels' roundings may do to it
(test infrastructure only).

Bounds of the gated delta rule.  Keys are no longer than sqrt(2 / beta), so a
step I - beta k k^T makes no error of the state larger, and a column n of the
state is a recurrence of its own.  With |.| the length of a vector:

* p is what a computed factor loses as it is held in planes (bfloat16 inputs:
  two planes, 2^-18; float32: three, 2^-26) and a product of two such factors
  loses 4 p at most; fp32 sums on the tensor cores, up to 50 products of
  sixteen one after the other at 2^-22 each, and everything in plain fp32 lose
  2^-16.  e = 4 p + 2^-16.
* A token's corrected value R_i = v_i - e^G S^T k_i - sum ... is off by what
  enters at i, four products of this kind,
    inj_i = 4 e (|v_i| + |k_i| (s + U)),  s the largest |S| and U the sum of
    |k_j| |u_j| over the 32 tokens before i,
  and by |k_i| times the error before it; the state's error is
    err_i = alpha_i err_(i-1) + |k_i| inj_i.
* out is off by scale |q_i| (err_i + 4 e (s + U)), in bfloat16 by three more
  roundings of 2^-9 (the state, T's product and P as its factors).
* dR and dS the same with the gradients' own injections, from behind.
* The other gradients are products of dO, dR, R, S and dS' as they are kept: up
  to four roundings of r = 2^-9 (bfloat16) or e (float32) of every term, 4 r
  times the formula of absolute values, beside what err makes of it.
"""
import numpy as np

C = 64


def qknorm(x, w, kind, eps, freqs=None, positions=None, interleaved=False, dy=None):
    """x [B, L, H, d] and positions [B, L]: y and, with dy, dx and dw."""
    d = x.shape[-1]
    n = 1 if kind == "l2" else d
    w = np.ones(d) if w is None else w
    r = 1 / np.sqrt((x * x).sum(-1, keepdims=True) / n + eps)

    def turn(y, sign):
        if freqs is None:
            return y
        m = len(freqs)
        a = positions[:, :, None, None] * freqs
        c, s = np.cos(a), sign * np.sin(a)
        i, j = (np.arange(m) * 2, np.arange(m) * 2 + 1) if interleaved else (np.arange(m), np.arange(m) + m)
        y = y.copy()
        y[..., i], y[..., j] = y[..., i] * c - y[..., j] * s, y[..., i] * s + y[..., j] * c
        return y

    out = {"y": turn(x * r * w, 1), "r": r}
    if dy is not None:
        dz = turn(dy, -1)
        g = dz * w
        out["dx"] = r * g - x * r ** 3 * (g * x).sum(-1, keepdims=True) / n
        out["dw"] = (dz * x * r).sum((0, 1, 2))
    return out


def walk(n, reverse):
    return list(range(n - 1, -1, -1)) if reverse else list(range(n))


def step(S, q, k, v, g, beta, scale):
    """One token of one head: (out, S)."""
    S = np.exp(g) * S
    S = S + np.outer(k, beta * (v - S.T @ k))
    return scale * (S.T @ q), S


def delta(q, k, v, g, beta, scale, h0=None, lengths=None, reverse=False, dout=None, bf16=False):
    """All outputs and, with dout, all gradients; the bound of each under its name with "~" before it."""
    B, L, Hk, dk = q.shape
    Hv, dv = v.shape[2:]
    n = [L] * B if lengths is None else lengths
    o = {"out": np.zeros(v.shape), "h": np.zeros((B, Hv, dk, dv))}
    if dout is not None:
        o.update(dq=np.zeros(q.shape), dk=np.zeros(k.shape), dv=np.zeros(v.shape), dg=np.zeros(g.shape),
                 dbeta=np.zeros(g.shape), dh0=np.zeros((B, Hv, dk, dv)))
    o.update({"~" + x: np.zeros(y.shape) for x, y in list(o.items())})
    for b in range(B):
        t = walk(n[b], reverse)
        for h in range(Hv):
            hk = h // (Hv // Hk)
            r = _head(q[b, t, hk], k[b, t, hk], v[b, t, h], g[b, t, h], beta[b, t, h], scale,
                      np.zeros((dk, dv)) if h0 is None else h0[b, h], None if dout is None else dout[b, t, h], bf16)
            for x, y in r.items():
                if x.strip("~") in ("h", "dh0"):
                    o[x][b, h] = y
                elif x.strip("~") in ("dq", "dk"):
                    o[x][b, t, hk] += y
                else:
                    o[x][b, t, h] = y
    return o


def _head(q, k, v, g, beta, scale, S, do, bf16):
    L, dv = v.shape
    e = 4 * (2.0 ** -18 if bf16 else 2.0 ** -26) + 2.0 ** -16
    al = np.exp(g)
    kn, qn = np.linalg.norm(k, axis=1), np.linalg.norm(q, axis=1)
    assert (beta * kn * kn <= 2).all()
    states, err, R, eR = [S], [np.zeros(dv)], np.zeros((L, dv)), np.zeros((L, dv))
    out, eout = np.zeros((L, dv)), np.zeros((L, dv))
    ku = np.zeros((L, dv))
    for i in range(L):
        R[i] = v[i] - (al[i] * S).T @ k[i]
        S = al[i] * S + np.outer(k[i], beta[i] * R[i])
        states.append(S)
        out[i] = scale * (S.T @ q[i])
        ku[i] = kn[i] * np.abs(beta[i] * R[i])
        size = np.max([np.linalg.norm(x, axis=0) for x in states[max(0, i - 32):]], axis=0)
        size = size + ku[max(0, i - 32):i + 1].sum(0)
        inj = 4 * e * (np.abs(v[i]) + kn[i] * size)
        eR[i] = inj + kn[i] * err[-1]
        err.append(al[i] * err[-1] + kn[i] * inj)
        eout[i] = scale * qn[i] * (err[-1] + (4 * e + (3 * 2.0 ** -9 if bf16 else 0)) * size)
    o = {"out": out, "~out": eout, "h": S, "~h": np.broadcast_to(err[-1], S.shape)}
    if do is None:
        return o
    # back: lam[i] is the state's gradient after token i - 1
    lam, elam = [None] * (L + 1), [None] * (L + 1)
    lam[L], elam[L] = np.zeros_like(S), np.zeros(dv)
    dR, edR = np.zeros((L, dv)), np.zeros((L, dv))
    dq, dk, dg, db = np.zeros(q.shape), np.zeros(k.shape), np.zeros(L), np.zeros(L)
    qd, kd = np.zeros((L, dv)), np.zeros((L, dv))
    for i in range(L - 1, -1, -1):
        G = lam[i + 1] + scale * np.outer(q[i], do[i])
        old = al[i] * states[i]
        du = G.T @ k[i]
        dR[i] = beta[i] * du
        db[i] = du @ R[i]
        dq[i] = scale * (states[i + 1] @ do[i])
        dk[i] = G @ (beta[i] * R[i]) - old @ dR[i]
        dS = G - np.outer(k[i], dR[i])
        dg[i] = (old * dS).sum()
        lam[i] = al[i] * dS
        qd[i], kd[i] = scale * qn[i] * np.abs(do[i]), kn[i] * np.abs(dR[i])
        size = np.max([np.linalg.norm(x, axis=0) for x in lam[i + 1:i + 34]], axis=0)
        size = size + qd[i:i + 33].sum(0) + kd[i:i + 33].sum(0)
        inj = 4 * e * kn[i] * size
        edR[i] = inj + kn[i] * elam[i + 1]
        elam[i] = al[i] * (elam[i + 1] + kn[i] * inj + 4 * e * qd[i])
    o.update(dq=dq, dk=dk, dv=dR, dg=dg, dbeta=db, dh0=lam[0])
    o["~dv"], o["~dh0"] = edR, np.broadcast_to(elam[0], S.shape)
    r = 4 * (2.0 ** -9 if bf16 else 0.0) + 4 * e
    o.update({"~" + x: np.zeros(o[x].shape) for x in ("dq", "dk", "dg", "dbeta")})
    a = np.abs
    for c0 in range(0, L, C):
        s = slice(c0, min(L, c0 + C))
        Gs = np.cumsum(g[s])
        D = np.tril(np.exp(np.minimum(0, Gs[:, None] - Gs[None])))
        grown, left = np.exp(Gs)[:, None], np.exp(Gs[-1] - Gs)[:, None]
        S0, dS1 = a(states[c0]), a(lam[s.stop])
        low = np.tril(D, -1)
        ones = np.ones(S0.shape)

        def terms(dO, dr, Rr, S0, dS1):
            """The formulas of absolute values, with what is given in their factors' places."""
            A, E = scale * D * (dO @ Rr.T), low * (dr @ Rr.T)
            dq1, f1, w1 = scale * grown * (dO @ S0.T), grown * (dr @ S0.T), left * (Rr @ dS1.T)
            K, Q, be = a(k[s]), a(q[s]), beta[s]
            W = w1 + A.T @ Q + E.T @ K
            pair = be[None] * (np.tril(A, -1) * (Q @ K.T) + E * (K @ K.T))
            inner = (Q * dq1).sum(1) + (K * f1).sum(1)
            before = be * (K * w1).sum(1)
            m = len(be)
            dgm = np.array([inner[i:].sum() + before[:i].sum() + pair[i:, :i].sum() for i in range(m)])
            dgm += grown[-1, 0] * (S0 * dS1).sum()
            return (dq1 + (A * be[None]) @ K, be[:, None] * W + f1 + (E * be[None]) @ K, dgm, (K * W).sum(1)), pair.sum()

        full = (a(do[s]), a(dR[s]), a(R[s]), S0, dS1)
        sizes, pairs = terms(*full)
        wrong = (0 * full[0], edR[s], eR[s], err[c0] * ones, elam[s.stop] * ones)
        for x, size in zip(("~dq", "~dk", "~dg", "~dbeta"), sizes):
            o[x][s] += r * size
        for i in range(1, 5):   # one factor's error at a time
            for x, size in zip(("~dq", "~dk", "~dg", "~dbeta"), terms(*full[:i], wrong[i], *full[i + 1:])[0]):
                o[x][s] += size
        o["~dg"][s] += 64 * 2.0 ** -23 * pairs   # sums of rows less sums of columns
    return o
