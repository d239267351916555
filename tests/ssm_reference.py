"""The state space block's operators in 64 bits, token by token from their
formulas, with a magnitude beside each result: the same formulas with every
term's absolute value, to which a rounding error is relative (test
infrastructure only)."""
import numpy as np


def _sig(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def _dsilu(x):
    s = _sig(x)
    return s * (1 + x * (1 - s))


def order(L, n, reverse):
    """The tokens of a sequence of n in the order they are walked."""
    return list(range(n - 1, -1, -1)) if reverse else list(range(n))


def layernorm(x, w, b, eps, dy=None):
    C = x.shape[-1]
    mean = x.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    xh = (x - mean) * rstd
    out = {"y": xh * w + (0 if b is None else b)}
    if dy is not None:
        g = dy * w
        out["dx"] = rstd * (g - g.mean(-1, keepdims=True) - xh * (g * xh).sum(-1, keepdims=True) / C)
        out["dweight"], out["dbias"] = (dy * xh).sum(0), dy.sum(0)
    return out


def conv(x, w, b, act, state=None, lengths=None, reverse=False, dy=None, absolute=False):
    m = np.abs if absolute else (lambda v: v)
    B, L, D = x.shape
    K = w.shape[1]
    n = [L] * B if lengths is None else lengths
    bias = np.zeros(D) if b is None else b
    y, fin, dx = np.zeros((B, L, D)), np.zeros((B, K - 1, D)), np.zeros((B, L, D))
    dst, dw, db = np.zeros((B, K - 1, D)), np.zeros((D, K)), np.zeros(D)
    for q in range(B):
        walk = order(L, n[q], reverse)
        line = np.concatenate([np.zeros((K - 1, D)) if state is None else state[q], x[q][walk]])
        dline = np.zeros_like(line)
        for i, t in enumerate(walk):
            win = line[i:i + K]
            p = bias + (w.T * win).sum(0)
            mp = m(bias) + (m(w).T * m(win)).sum(0)
            y[q, t] = (mp if absolute else p * _sig(p)) if act else (mp if absolute else p)
            if dy is not None:
                # |act'| <= 1.1 and |act''| <= 0.5, which the error of p goes through
                d = dy[q, t] * (_dsilu(p) if act else 1.0)
                d = np.abs(dy[q, t]) * (1.1 + 0.5 * mp if act else 1.0) if absolute else d
                dline[i:i + K] += m(w).T * d
                dw += (m(win) * d).T
                db += d
        fin[q] = line[len(walk):]
        dst[q] = dline[:K - 1]
        dx[q][walk] = dline[K - 1:]
    return {"y": y, "state": fin, "dx": dx, "dweight": dw, "dbias": db, "dstate": dst}


def scan(u, dt, A, Bm, Cm, Dskip=None, z=None, dt_bias=None, dt_softplus=True, h0=None, lengths=None, reverse=False,
         dout=None, absolute=False):
    """Bm, Cm [B, L, G, N].  All outputs and, with dout, all gradients."""
    m = np.abs if absolute else (lambda v: v)
    B, L, D = u.shape
    N, G = A.shape[1], Bm.shape[2]
    of = np.arange(D) // (D // G)
    n = [L] * B if lengths is None else lengths
    raw = dt + (0 if dt_bias is None else dt_bias)
    delta = np.logaddexp(0, raw) if dt_softplus else raw
    skip = np.zeros(D) if Dskip is None else Dskip
    gate = np.ones_like(u) if z is None else z * _sig(z)
    out, hT = np.zeros((B, L, D)), np.zeros((B, D, N))
    r = {k: np.zeros((B, L, D)) for k in ("du", "ddt", "dz")}
    r.update(dB=np.zeros(Bm.shape), dC=np.zeros(Bm.shape), dA=np.zeros((D, N)), dDskip=np.zeros(D),
             ddt_bias=np.zeros(D), dh0=np.zeros((B, D, N)))
    u, Bm, Cm, skip = m(u), m(Bm), m(Cm), m(skip)
    md, mA = m(delta), m(A)
    for q in range(B):
        walk = order(L, n[q], reverse)
        h = np.zeros((D, N)) if h0 is None else m(h0[q]).copy()
        hs, ys = [h], []
        for t in walk:
            a = np.exp(delta[q, t][:, None] * A)
            h = a * h + (md[q, t] * u[q, t])[:, None] * Bm[q, t][of]
            hs.append(h)
            y = (Cm[q, t][of] * h).sum(1) + skip * u[q, t]
            ys.append(y)
            out[q, t] = y * m(gate[q, t])
        hT[q] = h
        if dout is None:
            continue
        g = np.zeros((D, N))
        for i in range(len(walk) - 1, -1, -1):
            t = walk[i]
            dy = m(dout[q, t] * gate[q, t])
            a = np.exp(delta[q, t][:, None] * A)
            Gt = Cm[q, t][of] * dy[:, None] + g
            g = a * Gt
            e = g * hs[i]
            gb = (Gt * Bm[q, t][of]).sum(1)
            dd = (e * mA).sum(1) + u[q, t] * gb
            dd = dd * (_sig(raw[q, t]) if dt_softplus else 1.0)
            r["ddt"][q, t] = dd
            r["ddt_bias"] += dd
            r["du"][q, t] = skip * dy + md[q, t] * gb
            r["dA"] += e * md[q, t][:, None]
            np.add.at(r["dB"][q, t], of, Gt * (md[q, t] * u[q, t])[:, None])
            np.add.at(r["dC"][q, t], of, hs[i + 1] * dy[:, None])
            r["dDskip"] += dy * u[q, t]
            if z is not None:
                r["dz"][q, t] = m(dout[q, t]) * ys[i] * (m(_dsilu(z[q, t])) + (0.5 if absolute else 0.0))
        r["dh0"][q] = g
    r.update(out=out, h=hT)
    return r
