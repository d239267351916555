"""The gated delta rule token by token in 64 bits, all heads at once, from its
formulas (test infrastructure only): for sequences of thousands of tokens,
which ``delta_reference.py``, one head after the other, takes minutes for."""
import torch


def recurrence(q, k, v, g, beta, scale, h0=None, lengths=None, reverse=False, dout=None):
    """``out``, ``h`` and, with dout, every gradient, on the inputs' device; and what they are made of, token by token in
    the order of the walk: ``walk`` = (states before each token and after the last, R, dR, the states' gradients)."""
    B, L, Hk, dk = q.shape
    Hv, dv = v.shape[2:]
    group, dev = Hv // Hk, q.device
    n = torch.as_tensor([L] * B if lengths is None else lengths, device=dev)[:, None]
    t = torch.arange(L, device=dev)
    there = t < n
    at = torch.where(there & reverse, n - 1 - t, t)   # the token that is walked t-th
    row = torch.arange(B, device=dev)[:, None]

    def walk(x, group=1):
        x = x[row, at].double()
        x = torch.where(there.view(B, L, *[1] * (x.dim() - 2)), x, 0.0)   # past the end: beta = 0 and a decay of 1
        return x.repeat_interleave(group, 2).transpose(0, 1)

    def back(x, group=1):
        x = x.transpose(0, 1)
        if group > 1:
            x = x.unflatten(2, (Hk, group)).sum(3)
        y = torch.zeros_like(x)
        y[row.expand(B, L)[there], at[there]] = x[there]
        return y

    Q, K, V, A, b = walk(q, group), walk(k, group), walk(v), walk(g).exp()[..., None, None], walk(beta)[..., None]
    S = torch.zeros(B, Hv, dk, dv, dtype=torch.float64, device=dev) if h0 is None else h0.double()
    states, R, out = [S], torch.zeros_like(V), torch.zeros_like(V)
    for i in range(L):
        S = A[i] * S
        R[i] = V[i] - (S * K[i][..., None]).sum(-2)
        S = S + K[i][..., None] * (b[i] * R[i])[..., None, :]
        out[i] = scale * (S * Q[i][..., None]).sum(-2)
        states.append(S if dout is not None else None)
    o = {"out": back(out), "h": S}
    if dout is None:
        return o
    DO = walk(dout)
    D = torch.zeros_like(S)
    dstates = [D]
    dq, dk_, dR, dg, db = (torch.zeros_like(x) for x in (Q, K, V, b[..., 0], b[..., 0]))
    for i in range(L - 1, -1, -1):
        G, old = D + scale * Q[i][..., None] * DO[i][..., None, :], A[i] * states[i]
        du = (G * K[i][..., None]).sum(-2)
        dR[i], db[i] = b[i] * du, (du * R[i]).sum(-1)
        dq[i] = scale * (states[i + 1] * DO[i][..., None, :]).sum(-1)
        dk_[i] = (G * (b[i] * R[i])[..., None, :]).sum(-1) - (old * dR[i][..., None, :]).sum(-1)
        dS = G - K[i][..., None] * dR[i][..., None, :]
        dg[i] = (old * dS).sum((-1, -2))
        D = A[i] * dS
        dstates.append(D)
    o["walk"] = states, R, dR, dstates[::-1]
    o.update(dq=back(dq, group), dk=back(dk_, group), dv=back(dR), dg=back(dg), dbeta=back(db), dh0=D)
    return o
