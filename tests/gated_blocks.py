"""Gated lightning attention and its gradients in 64 bits, a block of tokens at a time, on any
device: a reference for sequences that are too long for ``oracle.gated``'s token-by-token one
(against which it is tested itself).  Errors are measured per sequence and head.
"""
import torch

STEP = 32


def _double(t):
    return None if t is None else t.double()


def gradients(x, cu):
    """``x``: q, k, v, g (may be None), do, and where there are any initial, d_state.  Returns a
    dict of o, state, dq, dk, dv, dg, d_initial in 64 bits, and `size` [T, H]: about the root sum of
    squares of the products that dg's state terms add up, |S| |dS| / D."""
    q, k, v, g, do = (_double(x.get(n)) for n in ("q", "k", "v", "g", "do"))
    initial, d_state = _double(x.get("initial")), _double(x.get("d_state"))
    T, H, D = q.shape
    g = q.new_zeros(T, H) if g is None else g.clamp(min=-800.0)   # e^-800 is 0 in 64 bits
    out = {n: torch.zeros_like(q) for n in ("o", "dq", "dk", "dv")}
    out["dg"], out["size"] = torch.zeros_like(g), torch.zeros_like(g)
    S = len(cu) - 1
    out["state"], out["d_initial"] = q.new_zeros(S, H, D, D), q.new_zeros(S, H, D, D)
    for s, (lo, hi) in enumerate(zip(cu, cu[1:])):
        X = q.new_zeros(H, D, D) if initial is None else initial[s]
        cuts = [(a, min(a + STEP, hi)) for a in range(lo, hi, STEP)]
        starts = []
        for a, b in cuts:
            starts.append(X)
            Q, K, V = (t[a:b].transpose(0, 1) for t in (q, k, v))
            G = g[a:b].T.cumsum(1)
            w = (G[:, :, None] - G[:, None, :]).tril().exp().tril()
            out["o"][a:b] = (((Q @ K.mT) * w) @ V + (Q @ X) * G.exp()[..., None]).transpose(0, 1)
            X = X * G[:, -1].exp()[:, None, None] + (K * w[:, -1, :, None]).mT @ V
        out["state"][s] = X
        starts.append(X)
        if do is None:
            continue
        Y = q.new_zeros(H, D, D) if d_state is None else d_state[s]
        for n in range(len(cuts) - 1, -1, -1):
            (a, b), X = cuts[n], starts[n]
            Q, K, V, O = (t[a:b].transpose(0, 1) for t in (q, k, v, do))
            G = g[a:b].T.cumsum(1)
            w = (G[:, :, None] - G[:, None, :]).tril().exp().tril()
            up, down = G.exp()[..., None], w[:, -1, :, None]   # e^{G_i}, e^{G_C - G_j}
            P, dP = (Q @ K.mT) * w, (O @ V.mT) * w
            dq, dk = (O @ X.mT) * up, (V @ Y.mT) * down
            out["dq"][a:b] = (dP @ K + dq).transpose(0, 1)
            out["dk"][a:b] = (dP.mT @ Q + dk).transpose(0, 1)
            out["dv"][a:b] = (P.mT @ O + (K @ Y) * down).transpose(0, 1)
            W = ((Q @ K.mT) * dP).tril(-1)
            ends, begins = (Q * dq).sum(-1), (K * dk).sum(-1) + W.sum(1) - W.sum(2)
            dg = ends.flip(1).cumsum(1).flip(1) + (begins.cumsum(1) - begins)
            dg = dg + (up[:, -1] * (X * Y).sum((1, 2))[:, None])
            before = Y
            Y = Y * up[:, -1, :, None] + (Q * up).mT @ O
            out["dg"][a:b] = dg.T
            big = torch.maximum(X.norm(dim=(1, 2)), starts[n + 1].norm(dim=(1, 2)))
            out["size"][a:b] = (big * torch.maximum(Y.norm(dim=(1, 2)), before.norm(dim=(1, 2))) / D)[None]
        out["d_initial"][s] = Y
    return out


def norms(t, cu):
    """2-norms [S, H] over each sequence's tokens (of [T, H, ...]) or states (of [S, H, ...])."""
    t = t.double()
    if cu is None:
        return t.flatten(2).norm(dim=2)
    H = t.shape[1]
    return torch.stack([t[a:b].transpose(0, 1).reshape(H, -1).norm(dim=1) for a, b in zip(cu, cu[1:])])


def worst(got, ref, cu):
    """Largest relative 2-norm error of any sequence and head."""
    assert got.shape == ref.shape and bool(torch.isfinite(got).all())
    off, norm = norms(got.double() - ref, cu), norms(ref, cu)
    return float(torch.where(off == 0, off, off / norm).max()) if off.numel() else 0.0
