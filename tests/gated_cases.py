"""Inputs and error measures that the tests of the gated operators share."""
import numpy as np
import torch

# Half a rounding step relative to the value.
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def gates(kind, T, H, dtype, seed, device):
    """Log-decays [T, H]: `mild` keeps hundreds of tokens, `steep` a few, `reset` has -inf
    in every ninth place, `mixed` is one head of each, `grow` is above 0 now and then."""
    if kind == "none":
        return None
    gen = torch.Generator().manual_seed(seed)
    x = torch.rand(T, H, generator=gen)
    if kind == "zero":
        g = torch.zeros(T, H)
    elif kind == "mild":
        g = -0.01 * x
    elif kind == "steep":
        g = -6.0 * x
    elif kind == "reset":
        g = -0.2 * x
        g[(torch.arange(T) * 7 + 3) % 9 == 0] = float("-inf")
    elif kind == "grow":
        g = 0.3 * (x - 0.6)
    else:
        g = -x * torch.tensor([0.003, 0.1, 1.0, 20.0])[torch.arange(H) % 4]
    return g.to(dtype).to(device)


def inputs(cu, H, D, dtype, seed, device, kind="mixed", grad=False, states=False):
    gen = torch.Generator().manual_seed(1000 + seed)
    T, S = cu[-1], len(cu) - 1

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen) * scale

    x = {n: normal(T, H, D, scale=D ** -0.5).to(dtype).to(device) for n in "qkv"}
    x["g"] = gates(kind, T, H, dtype, seed, device)
    if grad:
        x["do"] = normal(T, H, D).to(dtype).to(device)
    if states:
        x["initial"] = normal(S, H, D, D, scale=8.0 / D).to(device)
        if grad:
            x["d_state"] = normal(S, H, D, D, scale=1.0 / D).to(device)
    return x


def rel(got, ref):
    """Largest relative 2-norm error over the heads of all sequences together."""
    got = got.detach().double().cpu().numpy() if hasattr(got, "detach") else np.asarray(got, np.float64)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert np.isfinite(got).all()
    if got.size == 0:
        return 0.0
    axes = (0,) + tuple(range(2, got.ndim))          # everything but the head axis
    off = np.sqrt(((got - ref) ** 2).sum(axis=axes))
    norm = np.sqrt((ref ** 2).sum(axis=axes))
    return float(np.max(np.where(off == 0, 0, off / np.maximum(norm, 1e-300))))
