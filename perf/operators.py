"""Gated lightning attention: the operators' plain forms, their cases and their work.

Three operators on a D x D fp32 state per sequence and head, with a log-decay g per token
and head (natural logarithm, the dtype of q):

    prefill   S_t = exp(g_t) S_{t-1} + k_t v_t^T,  o_t = S_t^T q_t over packed sequences
    backward  dq, dk, dv, dg (and the initial state's gradient) from do (and the final
              state's gradient)
    decode    one token for each sequence, the state updated in place in a pool of slots

``run`` takes the plain form in elementary torch operations, or with ``own`` the
framework's calls.
"""
import math

import torch

own = False


def listed():
    return [
        # a first short prompt in full precision: latency
        dict(name="prefill fp32 256x2x64", op="prefill", dtype="fp32", T=256, H=2, D=64, S=1, state=False),
        # one user's short prompt on all heads: latency
        dict(name="prefill bf16 130x64x128", op="prefill", dtype="bf16", T=130, H=64, D=128, S=1, state=False),
        # one layer over a training-length sequence
        dict(name="prefill bf16 8192x64x128", op="prefill", dtype="bf16", T=8192, H=64, D=128, S=1, state=False),
        # chunked prefill of eight ragged requests, each from its state
        dict(name="prefill bf16 packed states", op="prefill", dtype="bf16", T=32768, H=64, D=128, S=8, state=True),
        # a long document on the heads that one of several GPUs holds
        dict(name="prefill bf16 long 8 heads", op="prefill", dtype="bf16", T=131072, H=8, D=128, S=1, state=True),
        # a long document on all heads
        dict(name="prefill bf16 131072x64x128", op="prefill", dtype="bf16", T=131072, H=64, D=128, S=1, state=False),
        # narrow heads, short ragged sequences packed into one training row
        dict(name="backward bf16 packed D=64", op="backward", dtype="bf16", T=4096, H=16, D=64, S=5, state=False),
        # gradients in full precision (checks of a training run)
        dict(name="backward fp32 1000x4x64", op="backward", dtype="fp32", T=1000, H=4, D=64, S=1, state=False),
        # one layer's training step
        dict(name="backward bf16 8192x64x128", op="backward", dtype="bf16", T=8192, H=64, D=128, S=1, state=False),
        # truncated backpropagation: ragged pieces between carried states
        dict(name="backward bf16 packed states", op="backward", dtype="bf16", T=16384, H=32, D=128, S=8, state=True),
        # one user's next token
        dict(name="decode bf16 1x64x128", op="decode", dtype="bf16", B=1, H=64, D=128, slots=4),
        # a full serving batch out of a larger pool of states
        dict(name="decode bf16 256x64x128", op="decode", dtype="bf16", B=256, H=64, D=128, slots=320),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["prefill", "prefill", "backward", "backward", "decode"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    D, H = rng.choice([64, 128]), spread(1, 64)
    if op == "decode":
        B = spread(1, 256)
        return dict(op=op, dtype=dtype, B=B, H=H, D=D, slots=B + rng.randrange(0, 65))
    most = {("prefill", "bf16"): 1 << 22, ("backward", "bf16"): 1 << 20}.get((op, dtype), 1 << 18)
    T = spread(1, min(131072, most // H))
    return dict(op=op, dtype=dtype, T=T, H=H, D=D, S=rng.randrange(1, min(T, 12) + 1),
                state=rng.random() < 0.5)


def _dtype(case):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[case["dtype"]]


def _gate(x, H):
    """Log-decays of heads whose memory reaches from about one token to some hundreds."""
    slope = torch.exp2(-8.0 * (torch.arange(H, device=x.device) + 1) / H)
    return -torch.nn.functional.softplus(x) * slope


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt, H, D = _dtype(case), case["H"], case["D"]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * scale

    n = case["B"] if case["op"] == "decode" else case["T"]
    state = dict(case=dict(case))
    for name in ("q", "k", "v"):
        state[name] = normal(n, H, D, scale=D ** -0.5).to(dt)
    state["g"] = _gate(normal(n, H), H).to(dt)
    if case["op"] == "decode":
        state["state"] = normal(case["slots"], H, D, D, scale=64 ** 0.5 / D)
        state["slots"] = torch.randperm(case["slots"], generator=gen, device="cuda")[:n].to(torch.int32)
        return state
    S = case["S"]
    cuts = torch.randint(0, n + 1, (S - 1,), generator=gen, device="cuda").sort().values.tolist()
    state["cu"] = [0] + cuts + [n]
    if case["state"]:
        state["initial"] = normal(S, H, D, D, scale=64 ** 0.5 / D)
    if case["op"] == "backward":
        state["do"] = normal(n, H, D).to(dt)
        if case["state"]:
            state["d_state"] = normal(S, H, D, D, scale=1 / D)
    return state


def work(case):
    e, H, D = (2 if case["dtype"] == "bf16" else 4), case["H"], case["D"]
    if case["op"] == "decode":
        rows = case["B"] * H
        return dict(bytes=rows * (8 * D * D + (4 * D + 1) * e), flops=rows * 4 * D * D)
    rows, states = case["T"] * H, 4 * D * D * case["S"] * H
    if case["op"] == "prefill":
        return dict(bytes=rows * (4 * D + 1) * e + states * (2 if case["state"] else 0),
                    flops=rows * 4 * D * D)
    return dict(bytes=rows * (7 * D + 2) * e + states * (3 if case["state"] else 0),
                flops=rows * 10 * D * D)


# ------------------------------------------------------------------------ plain forms
CHUNK = 128


def _rows(cu, device):
    """Where each token of a packed batch stands in a padded one: (sequence, position), and
    the padded length, a multiple of CHUNK."""
    bounds = torch.tensor(cu, device=device)
    lengths = bounds[1:] - bounds[:-1]
    seq = torch.repeat_interleave(torch.arange(len(cu) - 1, device=device), lengths,
                                  output_size=cu[-1])
    pos = torch.arange(cu[-1], device=device) - bounds[seq]
    longest = max(b - a for a, b in zip(cu, cu[1:]))
    return seq, pos, max(1, -(-longest // CHUNK)) * CHUNK


def _padded(x, seq, pos, S, N):
    """[T, H, ...] packed -> [S, H, N, ...] in 32 bits, zeros behind each sequence."""
    y = x.new_zeros((S, N) + tuple(x.shape[1:]), dtype=torch.float32)
    y[seq, pos] = x.float()
    return y.transpose(1, 2)


def _scan(q, k, v, g, initial):
    """o and the final state of padded sequences [S, H, N, ...]: within chunks by the masked
    product, across chunks by the decays between all pairs of chunks."""
    S, H, N, D = q.shape
    c = N // CHUNK
    q, k, v = (x.reshape(S, H, c, CHUNK, D) for x in (q, k, v))
    G = g.double().reshape(S, H, c, CHUNK).cumsum(-1)
    total = G[..., -1]
    decay = (G[..., :, None] - G[..., None, :]).float().exp_().tril_()
    o = ((q @ k.transpose(-1, -2)) * decay) @ v
    del decay
    inside = (k * (total[..., None] - G).float().exp()[..., None]).transpose(-1, -2) @ v
    every = torch.cat([initial.reshape(S, H, 1, D * D), inside.reshape(S, H, c, D * D)], 2)
    del inside
    # entry m of `every` is worth exp(sum of totals m .. n-1) at the start of chunk n
    upto = torch.cat([torch.zeros_like(total[..., :1]), total.cumsum(-1)], -1)
    between = (upto[..., :, None] - upto[..., None, :]).float()
    states = torch.exp(between).tril_() @ every
    del every
    states = states.reshape(S, H, c + 1, D, D)
    o += (q @ states[:, :, :c]) * G.float().exp()[..., None]
    return o.reshape(S, H, N, D), states[:, :, c].clone()


def _plain_prefill(q, k, v, g, cu, initial):
    S, (H, D) = len(cu) - 1, q.shape[1:]
    seq, pos, N = _rows(cu, q.device)
    if initial is None:
        initial = torch.zeros(S, H, D, D, device=q.device)
    o, last = _scan(*(_padded(x, seq, pos, S, N) for x in (q, k, v, g)), initial)
    return o.transpose(1, 2)[seq, pos].to(q.dtype), last


def _plain_backward(q, k, v, g, do, cu, initial, d_state):
    S, (H, D) = len(cu) - 1, q.shape[1:]
    seq, pos, N = _rows(cu, q.device)
    zero = torch.zeros(S, H, D, D, device=q.device)
    x0 = zero if initial is None else initial
    d1 = zero if d_state is None else d_state
    pq, pk, pv, pg, pdo = (_padded(x, seq, pos, S, N) for x in (q, k, v, g, do))
    # dq runs forward in time: the scan of (do, v, k); dk and dv run backward
    dq, last = _scan(pdo, pv, pk, pg, x0.transpose(-1, -2))
    later = torch.cat([pg[..., 1:], torch.zeros_like(pg[..., :1])], -1).flip(-1)
    fq, fk, fv, fdo = (x.flip(2) for x in (pq, pk, pv, pdo))
    dk = _scan(fv, fdo, fq, later, d1.transpose(-1, -2))[0].flip(2)
    dv, first = _scan(fk, fq, fdo, later, d1)
    dv = dv.flip(2)
    first = first * pg[..., 0].exp()[..., None, None]
    # dg_t gathers every pair (j < t <= i): what ends at or after t less what starts there
    pairs = (pq.double() * dq.double() - pk.double() * dk.double()).sum(-1)
    dg = pairs.flip(-1).cumsum(-1).flip(-1) + (last.transpose(-1, -2).double() * d1.double()).sum((-1, -2))[..., None]
    out = {n: x.transpose(1, 2)[seq, pos].to(q.dtype) for n, x in dict(dq=dq, dk=dk, dv=dv, dg=dg).items()}
    if initial is not None:
        out["d_initial"] = first
    return out


def _plain_decode(q, k, v, g, state, slots):
    at = slots.long()
    new = state[at] * g.float().exp()[..., None, None] + k.float()[..., :, None] * v.float()[..., None, :]
    state[at] = new
    return (q.float()[..., None, :] @ new).squeeze(-2).to(q.dtype)


def run(state):
    s, case = state, state["case"]
    if case["op"] == "decode":
        args = (s["q"], s["k"], s["v"], s["g"], s["state"])
        if own:
            from long_context_04_b200 import api
            return dict(o=api.gated_decode_step(*args, slots=s["slots"]), state=s["state"])
        return dict(o=_plain_decode(*args, s["slots"]), state=s["state"])
    args = (s["q"], s["k"], s["v"], s["g"])
    if case["op"] == "prefill":
        if own:
            from long_context_04_b200 import api
            if not case["state"]:
                return dict(o=api.gated_prefill(*args, cu_seqlens=s["cu"]))
            o, last = api.gated_prefill(*args, cu_seqlens=s["cu"], initial_state=s["initial"], return_state=True)
            return dict(o=o, state=last)
        o, last = _plain_prefill(*args, s["cu"], s.get("initial"))
        return dict(o=o, state=last) if case["state"] else dict(o=o)
    if own:
        from long_context_04_b200 import api
        got = api.gated_prefill_backward(*args, s["do"], cu_seqlens=s["cu"], initial_state=s.get("initial"),
                                         d_state=s.get("d_state"))
        return dict(zip(("dq", "dk", "dv", "dg", "d_initial"), got))
    return _plain_backward(*args, s["do"], s["cu"], s.get("initial"), s.get("d_state"))


# ------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The recurrence itself in 64 bits, a few tokens at a time, sequence by sequence."""
    s = prepare(case, seed)
    q, k, v, g = (s[n].double() for n in ("q", "k", "v", "g"))
    if case["op"] == "decode":
        at = s["slots"].long()
        state = s["state"].double()
        a = g.exp()
        # o = q^T (a S + k v^T), written without forming the new state first
        o = a[..., None] * torch.einsum("bhi,bhij->bhj", q, state[at]) + (q * k).sum(-1, keepdim=True) * v
        state[at] = torch.einsum("bh,bhij->bhij", a, state[at]) + torch.einsum("bhi,bhj->bhij", k, v)
        return dict(o=o, state=state)
    H, D = case["H"], case["D"]
    step = 48
    back = case["op"] == "backward"
    do = s["do"].double() if back else None
    o = torch.zeros_like(q)
    dq, dk, dv, dg = (torch.zeros_like(x) for x in (q, k, v, g)) if back else (None,) * 4
    lasts, firsts = [], []
    for n, (lo, hi) in enumerate(zip(s["cu"], s["cu"][1:])):
        X = s["initial"][n].double() if case["state"] else q.new_zeros(H, D, D)
        starts, pieces = [], [slice(a, min(a + step, hi)) for a in range(lo, hi, step)]
        for at in pieces:
            starts.append(X if back else None)
            a = g[at].cumsum(0)
            w = torch.exp(a[:, None] - a[None]) * torch.ones(len(a), len(a), device=a.device).double().tril()[..., None]
            if not back:
                o[at] = torch.einsum("ihx,jhx,ijh,jhy->ihy", q[at], k[at], w, v[at]) \
                    + torch.einsum("ihx,hxy,ih->ihy", q[at], X, a.exp())
            X = X * a[-1].exp()[:, None, None] + torch.einsum("jhx,jhy,jh->hxy", k[at], v[at], w[-1])
        lasts.append(X)
        if not back:
            continue
        Y = s["d_state"][n].double() if case["state"] else q.new_zeros(H, D, D)
        through = (Y * X).sum((-1, -2))
        for at, X in zip(pieces[::-1], starts[::-1]):
            a = g[at].cumsum(0)
            w = torch.exp(a[:, None] - a[None]) * torch.ones(len(a), len(a), device=a.device).double().tril()[..., None]
            dp = torch.einsum("ihy,jhy,ijh->ijh", do[at], v[at], w)
            p = torch.einsum("ihx,jhx,ijh->ijh", q[at], k[at], w)
            dq[at] = torch.einsum("ijh,jhx->ihx", dp, k[at]) + torch.einsum("ihy,hxy,ih->ihx", do[at], X, a.exp())
            dk[at] = torch.einsum("ijh,ihx->jhx", dp, q[at]) + torch.einsum("jhy,hxy,jh->jhx", v[at], Y, w[-1])
            dv[at] = torch.einsum("ijh,ihy->jhy", p, do[at]) + torch.einsum("jhx,hxy,jh->jhy", k[at], Y, w[-1])
            Y = Y * a[-1].exp()[:, None, None] + torch.einsum("ihx,ihy,ih->hxy", q[at], do[at], a.exp())
        pairs = (q[lo:hi] * dq[lo:hi] - k[lo:hi] * dk[lo:hi]).sum(-1)
        dg[lo:hi] = through + pairs.flip(0).cumsum(0).flip(0)
        firsts.append(Y)
    if not back:
        return dict(o=o, state=torch.stack(lasts)) if case["state"] else dict(o=o)
    out = dict(dq=dq, dk=dk, dv=dv, dg=dg)
    if case["state"]:
        out["d_initial"] = torch.stack(firsts)
    return out
