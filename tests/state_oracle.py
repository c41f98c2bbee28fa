"""Linear attention with a decay per head, from its definition: token by token in 64 bits, with the bounds that a result in
fewer bits is held to."""
import torch

U = 2.0 ** -24  # half a step of fp32, relative


def walk(q, k, v, g, S0, parents, scale):
    """One request: q, k [n, Hk, Dk], v [n, H, Dv], g [n, H], S0 [H, Dk, Dv] (64 bits), row i behind row parents[i] (-1: S0)
    -> out [n, H, Dv], every row's state, and for both the sum of the terms' magnitudes (as they are, and with decays of half
    the exponent: a factor e^G off by |G| parts is off by at most 0.74 e^{G/2})."""
    n, H, Dv = v.shape
    G = H // k.shape[1]
    q, k = (x.double().repeat_interleave(G, 1) for x in (q, k))
    v, g, S0 = v.double(), g.double(), S0.double()
    states, out = [], []
    start = (S0, S0.abs(), S0.abs())
    for i in range(n):
        S, T, T2 = start if parents[i] < 0 else states[parents[i]]
        kv = k[i][:, :, None] * v[i][:, None, :]
        f, h = torch.exp(g[i])[:, None, None], torch.exp(g[i] / 2)[:, None, None]
        states.append((S * f + kv, T * f + kv.abs(), T2 * h + kv.abs()))
        S, T, T2 = states[-1]
        qi = q[i][:, :, None]
        out.append(tuple(scale * (a * b).sum(1) for a, b in ((qi, S), (qi.abs(), T), (qi.abs(), T2))))
    last = states[-1] if n else start
    outs = [torch.stack(x) for x in zip(*out)] if n else [torch.zeros(0, H, Dv, dtype=torch.float64)] * 3
    return outs, last


def chain(n):
    return [i - 1 for i in range(n)]


def bound(terms, halved, Dk, n, pieces=0.0):
    """What fp32 sums of Dk and n terms with factors e^G may be off, by the terms' magnitudes: a rounding for each addition of a
    sum, some forty for what else a term passes through, the decays' own; pieces: what an operand of fewer bits leaves out."""
    return ((Dk + 2 * n + 40) * U + pieces) * terms + 4 * U * halved


def check_out(got, want, Dk, n, dtype, pieces=0.0):
    """Within the bound and one rounding to dtype (half a step of the value, or of fp16's subnormals)."""
    w, terms, halved = want
    half = torch.finfo(dtype).eps / 2
    tol = bound(terms, halved, Dk, n, pieces)
    tol = tol + half * (w.abs() + tol) + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -133)
    worst = ((got.double().cpu() - w).abs() / tol)
    assert bool((worst <= 1).all()), float(worst.max()) if worst.numel() else 0.0


def check_state(got, want, Dk, n, pieces=0.0):
    w, terms, halved = want
    tol = bound(terms, halved, 0, n, pieces) + 2.0 ** -126
    worst = (got.double().cpu() - w).abs() / tol
    assert bool((worst <= 1).all()), float(worst.max())
