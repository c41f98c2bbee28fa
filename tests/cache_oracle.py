"""Plain 64-bit forms of the 8-bit cache's operators, on the CPU, for the tests."""
import math

import torch

F8 = torch.float8_e4m3fn


def e4m3(x):
    """x (float64) rounded to e4m3: halves to even, saturated; infinities and NaN to NaN."""
    a = x.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -40, max=1e30))).clamp(min=-6)
    step = torch.exp2(e - 3)
    y = (torch.round(x / step) * step).clamp(-448, 448)
    return torch.where(torch.isfinite(x), y, math.nan)


def block_scale(x):
    a = x.abs()
    a = a[torch.isfinite(a)]
    top = float(a.max()) if a.numel() else 0.0
    e = -60
    while e < 60 and top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def decode(codes):
    return codes.cpu().view(torch.uint8).view(F8).double()


class Cache64:
    """A copy of a device cache: stored values (without their scale) and scales, in 64 bits."""

    def __init__(self, cache, table):
        self.val = [decode(cache[0]), decode(cache[1])]
        self.scale = [cache[2].cpu().double(), cache[3].cpu().double()]
        self.table = table.cpu().long()
        self.P = self.val[0].shape[2]

    def rows(self, which, b, T):
        """[H, T, D]"""
        n = -(-T // self.P)
        p = self.table[b, :n]
        y = self.val[which][p] * self.scale[which][p][:, :, None, None]
        return y.permute(1, 0, 2, 3).reshape(y.shape[1], -1, y.shape[3])[:, :T]

    def append(self, b, base, k, v):
        """k, v [count, H, D]"""
        for which, x in ((0, k.double()), (1, v.double())):
            count, H, _ = x.shape
            for w in range(base // self.P, -(-(base + count) // self.P)):
                page = int(self.table[b, w])
                lo, hi = max(base, w * self.P), min(base + count, (w + 1) * self.P)
                a, z = lo - w * self.P, hi - w * self.P
                for h in range(H):
                    part = x[lo - base:hi - base, h]
                    s = block_scale(part)
                    if a:
                        was = float(self.scale[which][page, h])
                        s = max(s, was)
                        old = self.val[which][page, h, :a]
                        self.val[which][page, h, :a] = e4m3(old * was / s)
                    self.val[which][page, h, a:z] = e4m3(part / s)
                    self.scale[which][page, h] = s


def scores(q, k, scale, cap):
    """q [R, D], k [T, D] -> capped scores and the sum of the products' magnitudes."""
    x = q @ k.T * scale
    size = (q.abs() @ torch.nan_to_num(k).abs().T) * abs(scale)
    return (cap * torch.tanh(x / cap) if cap else x), size


def attend(c64, q, lens, n_query, mask, scale, cap):
    """out, lse [B, N, Hq(, D)] and the tolerances that the kernel's roundings give them.

    Scores: sums of head_dim products in fp32 (2^-24 each, head_dim <= 256, a product's error counted with its sum: 2^-17 of
    the products' magnitudes) and q carried to 2^-18 of its row's largest magnitude.  Probabilities: 16-bit floats of 11 bits
    (half a step: 2^-11) relative, with a floor of 2^-32 of the row's largest.  out: one rounding to its own type."""
    B, N, Hq, D = q.shape
    H = c64.val[0].shape[1]
    G = Hq // H
    eps = torch.finfo(q.dtype).eps / 2
    out, lse = torch.zeros(q.shape, dtype=torch.float64), torch.full((B, N, Hq), -math.inf, dtype=torch.float64)
    t_out, t_lse = torch.zeros_like(out), torch.zeros_like(lse)
    q = q.cpu().double()
    for b in range(B):
        n, base = int(n_query[b]), int(lens[b])
        T = base + n
        if T == 0 or n == 0:
            continue
        sees = torch.ones((n, T), dtype=torch.bool)
        sees[:, base:] = torch.tril(torch.ones((n, n))).bool() if mask is None else mask[b, :n, :n].cpu().bool()
        k, v = c64.rows(0, b, T), c64.rows(1, b, T)
        for hq in range(Hq):
            kk, vv = k[hq // G], v[hq // G]
            x, size = scores(q[b, :n, hq], kk, scale, cap)
            x = torch.where(sees, x, -math.inf)
            top = x.amax(1, keepdim=True).nan_to_num(neginf=0.0)
            p = torch.where(sees, torch.exp(x - top), 0.0)
            total = p.sum(1, keepdim=True)
            some = sees.any(1)
            vz = torch.where(sees[:, :, None], vv[None], 0.0)
            o = torch.einsum("nt,ntd->nd", p, vz) / total
            ds = torch.where(sees, size, 0.0).amax(1) * 2.0 ** -17
            qmax = q[b, :n, hq].abs().amax(1)
            ds = ds + abs(scale) * 2.0 ** -18 * qmax * torch.nan_to_num(kk).abs().sum(1).max()
            o_size = torch.einsum("nt,ntd->nd", p, vz.abs()) / total
            v_size = vz.abs().sum(1) / total
            out[b, :n, hq] = torch.where(some[:, None], o, 0.0)
            t_out[b, :n, hq] = eps * o.abs() + (2.0 ** -11 + 2 * ds[:, None] + 2.0 ** -18) * o_size + 2.0 ** -32 * v_size + 1e-30
            lse[b, :n, hq] = torch.where(some, (top + torch.log(total))[:, 0], -math.inf)
            t_lse[b, :n, hq] = ds + 2.0 ** -20 * (1 + lse[b, :n, hq].abs().nan_to_num(posinf=0.0))
    return out, lse, t_out, t_lse


def weights(c64, q, lse, lens, counts, index, scale, cap, prev):
    """out and its tolerance: scores as above but q carried to 2^-21, exponentials to 2^-19 of their exponent."""
    B, N, Hq, D = q.shape
    H = c64.val[0].shape[1]
    G = Hq // H
    out = prev.cpu().double().clone()
    tol = out.abs() * 2.0 ** -23
    q, lse = q.cpu().double(), lse.cpu().double()
    for b in range(B):
        n, base = int(counts[b]), int(lens[b])
        T = base + n
        if n == 0:
            continue
        k = c64.rows(0, b, T)
        for i in range(n):
            t = int(index[b, i]) if index is not None else i
            for hq in range(Hq):
                z = float(lse[b, t, hq])
                if z == -math.inf:
                    continue
                seen = base + i + 1
                x, size = scores(q[b, t, hq][None], k[hq // G, :seen], scale, cap)
                p = torch.exp(x[0] - z)
                ds = size[0] * 2.0 ** -17 + abs(scale) * 2.0 ** -21 * q[b, t, hq].abs().max() * k[hq // G, :seen].abs().sum(1)
                out[b, hq // G, :seen] += p
                tol[b, hq // G, :seen] += p * (2 * ds + 2.0 ** -19 * (1 + x[0].abs() + abs(z)))
    return out, tol + 1e-30


def evict(c64, weights, b, T, keep, recent):
    """Kept positions of a request [H][...]."""
    n = min(keep, T)
    late = min(recent, n)
    kept = []
    for h in range(c64.val[0].shape[1]):
        w = [float(x) for x in weights[b, h, :T - late]]
        order = sorted(range(T - late), key=lambda j: (math.inf if w[j] != w[j] else -w[j], j))
        kept.append(sorted(order[:n - late]) + list(range(T - late, T)))
    return kept
