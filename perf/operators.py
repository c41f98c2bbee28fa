"""The 8-bit cache operators on work as it comes up around speculative verification.

Four operators: rows written into a paged e4m3 cache (`append`), attention of the drafted rows over it (`attend`), the weight
that attention gave each cached token (`weights`), and a smaller cache of the heaviest tokens (`evict`).  With `own` false each
is computed from elementary torch operations in 32 bits; with `own` true by the library's entry points on the same tensors.

Sizes are those of the repository's benchmark (one request with k = 4, 64 requests with k = 8, 16 trees of 60 nodes) with the
usual head layouts (64 or 128 wide heads, 1 to 8 query heads to a cached head), and contexts from a few tokens to 131,072.
"""
import math

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
LOWEST, HIGHEST = -60, 60  # the exponents that a block's scale can have


# ------------------------------------------------------------------ cases

def listed():
    bf, hf = "bfloat16", "float16"
    return [
        # the 64 requests' step: 9 rows each (root and 8 drafted tokens) written behind contexts of their own length
        dict(name="append_batch64", op="append", B=64, n=9, Hkv=8, D=128, P=64, L=700, ragged=True, path=0, dtype=bf),
        # the accepted path of each of 16 trees, picked from its 60 nodes' rows
        dict(name="append_path", op="append", B=16, n=60, Hkv=8, D=128, P=32, L=333, ragged=True, path=7, dtype=hf),
        # four prompts
        dict(name="append_prompt", op="append", B=4, n=8001, Hkv=8, D=128, P=128, L=0, ragged=True, path=0, dtype=bf),
        # a single token of one request: latency
        dict(name="attend_token", op="attend", B=1, n=1, Hkv=8, G=4, D=128, P=64, L=1999, ragged=False, tree=False, cap=0.0, dtype=bf),
        # one request, k = 4, over a long document
        dict(name="attend_long", op="attend", B=1, n=5, Hkv=8, G=4, D=128, P=128, L=131067, ragged=False, tree=False, cap=0.0, dtype=bf),
        # 64 requests, k = 8, contexts of every length
        dict(name="attend_batch64", op="attend", B=64, n=9, Hkv=8, G=4, D=128, P=64, L=12000, ragged=True, tree=False, cap=0.0, dtype=bf),
        # 16 draft trees of 60 nodes with their ancestor masks
        dict(name="attend_tree60", op="attend", B=16, n=60, Hkv=8, G=4, D=128, P=64, L=6000, ragged=True, tree=True, cap=0.0, dtype=bf),
        # a small drafter's tokens: narrow heads, none shared, capped scores
        dict(name="attend_drafter", op="attend", B=32, n=1, Hkv=16, G=1, D=64, P=16, L=1501, ragged=True, tree=False, cap=30.0, dtype=hf),
        # the weights that one token gave a long document, and that a batch's committed rows gave theirs
        dict(name="weights_long", op="weights", B=1, n=1, Hkv=8, G=4, D=128, P=128, L=131067, ragged=False, path=False, cap=0.0, dtype=bf),
        dict(name="weights_batch64", op="weights", B=64, n=9, Hkv=8, G=4, D=128, P=64, L=5000, ragged=True, path=True, cap=0.0, dtype=bf),
        # a drafter's cache out of the target's: one long document, and a batch
        dict(name="evict_long", op="evict", B=1, Hkv=8, D=128, P=64, L=131071, ragged=False, keep=4096, recent=256),
        dict(name="evict_batch", op="evict", B=32, Hkv=8, D=64, P=32, L=7001, ragged=True, keep=1000, recent=65),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "weights", "evict"])
    c = dict(op=op, B=_spread(rng, 1, 64), Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]), P=rng.choice([16, 32, 64, 128]),
             ragged=rng.random() < 0.7)
    room = 1 << 20  # tokens times cached heads
    c["L"] = min(_spread(rng, 1, 131072), max(1, room // (c["B"] * c["Hkv"])))
    if op == "evict":
        c["keep"] = _spread(rng, 1, max(2, c["L"]))
        c["recent"] = rng.randint(0, c["keep"])
        return c
    c["dtype"] = rng.choice(["bfloat16", "float16"])
    c["n"] = _spread(rng, 1, 64)
    if op == "append":
        c["path"] = rng.choice([0, min(c["n"], 9)])
        if not c["path"]:
            c["n"] = _spread(rng, 1, max(2, (1 << 18) // (c["B"] * c["Hkv"])))
            c["L"] = min(c["L"], 2000)
        return c
    c["G"] = rng.choice([1, 2, 4, 8])
    c["cap"] = rng.choice([0.0, 0.0, 30.0])
    while c["B"] * c["n"] * c["G"] * c["Hkv"] * c["L"] > 1 << 28:
        c["n"], c["L"] = max(1, c["n"] // 2), max(1, c["L"] * 3 // 4)
    if op == "attend":
        c["tree"] = rng.random() < 0.5
    else:
        c["path"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------ inputs

def _lens(c, g, least=0):
    """Each request's context: L, or spread between a quarter of it and L."""
    if not c["ragged"]:
        return torch.full((c["B"],), c["L"], dtype=torch.int32, device="cuda")
    lo = max(least, c["L"] // 4)
    return torch.randint(lo, max(c["L"], lo) + 1, (c["B"],), generator=g, device="cuda", dtype=torch.int32)


def _pages(c, g, width):
    """A page table: every request's pages in the pool's order of hand-out, which is any."""
    B = c["B"]
    return torch.randperm(B * width, generator=g, device="cuda").to(torch.int32).reshape(B, width)


def _pool(c, g, pages):
    """A pool in use: e4m3 values over most of their range and each block's scale, keys with a few wide channels."""
    shape = (pages, c["Hkv"], c["P"], c["D"])
    pool = []
    for wide in (True, False):
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        if wide:
            x[..., ::16] *= 3
        e = torch.randint(-9, -6, (pages, c["Hkv"]), generator=g, device="cuda")
        scale = torch.exp2(e.float())
        pool += [(x * 64).clamp(-448, 448).to(E4M3), scale]
    return [pool[0], pool[2], pool[1], pool[3]]


def _tree(n, B, g):
    """Ancestor masks of random draft trees: each node's parent is one of the nodes shortly before it."""
    rows = np.random.RandomState(int(torch.randint(1 << 30, (1,), generator=g, device="cuda").item()))
    m = np.zeros((B, n, n), dtype=np.uint8)
    m[:, 0, 0] = 1
    for i in range(1, n):
        p = rows.randint(max(0, i - 8), i, B)
        m[:, i] = m[np.arange(B), p]
        m[:, i, i] = 1
    return torch.from_numpy(m).cuda()


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    B, Hkv, D, P = c["B"], c["Hkv"], c["D"], c["P"]
    s = dict(case=c)
    if c["op"] == "evict":
        lens, W = _lens(c, g, 1), -(-c["L"] // P)
        D_W = -(-c["keep"] // P)
        every = torch.randperm(B * (W + D_W), generator=g, device="cuda").to(torch.int32)
        s["table"] = every[:B * W].reshape(B, W)
        s["dst"] = every[B * W:].reshape(B, D_W)
        s["cache"] = _pool(c, g, B * (W + D_W))
        w = torch.randn((B, Hkv, c["L"]), generator=g, device="cuda")
        s.update(lens=lens, weights=torch.exp(2 * w) * 1e-3)
        s["out"] = dict(kept=torch.empty((B, Hkv, c["keep"]), dtype=torch.int32, device="cuda"),
                        weights=torch.empty((B, Hkv, c["keep"]), device="cuda"),
                        new_len=torch.empty(B, dtype=torch.int32, device="cuda"),
                        status=torch.empty(B, dtype=torch.int32, device="cuda"))
        return s
    dtype = getattr(torch, c["dtype"])
    lens = _lens(c, g)
    rows = c["path"] if c["op"] == "append" and c["path"] else c["n"]
    W = -(-(c["L"] + rows) // P)
    s.update(lens=lens, table=_pages(c, g, W), cache=_pool(c, g, B * W))
    if c["op"] == "append":
        shape = (B, c["n"], Hkv, D)
        s["k"] = (torch.randn(shape, generator=g, device="cuda") * (2 * torch.rand((1, 1, Hkv, D), generator=g, device="cuda"))).to(dtype)
        s["v"] = torch.randn(shape, generator=g, device="cuda").to(dtype)
        s["counts"] = torch.randint(max(1, rows // 2), rows + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if c["ragged"] else torch.full(
            (B,), rows, dtype=torch.int32, device="cuda")
        s["index"] = None
        if c["path"]:
            pick = torch.rand((B, c["n"]), generator=g, device="cuda").argsort(1)[:, :rows].sort(1).values
            s["index"] = pick.to(torch.int32).contiguous()
        s["out"] = dict(new_len=torch.empty(B, dtype=torch.int32, device="cuda"), status=torch.empty(B, dtype=torch.int32, device="cuda"))
        return s
    Hq = Hkv * c["G"]
    s["q"] = (torch.randn((B, c["n"], Hq, D), generator=g, device="cuda") * 1.5).to(dtype)
    if c["op"] == "attend":
        s["mask"] = _tree(c["n"], B, g) if c["tree"] else None
        s["out"] = dict(out=torch.empty((B, c["n"], Hq, D), dtype=dtype, device="cuda"), lse=torch.empty((B, c["n"], Hq), device="cuda"),
                        status=torch.empty(B, dtype=torch.int32, device="cuda"))
        return s
    s["counts"] = s["index"] = None
    if c["path"]:
        s["index"] = torch.rand((B, c["n"]), generator=g, device="cuda").argsort(1).sort(1).values.to(torch.int32).contiguous()
        s["counts"] = torch.randint(1, c["n"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    s["prev"] = torch.rand((B, Hkv, W * P), generator=g, device="cuda") * 1e-3
    # the rows' normalisers, as the attention over the same cache gave them
    q, kk, _, t = _gathered(s, s["index"], s["counts"])
    seen = _visible(s, t, None, s["counts"])
    x = _scores(s, q, kk).masked_fill(~seen[:, None, :, None, :], -math.inf)
    lse = torch.logsumexp(x, -1).permute(0, 2, 1, 3).reshape(B, c["n"], Hq)
    s["lse"] = torch.zeros_like(lse)
    at = s["index"].long() if s["index"] is not None else torch.arange(c["n"], device="cuda").expand(B, -1)
    s["lse"].scatter_(1, at[:, :, None].expand(-1, -1, Hq), lse)
    s["out"] = dict(weights=s["prev"].clone(), status=torch.empty(B, dtype=torch.int32, device="cuda"))
    return s


# ------------------------------------------------------------------ the plain forms

def _dense(cache, table, wide=torch.float32):
    """The cache's values in the order of positions: [B, Hkv, W * P, D]."""
    out = []
    for x, scale in ((cache[0], cache[2]), (cache[1], cache[3])):
        y = x.view(torch.uint8)[table.long()].view(E4M3).to(wide) * scale[table.long()].to(wide)[..., None, None]
        B, W, H, P, D = y.shape
        out.append(y.permute(0, 2, 1, 3, 4).reshape(B, H, W * P, D))
    return out


def _gathered(s, index=None, counts=None, wide=torch.float32):
    """The query rows grouped by cached head [B, Hkv, n, G, D], the dense keys and values, the positions."""
    c = s["case"]
    kk, vv = _dense(s["cache"], s["table"], wide)
    q = s["q"].to(wide)
    if index is not None:
        q = torch.gather(q, 1, index.long()[:, :, None, None].expand(-1, -1, q.shape[2], q.shape[3]))
    B, n, Hq, D = q.shape
    q = q.reshape(B, n, c["Hkv"], c["G"], D).permute(0, 2, 1, 3, 4)
    return q, kk, vv, torch.arange(kk.shape[2], device=kk.device)


def _scores(s, q, kk):
    """Capped, scaled scores [B, Hkv, n, G, T]."""
    c = s["case"]
    B, H, n, G, D = q.shape
    x = torch.matmul(q.reshape(B, H, n * G, D), kk.transpose(-1, -2)).reshape(B, H, n, G, -1) * (1 / math.sqrt(D))
    return c["cap"] * torch.tanh(x / c["cap"]) if c["cap"] else x


def _visible(s, t, mask=None, counts=None):
    """[B, n, T]: the context, and of the drafted rows a row's ancestors (or the rows up to it) and itself."""
    n = s["case"]["n"]
    base = s["lens"].long()[:, None, None]
    j = t[None, None, :] - base
    i = torch.arange(n, device=t.device)[None, :, None]
    top = n if counts is None else counts.long()[:, None, None]
    if mask is None:
        draft = (j >= 0) & (j <= i)
    else:
        draft = (j >= 0) & (j < n) & torch.gather(mask.bool(), 2, j.clamp(0, n - 1).expand(-1, n, -1))
    return ((j < 0) | draft) & (j < top) & (i < top)


def _needed(amax):
    """The power of two that a block's largest value asks for."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(LOWEST, HIGHEST)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.full_like(amax, 2.0 ** LOWEST))


def _plain_append(s):
    c = s["case"]
    B, H, D, P = c["B"], c["Hkv"], c["D"], c["P"]
    base, cnt = s["lens"].long(), s["counts"].long()
    rows = c["path"] or c["n"]
    touched = (rows + P - 2) // P + 1
    first = base // P
    which = first[:, None] + torch.arange(touched, device="cuda")  # [B, touched] pages of a request
    live = (which * P < (base + cnt)[:, None]) & (which < s["table"].shape[1])
    page = torch.gather(s["table"].long(), 1, which.clamp(max=s["table"].shape[1] - 1))
    pos = which[:, :, None] * P + torch.arange(P, device="cuda")  # [B, touched, P]
    src = pos - base[:, None, None]
    new = (src >= 0) & (src < cnt[:, None, None])
    src = src.clamp(0, rows - 1)
    if s["index"] is not None:
        src = torch.gather(s["index"].long(), 1, src.reshape(B, -1)).reshape(src.shape)
    older = pos < base[:, None, None]
    held = older.any(-1)  # [B, touched]
    to = page[live]
    for pool, scales, x in ((s["cache"][0], s["cache"][2], s["k"]), (s["cache"][1], s["cache"][3], s["v"])):
        fresh = torch.gather(x, 1, src.reshape(B, -1)[:, :, None, None].expand(-1, -1, H, D)).float()
        fresh = fresh.reshape(B, touched, P, H, D).permute(0, 1, 3, 2, 4)
        fresh = torch.where(new[:, :, None, :, None], fresh, 0.0)
        was = scales[page]
        scale = torch.where(held[:, :, None], was, 0.0).maximum(_needed(fresh.abs().amax((-1, -2))))
        old = pool.view(torch.uint8)[page].view(E4M3).float() * was[..., None, None]
        values = torch.where(new[:, :, None, :, None], fresh, old) / scale[..., None, None]
        code = values.clamp(-448, 448).to(E4M3).view(torch.uint8)
        keep = (new | older)[:, :, None, :, None]
        code = torch.where(keep, code, pool.view(torch.uint8)[page])
        pool.view(torch.uint8)[to] = code[live]
        scales[to] = scale[live]
    return dict(k=s["cache"][0], v=s["cache"][1], k_scale=s["cache"][2], v_scale=s["cache"][3], new_len=s["lens"] + s["counts"])


def _plain_attend(s):
    c = s["case"]
    q, kk, vv, t = _gathered(s)
    x = _scores(s, q, kk).masked_fill_(~_visible(s, t, s["mask"])[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    B, H, n, G, T = p.shape
    T_all = torch.arange(T, device="cuda")
    vv = torch.where((T_all < (s["lens"] + n)[:, None])[:, None, :, None], vv, 0.0)
    o = torch.matmul(p.reshape(B, H, n * G, T), vv).reshape(B, H, n, G, -1) / total
    lse = (top + torch.log(total))[..., 0].permute(0, 2, 1, 3).reshape(B, n, H * G)
    return dict(out=o.permute(0, 2, 1, 3, 4).reshape(B, n, H * G, -1).to(s["q"].dtype), lse=lse)


def _plain_weights(s):
    q, kk, _, t = _gathered(s, s["index"], s["counts"])
    lse = s["lse"]
    if s["index"] is not None:
        lse = torch.gather(lse, 1, s["index"].long()[:, :, None].expand(-1, -1, lse.shape[2]))
    B, H, n, G, D = q.shape
    lse = lse.reshape(B, n, H, G).permute(0, 2, 1, 3)[..., None]
    p = torch.exp(_scores(s, q, kk) - lse)
    p = torch.where(_visible(s, t, None, s["counts"])[:, None, :, None, :], p, 0.0)
    return dict(weights=s["prev"] + p.sum((2, 3)))


def _plain_evict(s):
    c = s["case"]
    B, H, D, P, keep = c["B"], c["Hkv"], c["D"], c["P"], c["keep"]
    L = c["L"]
    n = s["lens"].long()[:, None, None]
    pos = torch.arange(L, device="cuda")[None, None, :]
    kc = n.clamp(max=keep)
    rc = kc.clamp(max=c["recent"])
    w = torch.where(pos >= n - rc, math.inf, s["weights"])
    w = torch.where(pos < n, w, -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    slot = torch.arange(order.shape[-1], device="cuda")
    order = torch.where(slot < kc, order, L).sort(-1).values
    if order.shape[-1] < keep:
        order = torch.nn.functional.pad(order, (0, keep - order.shape[-1]), value=L)
    real = order < L
    kept = torch.where(real, order, -1).to(torch.int32)
    at = order.clamp(max=L - 1)
    weights = torch.where(real, torch.gather(s["weights"], 2, at), 0.0)
    Wd = s["dst"].shape[1]
    full = torch.nn.functional.pad(at, (0, Wd * P - keep))
    mine = torch.nn.functional.pad(real, (0, Wd * P - keep))
    page = torch.gather(s["table"].long(), 1, (full // P).reshape(B, -1)).reshape(full.shape)
    head = torch.arange(H, device="cuda")[None, :, None].expand(B, H, Wd * P)
    to = s["dst"].long()
    live = torch.arange(Wd, device="cuda")[None, :] * P < kc[:, 0]
    for pool, scales in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])):
        raw = pool.view(torch.uint8)
        x = raw[page, head, full % P].view(E4M3).float() * scales[page, head][..., None]
        x = torch.where(mine[..., None], x, 0.0).reshape(B, H, Wd, P, D)
        scale = _needed(x.abs().amax((-1, -2)))
        code = (x / scale[..., None, None]).clamp(-448, 448).to(E4M3).view(torch.uint8)
        code, scale = code.transpose(1, 2), scale.transpose(1, 2)
        code = torch.where(mine.reshape(B, H, Wd, P, 1).transpose(1, 2), code, raw[to])
        raw[to[live]] = code[live]
        scales[to[live]] = scale[live]
    return dict(kept=kept, weights=weights, new_len=kc[:, 0, 0].to(torch.int32), k=s["cache"][0], v=s["cache"][1],
                k_scale=s["cache"][2], v_scale=s["cache"][3])


# ------------------------------------------------------------------ a pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return dict(append=_plain_append, attend=_plain_attend, weights=_plain_weights, evict=_plain_evict)[c["op"]](s)
    from speculative_decoding_verification_02_gb300 import api
    k, v, ks, vs = cache = s["cache"]
    if c["op"] == "append":
        o = api.spec_cache_append(cache, s["table"], s["lens"], s["k"], s["v"], counts=s["counts"], index=s["index"], out=s["out"])
        return dict(k=k, v=v, k_scale=ks, v_scale=vs, new_len=o["new_len"])
    if c["op"] == "attend":
        o = api.spec_cache_attend(s["q"], cache, s["table"], s["lens"], mask=s["mask"], softcap=c["cap"], out=s["out"])
        return dict(out=o["out"], lse=o["lse"])
    if c["op"] == "weights":
        o = api.spec_cache_weights(s["q"], s["lse"], cache, s["table"], s["lens"], prev=s["prev"], counts=s["counts"], index=s["index"],
                                   softcap=c["cap"], out=s["out"])
        return dict(weights=o["weights"])
    o = api.spec_cache_evict(cache, s["table"], s["lens"], s["weights"], c["keep"], c["recent"], s["dst"], out=s["out"])
    return dict(kept=o["kept"], weights=o["weights"], new_len=o["new_len"], k=k, v=v, k_scale=ks, v_scale=vs)


def work(case):
    """Bytes and operations of one pass, with each request's context at its mean."""
    c = case
    B, H, D = c["B"], c["Hkv"], c["D"]
    L = c["L"] * (0.625 if c["ragged"] else 1.0)
    if c["op"] == "append":
        n = (c["path"] or c["n"]) * (0.75 if c["ragged"] else 1.0)
        return dict(bytes=B * n * H * D * 2 * (2 + 1), flops=B * n * H * D * 2 * 2)
    if c["op"] == "evict":
        n = min(c["keep"], L)
        return dict(bytes=B * H * (4 * L + n * (4 * D + 8)), flops=B * H * L)
    rows = c["n"] * (0.5 if c["op"] == "weights" and c["path"] else 1.0)
    T = L + rows
    q = B * rows * H * c["G"] * D
    if c["op"] == "attend":
        return dict(bytes=B * T * H * D * 2 + 4 * q + 4 * q / D + (B * c["n"] ** 2 if c["tree"] else 0), flops=4.0 * q * T)
    return dict(bytes=B * T * H * (D + 8) + 2 * q, flops=2.0 * q * T)


# ------------------------------------------------------------------ the definitions in 64 bits

def _e4m3(x):
    """x rounded to e4m3: three bits after the leading one, exponents from -6, halves to even, at most 448."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _block_scale(amax):
    e = LOWEST
    while e < HIGHEST and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def _exact_append(s):
    c = s["case"]
    P, H = c["P"], c["Hkv"]
    done = {}
    for name, pool, scales, x in (("k", s["cache"][0], s["cache"][2], s["k"]), ("v", s["cache"][1], s["cache"][3], s["v"])):
        vals, sc = pool.cpu().double(), scales.cpu().double()
        x = x.cpu().double()
        for b in range(c["B"]):
            base, cnt = int(s["lens"][b]), int(s["counts"][b])
            pick = s["index"][b, :cnt].cpu().long() if s["index"] is not None else torch.arange(cnt)
            rows = x[b, pick]
            for w in range(base // P, -(-(base + cnt) // P)):
                page = int(s["table"][b, w])
                lo, hi = max(base, w * P), min(base + cnt, w * P + P)
                part = rows[lo - base:hi - base]
                top = part.abs().amax((0, 2))
                for h in range(H):
                    new = _block_scale(float(top[h]))
                    held = lo - w * P
                    if held:
                        new = max(new, float(sc[page, h]))
                        vals[page, h, :held] = _e4m3(vals[page, h, :held] * float(sc[page, h]) / new)
                    vals[page, h, held:hi - w * P] = _e4m3(part[:, h] / new)
                    sc[page, h] = new
        done[name], done[name + "_scale"] = vals, sc
    return dict(k=done["k"], v=done["v"], k_scale=done["k_scale"], v_scale=done["v_scale"], new_len=None)


def _rows_of(s, b, T):
    """Request b's keys and values [T, Hkv, D] in 64 bits."""
    P = s["case"]["P"]
    pages = s["table"][b, :-(-T // P)].long()
    out = []
    for x, scale in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])):
        y = x.view(torch.uint8)[pages].view(E4M3).double() * scale[pages].double()[:, :, None, None]
        out.append(y.permute(0, 2, 1, 3).reshape(-1, y.shape[1], y.shape[3])[:T])
    return out


def _exact_scores(c, q, k):
    x = torch.einsum("nhgd,thd->hngt", q, k) / math.sqrt(c["D"])
    return c["cap"] * torch.tanh(x / c["cap"]) if c["cap"] else x


def _seen(n, base, T, mask=None):
    sees = torch.ones((n, T), dtype=torch.bool, device="cuda")
    sees[:, base:base + n] = (torch.tril(torch.ones((n, n), device="cuda")) if mask is None else mask)[:, :T - base].bool()
    return sees


def _exact_attend(s):
    c = s["case"]
    n, H, G = c["n"], c["Hkv"], c["G"]
    out, lse = [], []
    for b in range(c["B"]):
        base = int(s["lens"][b])
        T = base + n
        k, v = _rows_of(s, b, T)
        x = _exact_scores(c, s["q"][b].double().reshape(n, H, G, -1), k)
        sees = _seen(n, base, T, None if s["mask"] is None else s["mask"][b])
        x = torch.where(sees[None, :, None, :], x, -math.inf)
        z = torch.logsumexp(x, -1)
        out.append(torch.einsum("hngt,thd->nhgd", torch.exp(x - z[..., None]), v).reshape(n, H * G, -1))
        lse.append(z.permute(1, 0, 2).reshape(n, H * G))
    return dict(out=torch.stack(out), lse=torch.stack(lse))


def _exact_weights(s):
    c = s["case"]
    H, G = c["Hkv"], c["G"]
    total = s["prev"].double().clone()
    for b in range(c["B"]):
        base = int(s["lens"][b])
        n = c["n"] if s["counts"] is None else int(s["counts"][b])
        pick = torch.arange(n, device="cuda") if s["index"] is None else s["index"][b, :n].long()
        k, _ = _rows_of(s, b, base + n)
        x = _exact_scores(c, s["q"][b, pick].double().reshape(n, H, G, -1), k)
        z = s["lse"][b, pick].double().reshape(n, H, G).permute(1, 0, 2)[..., None]
        p = torch.exp(x - z) * _seen(n, base, base + n)[None, :, None, :]
        total[b, :, :base + n] += p.sum((1, 2))
    return dict(weights=total)


def _exact_evict(s):
    c = s["case"]
    H, P, keep = c["Hkv"], c["P"], c["keep"]
    weights = torch.zeros((c["B"], H, keep), dtype=torch.float64)
    pools = [x.cpu().double() for x in s["cache"]]
    for b in range(c["B"]):
        T = int(s["lens"][b])
        n = min(keep, T)
        late = min(c["recent"], n)
        k, v = (x.cpu() for x in _rows_of(s, b, T))
        w = s["weights"][b].cpu().double().numpy()
        for h in range(H):
            heavy = np.lexsort((np.arange(T - late), -w[h, :T - late]))[:n - late]
            at = torch.from_numpy(np.concatenate([np.sort(heavy), np.arange(T - late, T)]))
            weights[b, h, :n] = torch.from_numpy(w[h])[at]
            for j in range(-(-n // P)):
                page = int(s["dst"][b, j])
                m = min(P, n - j * P)
                for vals, scales, x in ((pools[0], pools[2], k), (pools[1], pools[3], v)):
                    part = x[at[j * P:j * P + m], h]
                    scales[page, h] = _block_scale(float(part.abs().max()))
                    vals[page, h, :m] = _e4m3(part / scales[page, h])
    return dict(kept=None, weights=weights, new_len=None, k=pools[0], v=pools[1], k_scale=pools[2], v_scale=pools[3])


def exact(case, seed):
    s = prepare(case, seed)
    return dict(append=_exact_append, attend=_exact_attend, weights=_exact_weights, evict=_exact_evict)[case["op"]](s)
