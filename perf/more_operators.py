"""Linear attention with a decay for each head, on work as it comes up around speculative verification.

A layer of this kind keeps one fp32 state [Dk, Dv] for each head of a request in place of a cache:

    S_t = exp(g_t) S_{t-1} + k_t v_t^T        o_t = scale q_t^T S_t

Three operators: tokens of a prompt, of a part of one, or a single token, with the new state (`forward`); the drafted rows or
tree nodes of a verify step, over a state that stays as it is (`attend`); the state advanced by the rows that verification
accepted (`commit`).  With `own` false each is computed from elementary torch operations in 32 bits (running sums of decays in
64); with `own` true by the library's entry points on the same tensors.

Sizes are those of the repository's benchmark (one request with k = 4, 64 requests with k = 8, 16 trees of 60 nodes) with the
heads of its survey's 144 MiB state (48 layers of 48 heads of 128 x 128, three to a query and key head), and of smaller layers.
"""
import math

import numpy as np
import torch

own = False

CHUNK = 64  # tokens that the plain form takes at once


# ------------------------------------------------------------------ cases

def listed():
    bf, hf = "bfloat16", "float16"
    return [
        # one request decoding: a single token of one layer, where latency counts
        dict(name="forward_token", op="forward", B=1, n=1, Hk=16, G=3, Dk=128, Dv=128, ragged=False, fresh=False, dtype=bf),
        # 64 requests decoding together
        dict(name="forward_batch64", op="forward", B=64, n=1, Hk=16, G=3, Dk=128, Dv=128, ragged=False, fresh=False, dtype=bf),
        # a long document, from no state
        dict(name="forward_document", op="forward", B=1, n=32003, Hk=16, G=3, Dk=128, Dv=128, ragged=False, fresh=True, dtype=bf),
        # prompts of every length behind states of their own, every head with its own query and key
        dict(name="forward_prompts", op="forward", B=8, n=8001, Hk=32, G=1, Dk=128, Dv=128, ragged=True, fresh=False, dtype=bf),
        # prompts of a small drafter: narrow heads, fp16
        dict(name="forward_drafter", op="forward", B=8, n=2000, Hk=16, G=1, Dk=64, Dv=64, ragged=True, fresh=True, dtype=hf),
        # one request's drafted chain, k = 4
        dict(name="attend_chain", op="attend", B=1, n=5, Hk=16, G=3, Dk=128, Dv=128, ragged=False, tree=False, dtype=bf),
        # 64 requests, k = 8, drafts of different lengths
        dict(name="attend_batch64", op="attend", B=64, n=9, Hk=16, G=3, Dk=128, Dv=128, ragged=True, tree=False, dtype=bf),
        # 16 draft trees of 60 nodes
        dict(name="attend_tree60", op="attend", B=16, n=60, Hk=16, G=3, Dk=128, Dv=128, ragged=False, tree=True, dtype=bf),
        # the accepted rows of one request; of 64; and of 16 trees, picked from their nodes' rows
        dict(name="commit_chain", op="commit", B=1, n=5, Hk=16, G=3, Dk=128, Dv=128, ragged=False, path=0, dtype=bf),
        dict(name="commit_batch64", op="commit", B=64, n=9, Hk=16, G=3, Dk=128, Dv=128, ragged=True, path=0, dtype=bf),
        dict(name="commit_path", op="commit", B=16, n=60, Hk=32, G=1, Dk=128, Dv=64, ragged=True, path=7, dtype=hf),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "attend", "commit"])
    c = dict(op=op, B=_spread(rng, 1, 64), Hk=rng.choice([1, 2, 4, 8, 16]), G=rng.choice([1, 2, 3]), Dk=rng.choice([64, 128]),
             Dv=rng.choice([64, 128]), ragged=rng.random() < 0.6, dtype=rng.choice(["bfloat16", "float16"]))
    if op == "forward":
        c["fresh"] = rng.random() < 0.4
        c["n"] = _spread(rng, 1, 20000)
        while c["B"] * c["n"] * c["Hk"] * c["G"] > 30000 * 48:
            c["B"], c["n"] = max(1, c["B"] // 2), max(1, c["n"] * 3 // 4)
    else:
        c["n"] = _spread(rng, 1, 60)
        if op == "attend":
            c["tree"] = rng.random() < 0.5
            c["B"] = min(c["B"], max(1, 960 // c["n"]))
        else:
            c["path"] = rng.choice([0, min(c["n"], 9)])
    return c


# ------------------------------------------------------------------ inputs

def _parents(n, B, g):
    """Random draft trees of depth 6 at most: each node hangs on one of the ten before it that are shallow enough."""
    rng = np.random.RandomState(int(torch.randint(1 << 30, (1,), generator=g, device="cuda").item()))
    parents = np.full((B, n), -1, dtype=np.int32)
    depth = np.zeros((B, n), dtype=np.int32)
    for b in range(B):
        for i in range(1, n):
            may = [j for j in range(max(0, i - 10), i) if depth[b, j] < 6] or [0]
            parents[b, i] = may[rng.randint(len(may))]
            depth[b, i] = depth[b, parents[b, i]] + 1
    return torch.from_numpy(parents).cuda()


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    B, n, Hk, H, Dk, Dv = c["B"], c["n"], c["Hk"], c["Hk"] * c["G"], c["Dk"], c["Dv"]
    dtype = getattr(torch, c["dtype"])
    s = dict(case=c)
    s["q"] = torch.randn((B, n, Hk, Dk), generator=g, device="cuda").to(dtype)
    k = torch.randn((B, n, Hk, Dk), generator=g, device="cuda")
    s["k"] = (k / torch.linalg.vector_norm(k, dim=-1, keepdim=True)).to(dtype)  # keys are normed, as such layers do
    del k
    s["v"] = torch.randn((B, n, H, Dv), generator=g, device="cuda").to(dtype)
    # heads that remember a token or so, and heads that remember thousands, each token with its own share of that
    rate = torch.exp(-7 * torch.rand((1, 1, H), generator=g, device="cuda"))
    s["decay"] = -rate * (0.1 + 1.8 * torch.rand((B, n, H), generator=g, device="cuda"))
    fresh = c["op"] == "forward" and c["fresh"]
    # a pool of slots with room to spare, handed out in any order
    pool = B + 2
    s["state"] = None if fresh else torch.randn((pool, H, Dk, Dv), generator=g, device="cuda") * (0.3 / torch.sqrt(rate.reshape(1, H, 1, 1) + 0.01))
    s["slots"] = torch.randperm(pool, generator=g, device="cuda")[:B].to(torch.int32)
    rows = c["path"] if c["op"] == "commit" and c["path"] else n
    s["counts"] = None
    if c["ragged"]:
        s["counts"] = torch.randint(max(1, rows // 4), rows + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    status = torch.empty(B, dtype=torch.int32, device="cuda")
    if c["op"] != "attend":  # the states after the call: a pool of their own
        s["to"] = torch.zeros((B, H, Dk, Dv), device="cuda")
    if c["op"] == "commit":
        s["index"] = None
        if c["path"]:
            pick = torch.rand((B, n), generator=g, device="cuda").argsort(1)[:, :rows].sort(1).values
            s["index"] = pick.to(torch.int32).contiguous()
        s["out"] = dict(status=status)
    else:
        s["out"] = dict(out=torch.empty((B, n, H, Dv), dtype=dtype, device="cuda"), status=status)
    if c["op"] == "attend":
        s["parents"] = _parents(n, B, g) if c["tree"] else None
    return s


# ------------------------------------------------------------------ the plain forms

def _heads(x, G):
    """[B, n, heads, D] -> fp32 [B, H, n, D], a key head's rows repeated for each of its G state heads."""
    x = x.float().transpose(1, 2)
    return x.repeat_interleave(G, 1) if G > 1 else x


def _start(s):
    """The requests' states [B, H, Dk, Dv]."""
    c = s["case"]
    if s["state"] is None:
        return torch.zeros((c["B"], c["Hk"] * c["G"], c["Dk"], c["Dv"]), device="cuda")
    return s["state"][s["slots"].long()]


def _live(s, rows):
    """Which of a request's rows count: [B, rows]."""
    i = torch.arange(rows, device="cuda")[None]
    return i < (s["counts"][:, None] if s["counts"] is not None else rows)


def _plain_forward(s):
    c = s["case"]
    B, n, G, scale = c["B"], c["n"], c["G"], c["Dk"] ** -0.5
    S = _start(s)
    live = _live(s, n)
    out = torch.empty((B, n, c["Hk"] * G, c["Dv"]), dtype=s["q"].dtype, device="cuda")
    for t in range(0, n, CHUNK):
        e = min(n, t + CHUNK)
        on = live[:, None, t:e, None]
        q = _heads(s["q"][:, t:e], G)
        k = torch.where(on, _heads(s["k"][:, t:e], G), 0.0)
        v = torch.where(on, _heads(s["v"][:, t:e], 1), 0.0)
        run = torch.where(live[:, t:e, None], s["decay"][:, t:e], 0.0).double().cumsum(1).transpose(1, 2)  # [B, H, C]
        between = torch.exp((run[..., :, None] - run[..., None, :]).float())
        a = torch.matmul(q, k.transpose(-1, -2)) * torch.tril(between)
        o = torch.matmul(q, S) * torch.exp(run.float())[..., None] + torch.matmul(a, v)
        out[:, t:e] = torch.where(on, o * scale, 0.0).transpose(1, 2).to(out.dtype)
        left = torch.exp((run[..., -1:] - run).float())
        S = S * torch.exp(run[..., -1].float())[..., None, None] + torch.matmul((k * left[..., None]).transpose(-1, -2), v)
    return dict(out=out, state=S)


def _plain_attend(s):
    c = s["case"]
    B, n, G, scale = c["B"], c["n"], c["G"], c["Dk"] ** -0.5
    live = _live(s, n)
    if s["parents"] is None:
        sees = torch.ones((n, n), device="cuda").tril()[None].expand(B, -1, -1)
    else:  # a node's ancestors and itself, by doubling the length of the paths that are followed
        eye = torch.eye(n, device="cuda")[None].expand(B, -1, -1)
        up = torch.where(s["parents"][..., None] == torch.arange(n, device="cuda"), 1.0, 0.0)
        sees, span = torch.clamp(eye + up, max=1.0), 1
        while span < n:
            sees, span = torch.clamp(torch.matmul(sees, sees), max=1.0), span * 2
    q, k, v = _heads(s["q"], G), _heads(s["k"], G), _heads(s["v"], 1)
    path = torch.matmul(sees.double(), s["decay"].double()).transpose(1, 2)  # [B, H, n]
    between = torch.where(sees[:, None] > 0, torch.exp((path[..., :, None] - path[..., None, :]).float()), 0.0)
    a = torch.matmul(q, k.transpose(-1, -2)) * between
    o = torch.matmul(q, _start(s)) * torch.exp(path.float())[..., None] + torch.matmul(a, v)
    return dict(out=torch.where(live[:, None, :, None], o * scale, 0.0).transpose(1, 2).to(s["q"].dtype))


def _picked(s, x):
    """The rows of x that are committed."""
    if s["index"] is None:
        return x
    at = s["index"].long().reshape(s["index"].shape + (1,) * (x.dim() - 2))
    return torch.gather(x, 1, at.expand(-1, -1, *x.shape[2:]))


def _plain_commit(s):
    G = s["case"]["G"]
    k, v, g = (_picked(s, s[x]) for x in ("k", "v", "decay"))
    live = _live(s, k.shape[1])
    run = torch.where(live[..., None], g, 0.0).double().cumsum(1).transpose(1, 2)
    left = torch.exp((run[..., -1:] - run).float())
    k = torch.where(live[:, None, :, None], _heads(k, G), 0.0) * left[..., None]
    v = torch.where(live[:, None, :, None], _heads(v, 1), 0.0)
    return dict(state=_start(s) * torch.exp(run[..., -1].float())[..., None, None] + torch.matmul(k.transpose(-1, -2), v))


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"forward": _plain_forward, "attend": _plain_attend, "commit": _plain_commit}[op](s)
    from speculative_decoding_verification_02_gb300 import api
    if op == "forward":
        api.spec_state_forward(s["q"], s["k"], s["v"], s["decay"], s["state"], slots=s["slots"], dst=s["to"], counts=s["counts"],
                               out=s["out"])
        return dict(out=s["out"]["out"], state=s["to"])
    if op == "attend":
        api.spec_state_attend(s["q"], s["k"], s["v"], s["decay"], s["state"], slots=s["slots"], parents=s["parents"],
                              n_query=s["counts"], out=s["out"])
        return dict(out=s["out"]["out"])
    api.spec_state_commit(s["k"], s["v"], s["decay"], s["state"], slots=s["slots"], dst=s["to"], index=s["index"],
                          counts=s["counts"], out=s["out"])
    return dict(state=s["to"])


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    B, n, Hk, H, Dk, Dv = c["B"], c["n"], c["Hk"], c["Hk"] * c["G"], c["Dk"], c["Dv"]
    rows = c["path"] if c["op"] == "commit" and c["path"] else n
    live = B * ((max(1, rows // 4) + rows) / 2 if c["ragged"] else rows)  # rows that count, on average
    S = B * H * Dk * Dv
    size = live * (Hk * Dk * 2 + H * Dv * 2 + H * 4)  # k, v, decay
    if c["op"] == "commit":
        return {"bytes": size + 2 * 4 * S, "flops": live * H * 2 * Dk * Dv}
    size += live * Hk * Dk * 2 + B * n * H * Dv * 2  # q; out, whose rows past the count are zeros
    if c["op"] == "forward":
        return {"bytes": size + 4 * S * (1 if c["fresh"] else 2), "flops": live * H * 4 * Dk * Dv}
    pairs = live * (4 if c["tree"] else (n + 1) / 2)
    return {"bytes": size + 4 * S, "flops": H * (live * 2 * Dk * Dv + pairs * 2 * (Dk + Dv))}


# ------------------------------------------------------------------ the definition, token by token in 64 bits

def _steps(s, at, wants_out):
    """The recurrence over the rows `at` [B, rows] of each request; a request's steps past its count do nothing."""
    c = s["case"]
    B, H, G, Dk, Dv, scale = c["B"], c["Hk"] * c["G"], c["G"], c["Dk"], c["Dv"], c["Dk"] ** -0.5
    S = torch.zeros((B, H, Dk, Dv), dtype=torch.float64, device="cuda")
    if s["state"] is not None:
        for b, slot in enumerate(s["slots"].tolist()):
            S[b] = s["state"][slot]
    counts = [at.shape[1]] * B if s["counts"] is None else s["counts"].tolist()
    head = torch.arange(H, device="cuda") // G
    who = torch.arange(B, device="cuda")
    out = torch.zeros((B, c["n"], H, Dv), dtype=torch.float64, device="cuda") if wants_out else None
    order = sorted(range(B), key=lambda b: -counts[b])  # the requests still running come first
    S = S[order]
    for t in range(at.shape[1]):
        m = sum(1 for x in counts if x > t)
        if m == 0:
            break
        b = who[order[:m]] if m < B else who[order]
        row = at[b, t]
        k = s["k"][b, row][:, head].double()
        v = s["v"][b, row].double()
        f = torch.exp(s["decay"][b, row].double())
        S[:m].mul_(f[:, :, None, None]).add_(k[..., :, None] * v[..., None, :])
        if wants_out:
            q = s["q"][b, row][:, head].double()
            out[b, row] = scale * torch.einsum("bhk,bhkv->bhv", q, S[:m])
    back = [0] * B
    for i, b in enumerate(order):
        back[b] = i
    return out, S[back]


def exact(case, seed):
    c = case
    B, n, H, Dk, Dv = c["B"], c["n"], c["Hk"] * c["G"], c["Dk"], c["Dv"]
    # a step reads and writes the states in 64 bits some three times
    steps = c["path"] if c["op"] == "commit" and c["path"] else n
    if steps * (5e-4 + 8.0 * B * H * Dk * Dv * 6 / 2.5e12) > 18:
        return None
    s = prepare(case, seed)
    every = torch.arange(n, device="cuda").expand(B, n)
    if c["op"] == "commit":
        return dict(state=_steps(s, s["index"].long() if s["index"] is not None else every, False)[1])
    if c["op"] == "forward":
        out, S = _steps(s, every, True)
        return dict(out=out, state=S)
    if s["parents"] is None:
        return dict(out=_steps(s, every, True)[0])
    # a tree: every node's own state from its parent's, a request at a time
    out = torch.zeros((B, n, H, Dv), dtype=torch.float64, device="cuda")
    head = torch.arange(H, device="cuda") // c["G"]
    parents = s["parents"].tolist()
    counts = [n] * B if s["counts"] is None else s["counts"].tolist()
    for b in range(B):
        S0 = s["state"][int(s["slots"][b])].double()
        made = []
        for i in range(counts[b]):
            before = S0 if parents[b][i] < 0 else made[parents[b][i]]
            k, v = s["k"][b, i, head].double(), s["v"][b, i].double()
            S = torch.exp(s["decay"][b, i].double())[:, None, None] * before + k[:, :, None] * v[:, None, :]
            made.append(S)
            out[b, i] = (s["q"][b, i, head].double()[:, :, None] * S).sum(1) * Dk ** -0.5
    return dict(out=out)
