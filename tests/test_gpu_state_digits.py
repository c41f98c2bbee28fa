"""How many digits the linear-attention kernels keep, and over which range: each kernel against the recurrence in 64 bits."""
import pytest
import torch

import state_oracle as ref

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
U = ref.U


@pytest.fixture(scope="module")
def api():
    from speculative_decoding_verification_02_gb300 import api, build
    build.build()
    torch.cuda.set_device(0)
    return api


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ what the products take

# Outputs that are differences of two terms next to one another: whatever an operand's pieces leave out stands alone in them.  The
# terms' sums have at most eight addends other than zero (three pieces of each term, the two parts of an output); an accumulator
# that cuts off loses 2^-23 of the largest for each, the factors e^G are off by 2^-22, and a term in two fp16 pieces by 2^-22: 2^-19
# of a term in all.  Two bf16 pieces leave out 2^-18 to 2^-17 of every other term, which 128 columns cannot miss.
NEXT_TO = 2.0 ** -19


def rounded(want, tol, dtype):
    """tol, and the result's own rounding: half a step of a value, or of fp16's subnormals (they lie 2^-24 apart)."""
    return tol + torch.finfo(dtype).eps / 2 * (want.abs() + tol) + (2.0 ** -25 if dtype == HF else 0.0)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,write", [(40, False), (64, False), (64, True), (150, True)])
def test_digits_of_the_state(api, dtype, D, n, write):
    """o = S[a] - S[b], in a lane each: S's digits as the products take them."""
    g = torch.Generator().manual_seed(n + D)
    S = torch.zeros(1, 1, D, D)
    S[0, 0, 5] = 1 + torch.rand(D, generator=g)
    S[0, 0, 9] = S[0, 0, 5] * (1 + 2.0 ** -10 * torch.randn(D, generator=g))
    q = torch.zeros(1, n, 1, D)
    q[..., 5], q[..., 9] = 1, -1
    k = torch.zeros(1, n, 1, D)
    v = torch.randn(1, n, 1, D, generator=g)
    decay = torch.zeros(1, n, 1)
    args = [x.to(dtype).cuda() for x in (q, k, v)] + [decay.cuda(), S.cuda()]
    o = api.spec_state_forward(*args, scale=1.0, write=write)["out"] if write else api.spec_state_attend(*args, scale=1.0)["out"]
    want = (S[0, 0, 5].double() - S[0, 0, 9].double()).expand(n, D)
    tol = NEXT_TO * S[0, 0, 5].double()
    worst = (o[0, :, 0].double().cpu() - want).abs() - rounded(want, tol, dtype)
    assert float(worst.max()) <= 0, float(worst.max())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,write", [(40, False), (64, False), (64, True), (150, True)])
def test_digits_of_the_weights(api, dtype, D, n, write):
    """Rows 2 i and 2 i + 1 hold values v and -v: what an odd row adds of its pair is the difference of two weights."""
    g = torch.Generator().manual_seed(n + D)
    k = torch.zeros(1, n, 1, D)
    k[..., 3] = 1
    q = torch.zeros(1, n, 1, D)
    q[..., 3] = 1.5
    v = torch.randn(1, n, 1, D, generator=g).to(dtype).float()
    v[:, 1::2] = -v[:, 0:n - n % 2:2]
    decay = torch.zeros(1, n, 1)
    decay[:, 1::2, 0] = -2.0 ** -9 * (1 + torch.rand(n // 2, generator=g))
    decay[:, 0::2, 0] = -200.0  # nothing but the pair itself
    args = [x.to(dtype).cuda() for x in (q, k, v)] + [decay.cuda()]
    if write:
        o = api.spec_state_forward(*args, None, dst=torch.zeros(1, 1, D, D, device="cuda"), scale=1.0)["out"]
    else:
        o = api.spec_state_attend(*args, torch.zeros(1, 1, D, D, device="cuda"), scale=1.0)["out"]
    for i in range(1, n, 2):
        w = 1.5 * torch.expm1(decay[0, i].double()) * v[0, i - 1].double()
        tol = NEXT_TO * 1.5 * v[0, i - 1].double().abs() + 2.0 ** -80
        worst = (o[0, i].double().cpu() - w).abs() - rounded(w, tol, dtype)
        assert float(worst.max()) <= 0, (i, float(worst.max()))


# ------------------------------------------------------------------ every kernel

KINDS = ["rows", "blocks", "chunk", "segments", "short", "short_tree", "large_tree", "commit"]
TOKENS = dict(rows=12, blocks=24, chunk=150, segments=600, short=40, short_tree=50, large_tree=100, commit=40)


def random_tree(n, seed, reach=3, depth=60):
    g = torch.Generator().manual_seed(seed)
    parents, d = [-1], [0]
    for i in range(1, n):
        may = [j for j in range(max(0, i - reach), i) if d[j] < depth] or [0]
        parents.append(may[int(torch.randint(len(may), (1,), generator=g))])
        d.append(d[parents[-1]] + 1)
    return parents


class Call:
    """Rows of one request for a kernel: q, k, v, g in the order of its nodes, depth the tokens in front of each."""

    def __init__(self, kind, dtype, D, seed, Hk=1, G=2):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.dtype, self.D, self.n = kind, dtype, D, TOKENS[kind]
        self.tree = kind.endswith("tree")
        self.parents = random_tree(self.n, seed) if self.tree else ref.chain(self.n)
        self.depth = []
        for p in self.parents:
            self.depth.append(0 if p < 0 else self.depth[p] + 1)
        n, H = self.n, Hk * G
        self.q = torch.randn(n, Hk, D, generator=g).to(dtype)
        self.k = (torch.randn(n, Hk, D, generator=g) / D ** 0.5).to(dtype)
        self.v = torch.randn(n, H, D, generator=g).to(dtype)
        self.g = -0.3 * torch.rand(n, H, generator=g)
        self.S0 = torch.randn(H, D, D, generator=g)
        self.scale = D ** -0.5

    def run(self, api):
        """-> out [n, H, D] or None, the state after or None"""
        q, k, v, g = (x[None].cuda() for x in (self.q, self.k, self.v, self.g))
        pool = self.S0[None].cuda()
        if self.kind == "commit":
            o, out = api.spec_state_commit(k, v, g, pool), None
        elif self.kind.startswith("short") or self.tree:
            o = api.spec_state_attend(q, k, v, g, pool, parents=i32([self.parents]) if self.tree else None)
            out, pool = o["out"][0], None
        elif self.kind == "blocks":  # rows that start off 16-byte boundaries: the kernel for a few rows, block after block
            room = [torch.zeros(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape) for x in (q, k, v)]
            for x, y in zip(room, (q, k, v)):
                x.copy_(y)
            o = api.spec_state_forward(*room, g, pool)
            out = o["out"][0]
        else:
            o = api.spec_state_forward(q, k, v, g, pool)
            out = o["out"][0]
        assert o["status"].tolist() == [0]
        return out, None if pool is None else pool[0]

    def want(self):
        g = torch.where(self.g < -120, -float("inf"), self.g.double())  # such a factor is 0
        return ref.walk(self.q, self.k, self.v, g, self.S0, self.parents, self.scale)

    def check(self, api):
        out, state = self.run(api)
        outs, last = self.want()
        if out is not None:
            ref.check_out(out, outs, self.D, self.n, self.dtype)
        if state is not None:
            ref.check_state(state, last, self.n, self.n)


# The states on the whole, in the root of their squares.  A token's term: its factor e^G (2^-22), K' exactly in three bf16 pieces (in
# two fp16 pieces, 2^-23 of the chunk's largest), the products' sum, which cuts off 2^-23 of itself at each of its last four steps
# (the steps before add pieces of 2^-8 of it), and one rounded addition for each block that it stays in, whose errors add up as the
# root of their number (150 tokens: 3 chunks or 10 blocks; 600: 10, joined once more): 2^-20 = 9.5e-7.  Two pieces of K' in bf16
# leave out 2^-18 of a value in the root of squares.
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["rows", "blocks", "chunk", "segments", "commit"])
def test_states_on_the_whole(api, kind, D, dtype):
    c = Call(kind, dtype, D, 40, Hk=2)
    c.g *= torch.tensor([1.0, 0.1, 1e-2, 1e-3])
    state = c.run(api)[1].double().cpu()
    run = c.g.double().cumsum(0)
    for h in range(4):
        k = c.k[:, h // 2].double() * torch.exp(run[-1, h] - run[:, h])[:, None]
        last = torch.exp(run[-1, h]) * c.S0[h].double() + k.T @ c.v[:, h].double()
        off = float((state[h] - last).norm() / last.norm())
        assert off <= 2.0 ** -20, (h, off)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kind", KINDS)
def test_ordinary_rows(api, kind, dtype):
    """The bounds of 32-bit sums, with nothing for operands of fewer bits."""
    Call(kind, dtype, 128, 41).check(api)


# ------------------------------------------------------------------ decays

@pytest.mark.parametrize("forget", [-float("inf"), -1e30, -150.0, torch.finfo(torch.float32).min])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kind", KINDS)
def test_forgotten_stays_forgotten(api, kind, dtype, forget):
    """A factor of 0, then growth by e^69: nothing from before comes back, however large it was."""
    c = Call(kind, dtype, 64, 42)
    d = torch.tensor(c.depth) % 70
    c.S0 *= 1e24
    c.q[torch.tensor(c.depth) < 3] = 0  # (fp16 has no such outputs)
    for at, x in ((3, forget), (4, 40.0), (5, 29.0)):
        c.g[d == at] = x
    c.k[(d >= 3) & (d <= 5)] = 0
    c.check(api)
    out, _ = c.run(api)
    if out is not None:  # nothing at all between the reset and the first key after it
        assert not out[((torch.tensor(c.depth) >= 3) & (torch.tensor(c.depth) <= 5)).cuda()].any()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n", [60, 1300, 3001])
def test_forgotten_before_long_growth(api, dtype, n):
    """A reset in one part of a long prompt and growth in all that follow: without keys, a state of zeros and outputs of zeros."""
    c = Call("chunk", dtype, 64, 43)
    c.q, c.k, c.v, c.g = (x[:1].repeat(n, 1, 1) if x.dim() == 3 else x[:1].repeat(n, 1) for x in (c.q, c.k, c.v, c.g))
    c.g[40] = -float("inf")
    c.g[41:] = 0.5
    c.k[40:] = 0
    c.n = n
    out, state = c.run(api)
    assert not state.any() and not out[40:].any()
    assert bool(out[:40].any(-1).all())


@pytest.mark.parametrize("size", [0.0, 1e-30])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kind", KINDS)
def test_a_state_that_grows(api, kind, dtype, size):
    """The state times e^115, which is no fp32 number: zeros stay zeros, a small state becomes what it should."""
    c = Call(kind, dtype, 64, 44)
    c.S0 *= size
    d = torch.tensor(c.depth)
    c.g[d == 0] = 60.0
    c.g[(d > 0) & (d < 12)] = 5.0
    out, state = c.run(api)
    outs, last = c.want()
    if state is not None:
        assert bool(state.isfinite().all())
        ref.check_state(state, last, c.n, c.n)
    if out is not None and dtype == BF:  # (fp16 has no such outputs)
        ref.check_out(out, outs, c.D, c.n, dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("forget,off", [(-87.4, 2.0 ** -18), (-92.0, 2.0 ** -16)])
def test_a_large_state_all_but_forgotten(api, kind, dtype, forget, off):
    """A state next to the largest number times a factor next to the least: ordinary numbers.  e^-92 is 2^-132.7, whose digits end at
    2^-149: half a step is 2^-17.3 of it (e^-87.4, 2^-126.1: 2^-23.9), beside 2^-20 for all else."""
    c = Call(kind, dtype, 64, 47)
    d = torch.tensor(c.depth)
    c.S0 = 1e38 * (1 + torch.rand(c.S0.shape, generator=torch.Generator().manual_seed(1)))
    c.q = (c.q.float() * 2.0 ** -10).to(dtype)
    c.k[:] = 0
    c.g[:] = 0
    c.g[d == 2] = forget
    c.q[d < 2] = 0  # (fp16 has no such outputs)
    out, state = c.run(api)
    outs, last = c.want()
    if state is not None:
        assert bool(((state.double().cpu() - last[0]).abs() <= off * last[0].abs()).all())
    if out is not None:
        tol = off * outs[1]
        assert bool(((out.double().cpu() - outs[0]).abs() <= rounded(outs[0], tol, dtype)).all())


@pytest.mark.parametrize("forget", [-90.0, -float("inf")])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kind", KINDS)
def test_growth_that_is_taken_back(api, kind, dtype, forget):
    """A state that would pass the largest number by e^100 and is forgotten, or comes back to e^10 of itself, within a block."""
    c = Call(kind, dtype, 64, 48)
    d = torch.tensor(c.depth)
    c.S0 *= 1e3
    c.g[d == 0] = 100.0
    c.g[d == 3] = forget
    c.q[d < 3] = 0  # (no such outputs)
    c.v[d == 0] = 0
    out, state = c.run(api)
    outs, last = c.want()
    if state is not None:
        ref.check_state(state, last, c.n, c.n)
    if out is not None and dtype == BF:  # (1e3 e^10 is 2.2e7, an infinity in fp16: no value to compare)
        ref.check_out(out, outs, c.D, c.n, dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_two_tokens_of_growth(api, dtype):
    """A fresh request, two factors of e^50: k_1 v_1 e^50 + k_2 v_2, whichever kernel."""
    for n in (2, 20, 70):
        c = Call("chunk", dtype, 128, 45)
        c.q, c.k, c.v, c.g = c.q[:n], c.k[:n], c.v[:n], torch.zeros(n, 2)
        c.g[:2] = 50.0
        c.n, c.parents = n, ref.chain(n)
        c.S0 *= 0
        _, state = c.run(api)
        ref.check_state(state, c.want()[1], n, n)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n", [8192, 16384])
def test_constant_decays(api, dtype, n):
    """One decay for all tokens, whose rounding is the same for each and adds up over all of them.  A chunk's factor is one fp32
    power, off by 2^-22 at most (two units in the last place): a term that is m chunks old is off by m 2^-22, n / 128 on average;
    and 2^-20 for all else.  A token's decay in units of 2^-25 log 2 would be off by up to 1e-8, n / 2 of them on average."""
    H, D = 8, 64
    g = torch.Generator().manual_seed(n)
    # 0.45 of such a unit beside a whole number of them, tokens that stay for the whole length or a tenth of it
    units = torch.tensor([3.0, 17.0, 40.0, 48.0, 300.0, 1000.0, 4000.0, 10000.0], dtype=torch.float64) + 0.45
    decay = (-units * 2.0 ** -25 * 0.6931471805599453).float()
    k = (torch.randn(1, n, H, D, generator=g) / 8).to(dtype)
    v = torch.randn(1, n, H, D, generator=g).to(dtype)
    pool = torch.zeros(1, H, D, D, device="cuda")
    api.spec_state_forward(k.cuda(), k.cuda(), v.cuda(), decay.cuda().expand(1, n, H), None, dst=pool)
    age = torch.arange(n - 1, -1, -1, dtype=torch.float64)
    for h in range(H):
        w = torch.exp(age * decay[h].double())
        want = (k[0, :, h].double() * w[:, None]).T @ v[0, :, h].double()
        off = float((pool[0, h].double().cpu() - want).norm() / want.norm())
        assert off <= n / 128 * 2.0 ** -22 + 2.0 ** -20, (h, off)


# ------------------------------------------------------------------ fp16's scales, and what is no number

@pytest.mark.parametrize("large", [3e4, float("inf")])
@pytest.mark.parametrize("n", [40, 150, 1300])
def test_small_keys_beside_large_ones(api, n, large):
    """fp16: a chunk's K' has one power of two for all, by its largest e^G k.  A key of 3e4 whose token is all but forgotten (e^-28)
    takes no digits from keys of 1e-3; nor does an infinite key, whose row of the state alone is no number."""
    D = 64
    g = torch.Generator().manual_seed(n)
    k = 1e-3 * torch.randn(1, n, 1, D, generator=g)
    v = torch.randn(1, n, 1, D, generator=g).to(HF)
    decay = torch.full((1, n, 1), -0.01)
    for at in range(2, n, 64):
        k[0, at] = 0
        k[0, at, 0, 0] = large
        decay[0, at + 1] = -28.0
    k = k.to(HF)
    pool = torch.zeros(1, 1, D, D, device="cuda")
    api.spec_state_forward(k.cuda(), k.cuda(), v.cuda(), decay.cuda(), None, dst=pool)
    G = torch.flip(torch.cumsum(torch.flip(decay[0, :, 0].double(), [0]), 0), [0]) - decay[0, :, 0].double()
    want = (k[0, :, 0].double() * torch.exp(G)[:, None]).T @ v[0, :, 0].double()
    got = pool[0, 0].double().cpu()
    # (as in test_states_on_the_whole)
    off = float((got[1:] - want[1:]).norm() / want[1:].norm())
    assert off <= 2.0 ** -20, off
    if large > 1e5:
        assert not got[0].isfinite().any()
    else:
        assert float((got[0] - want[0]).norm() / want[0].norm()) <= 2.0 ** -20


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kind", KINDS)
def test_keys_of_zeros_before_growth(api, kind, dtype):
    """Tokens without keys whose factor is e^60 beside keys whose factor is e^-40: nothing times the one, all digits of the other."""
    c = Call(kind, dtype, 64, 49)
    d = torch.tensor(c.depth)
    c.S0 *= 0
    c.g[d == 4] = -100.0
    c.k[d >= 4] = 0
    c.g[d == 8] = 60.0
    c.check(api)


@pytest.mark.parametrize("n,write", [(5, False), (5, True), (40, False), (64, True), (150, True), (900, True)])
def test_states_next_to_the_largest_number(api, n, write):
    """bf16: values beyond its largest number (3.3895e38), finite in fp32, give finite outputs and come out as they went in."""
    D = 128
    g = torch.Generator().manual_seed(n)
    S = 3.4e38 * (1 - 2e-3 * torch.rand(1, 1, D, D, generator=g)) * torch.where(torch.rand(1, 1, D, D, generator=g) < 0.5, -1.0, 1.0)
    q = torch.zeros(1, n, 1, D)
    for i in range(n):
        q[0, i, 0, i % D] = 2.0 ** -10
    q, k, v = q.to(BF), torch.zeros(1, n, 1, D, dtype=BF), torch.randn(1, n, 1, D, generator=g).to(BF)
    pool = S.cuda()
    args = [x.cuda() for x in (q, k, v)] + [torch.zeros(1, n, 1, device="cuda"), pool]
    o = api.spec_state_forward(*args, scale=1.0) if write else api.spec_state_attend(*args, scale=1.0)
    assert torch.equal(pool.cpu(), S)
    want = torch.stack([S[0, 0, i % D].double() * 2.0 ** -10 for i in range(n)])
    worst = ((o["out"][0, :, 0].double().cpu() - want).abs() / want.abs()).max()
    assert float(worst) <= 2.0 ** -8 + 2.0 ** -20


@pytest.mark.parametrize("where", ["state", "k", "v", "q", "g"])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kind", KINDS)
def test_no_numbers_where_the_recurrence_has_none(api, kind, dtype, value, where):
    """An infinity or a NaN: outputs and states are finite where the recurrence's are, and only there."""
    if where == "g" and value == -float("inf"):
        pytest.skip("a factor of 0 is an ordinary one")
    c = Call(kind, dtype, 64, 46)
    at = min(c.n // 2 + 3, c.n - 2)
    if where == "state":
        c.S0[1, 7, 20] = value
    elif where == "g":
        c.g[at, 1] = value
    else:
        getattr(c, where)[at, 0, 20] = value
    out, state = c.run(api)
    outs, last = c.want()
    if state is not None:
        assert torch.equal(state.isfinite().cpu(), last[0].isfinite())
        ok = last[0].isfinite()
        assert float((state.double().cpu() - last[0])[ok].norm() / last[0][ok].norm()) <= 2.0 ** -18
    if out is not None:
        assert torch.equal(out.isfinite().cpu(), outs[0].isfinite())
        ok = outs[0].isfinite()
        assert float((out.double().cpu() - outs[0])[ok].norm() / outs[0][ok].norm()) <= torch.finfo(dtype).eps


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n", [60, 150, 1300])
def test_rows_before_a_spoilt_one(api, n, dtype, D):
    """Infinities and NaN in a token's k or v: the rows before it as they are without it, prompts cut into segments too."""
    g = torch.Generator().manual_seed(n + D)
    q, k, v = (torch.randn(1, n, 1, D, generator=g).to(dtype) for _ in range(3))
    k = (k.float() / D ** 0.5).to(dtype)
    decay = -0.2 * torch.rand(1, n, 1, generator=g)
    S0 = torch.randn(1, D, D, generator=g)
    outs, _ = ref.walk(q[0], k[0], v[0], decay[0], S0, ref.chain(n), D ** -0.5)
    for at in (1, 37, n - 30, n - 1):
        for name in ("k", "v"):
            x = dict(k=k.clone(), v=v.clone())
            x[name][0, at, 0, 5], x[name][0, at, 0, 40] = float("inf"), float("nan")
            got = api.spec_state_forward(q.cuda(), x["k"].cuda(), x["v"].cuda(), decay.cuda(), S0[None].cuda())["out"]
            ref.check_out(got[0, :at], [y[:at] for y in outs], D, n, dtype)
            assert bool(got[0, at].isnan().any())
