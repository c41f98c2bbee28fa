"""Linear attention over states on the GPU against the recurrence in 64 bits."""
import pytest
import torch

import state_oracle as ref

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
# What the tensor-core kernels' operands leave out of S, of the pairs' weights and of the keys, each the sum of two pieces of the
# rows' type.  In bf16 the first leaves out at most half of its step, 2^(e - 8) of a value from 2^e on; that lies in the binade
# below, so the second, of 8 bits too, leaves out at most half of 2^(e - 9 - 7): 2^-17 of the value (fp16: 2^-23).  An output
# passes S's pieces, and S is made of keys' pieces: twice that.
# Three pieces hold all of a bf16 operand's digits now; tests/test_gpu_state_digits.py holds every kernel to what it reaches, without this.
PIECES = 2.0 ** -16


@pytest.fixture(scope="module")
def api():
    from speculative_decoding_verification_02_gb300 import api, build
    build.build()
    torch.cuda.set_device(0)
    return api


class Rows:
    """Inputs of a call on the host (64-bit views of what the GPU gets) and on the GPU."""

    def __init__(self, B, n, Hk, G, Dk, Dv, dtype, seed, slots=None, remember=4.0):
        g = torch.Generator().manual_seed(seed)
        H = Hk * G
        self.B, self.n, self.H, self.Dk, self.Dv, self.dtype = B, n, H, Dk, Dv, dtype
        self.q = torch.randn(B, n, Hk, Dk, generator=g).to(dtype)
        self.k = (torch.randn(B, n, Hk, Dk, generator=g) / Dk ** 0.5).to(dtype)
        self.v = torch.randn(B, n, H, Dv, generator=g).to(dtype)
        rate = torch.exp(-remember * torch.rand(1, 1, H, generator=g))
        self.g = -rate * 2 * torch.rand(B, n, H, generator=g)
        self.pool = torch.randn(slots or B, H, Dk, Dv, generator=g)

    def gpu(self, *names):
        return [getattr(self, x).cuda() for x in names]

    def want(self, b, S0, rows=None, parents=None, scale=None):
        at = list(range(self.n)) if rows is None else rows
        return ref.walk(self.q[b, at], self.k[b, at], self.v[b, at], self.g[b, at], S0, parents or ref.chain(len(at)),
                        self.Dk ** -0.5 if scale is None else scale)

    def zeros(self):
        return torch.zeros(self.H, self.Dk, self.Dv)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


SHAPES = [(128, 128, 2, 3, BF), (64, 64, 3, 1, HF), (128, 64, 2, 1, HF), (64, 128, 1, 2, BF), (16, 16, 1, 1, BF), (80, 48, 2, 1, HF),
          (256, 256, 1, 1, BF), (192, 112, 1, 2, HF), (112, 240, 1, 1, BF), (128, 256, 1, 1, HF)]


@pytest.mark.parametrize("Dk,Dv,Hk,G,dtype", SHAPES)
@pytest.mark.parametrize("n,counts", [(1, None), (2, [0, 2, 1]), (7, None), (16, [16, 3, 0]), (17, None), (40, [33, 40, 1]), (64, None),
                                      (65, [65, 64, 63]), (200, [200, 1, 129])])
def test_forward(api, Dk, Dv, Hk, G, dtype, n, counts):
    r = Rows(3, n, Hk, G, Dk, Dv, dtype, 100 + n, slots=5)
    slots, to = [4, -1, 2], [1, 0, 2]
    pool = r.pool.cuda()
    dst = torch.full((3, r.H, Dk, Dv), 7.0, device="cuda")
    o = api.spec_state_forward(*r.gpu("q", "k", "v", "g"), pool, slots=i32(slots), dst=dst, dst_slots=i32(to),
                               counts=None if counts is None else i32(counts))
    assert o["status"].tolist() == [0, 0, 0] and torch.equal(pool.cpu(), r.pool)
    for b in range(3):
        m = n if counts is None else counts[b]
        outs, last = r.want(b, r.pool[slots[b]] if slots[b] >= 0 else r.zeros(), list(range(m)))
        ref.check_out(o["out"][b, :m], outs, Dk, n, dtype, PIECES)
        assert not o["out"][b, m:].any()
        ref.check_state(dst[to[b]], last, Dk, n, PIECES)


@pytest.mark.parametrize("n", [1, 5, 100, 300])
def test_forward_in_place(api, n):
    """In place, a request without a state to read refused there, the other slots left alone."""
    r = Rows(2, n, 2, 2, 128, 128, BF, 7, slots=6)
    pool = r.pool.cuda()
    api.spec_state_forward(*r.gpu("q", "k", "v", "g"), pool, slots=i32([5, 1]))
    for b, s in enumerate((5, 1)):
        ref.check_state(pool[s], r.want(b, r.pool[s])[1], 128, n, PIECES)
    for s in (0, 2, 3, 4):
        assert torch.equal(pool[s].cpu(), r.pool[s])


@pytest.mark.parametrize("Dk,Dv,Hk,G,dtype", [(128, 128, 1, 2, BF), (64, 64, 1, 1, HF), (128, 64, 2, 1, HF), (112, 240, 1, 1, BF)])
@pytest.mark.parametrize("n,counts", [(1000, None), (1300, [1300, 70, 0]), (2111, [520, 2111, 1])])
def test_forward_in_segments(api, Dk, Dv, Hk, G, dtype, n, counts):
    """Long prompts of few heads, which several CTAs share: behind a state and from none, in place and not."""
    r = Rows(3, n, Hk, G, Dk, Dv, dtype, 600 + n, slots=4, remember=7.0)
    slots = [2, -1, 0]
    pool, dst = r.pool.cuda(), torch.full((3, r.H, Dk, Dv), 7.0, device="cuda")
    args, c = r.gpu("q", "k", "v", "g"), None if counts is None else i32(counts)
    o = api.spec_state_forward(*args, pool, slots=i32(slots), dst=dst, counts=c)
    assert o["status"].tolist() == [0, 0, 0] and torch.equal(pool.cpu(), r.pool)
    for b in range(3):
        m = n if counts is None else counts[b]
        outs, last = r.want(b, r.pool[slots[b]] if slots[b] >= 0 else r.zeros(), list(range(m)))
        ref.check_out(o["out"][b, :m], outs, Dk, n, dtype, PIECES)
        assert not o["out"][b, m:].any()
        ref.check_state(dst[b], last, Dk, n, PIECES)
    again = api.spec_state_forward(*args, pool, slots=i32([2, 1, 0]), counts=c)
    assert torch.equal(again["out"][0], o["out"][0]) and torch.equal(again["out"][2], o["out"][2]) and torch.equal(pool[[2, 0]], dst[[0, 2]])
    pool.copy_(r.pool)
    bad = api.spec_state_forward(*args, pool, slots=i32([1, 9, 3]), counts=i32([n, n, n + 1]))
    assert bad["status"].tolist() == [0, api.STATUS_BAD_SLOT, api.STATUS_BAD_LENGTH] and not bad["out"][1:].any()
    assert torch.equal(pool[3].cpu(), r.pool[3])


def test_forward_in_parts_of_segments(api):
    """As many heads as leave the launch before the main one several CTAs to a segment."""
    n = 3001
    r = Rows(1, n, 16, 3, 32, 16, BF, 40, remember=7.0)
    pool = r.pool.cuda()
    o = api.spec_state_forward(*r.gpu("q", "k", "v", "g"), pool)
    outs, last = r.want(0, r.pool[0])
    ref.check_out(o["out"][0], outs, 32, n, BF, PIECES)
    ref.check_state(pool[0], last, 32, n, PIECES)


@pytest.mark.parametrize("n", [3, 90])
def test_forward_from_nothing_and_unwritten(api, n):
    r = Rows(2, n, 2, 1, 128, 128, BF, 8)
    args = r.gpu("q", "k", "v", "g")
    dst = torch.full((4, 2, 128, 128), 3.0, device="cuda")
    o = api.spec_state_forward(*args, None, dst=dst, dst_slots=i32([3, 1]), scale=0.7)
    for b, s in enumerate((3, 1)):
        outs, last = r.want(b, r.zeros(), scale=0.7)
        ref.check_out(o["out"][b], outs, 128, n, BF, PIECES)
        ref.check_state(dst[s], last, 128, n, PIECES)
    assert bool((dst[0] == 3).all()) and bool((dst[2] == 3).all())
    again = api.spec_state_forward(*args, None, write=False, scale=0.7)
    assert torch.equal(again["out"], o["out"])
    pool = r.pool.cuda()
    o = api.spec_state_forward(*args, pool, write=False)
    for b in range(2):
        ref.check_out(o["out"][b], r.want(b, r.pool[b])[0], 128, n, BF, PIECES)
    assert torch.equal(pool.cpu(), r.pool)
    with pytest.raises(ValueError):
        api.spec_state_forward(*args, None)


@pytest.mark.parametrize("n", [4, 150])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_forward_strides(api, n, dtype):
    """Rows as slices of one projection, a decay for each head alone, outputs into a wider tensor, pools with room between slots."""
    B, Hk, G, D = 2, 2, 2, 64
    r = Rows(B, n, Hk, G, D, D, dtype, 9)
    H = Hk * G
    packed = torch.zeros(B, n, 2 * Hk + H, D, dtype=dtype, device="cuda")
    q, k, v = packed[:, :, :Hk], packed[:, :, Hk:2 * Hk], packed[:, :, 2 * Hk:]
    q.copy_(r.q), k.copy_(r.k), v.copy_(r.v)
    r.g = r.g[:1, :1].expand(B, n, H)
    g = r.g[0, 0].cuda().expand(B, n, H)
    assert g.stride() == (0, 0, 1)
    room = torch.full((B, H * D * D + 12), 5.0, device="cuda")
    pool = torch.as_strided(room, (B, H, D, D), (H * D * D + 12, D * D, D, 1))
    pool.copy_(r.pool)
    wide = torch.full((B, H, n, 2, D), 9.0, dtype=dtype, device="cuda")
    o = dict(out=wide[:, :, :, 1].transpose(1, 2), status=i32([9, 9]))
    api.spec_state_forward(q, k, v, g, pool, out=o)
    for b in range(B):
        outs, last = r.want(b, r.pool[b])
        ref.check_out(o["out"][b], outs, D, n, dtype, PIECES)
        ref.check_state(pool[b], last, D, n, PIECES)
    assert bool((wide[:, :, :, 0] == 9).all()) and bool((room[:, H * D * D:] == 5).all())


@pytest.mark.parametrize("n", [3, 70])
@pytest.mark.parametrize("offset", [1, 4])
def test_forward_unaligned_rows(api, n, offset):
    r = Rows(1, n, 1, 2, 128, 64, BF, 10)
    flat = torch.zeros(8192 * n, dtype=BF, device="cuda")
    at, views = offset, []
    for x in (r.q, r.k, r.v):
        views.append(flat[at:at + x.numel()].view(x.shape))
        views[-1].copy_(x)
        at += x.numel()
    out = flat[at + 1:at + 1 + r.v.numel()].view(r.v.shape)
    pool = r.pool.cuda()
    api.spec_state_forward(*views, r.g.cuda(), pool, counts=i32([n - 1]), out=dict(out=out, status=i32([0])))
    outs, last = r.want(0, r.pool[0], list(range(n - 1)))
    ref.check_out(out[0, :n - 1], outs, 128, n, BF, PIECES)
    assert not out[0, n - 1].any()
    ref.check_state(pool[0], last, 128, n, PIECES)


@pytest.mark.parametrize("n", [2, 12, 100])
def test_wrong_requests(api, n):
    """Bad counts and slots among good requests: theirs alone are refused, their states left as they were, their rows 0."""
    r = Rows(6, n, 1, 2, 128, 128, BF, 11, slots=6)
    pool = r.pool.cuda()
    slots, counts = [0, 1, 6, 3, -2, -1], [n, n + 1, n, -1, n, n]
    out = torch.full(r.v.shape, 3.0, dtype=BF, device="cuda")
    o = api.spec_state_forward(*r.gpu("q", "k", "v", "g"), pool, slots=i32(slots), counts=i32(counts), out=dict(out=out, status=i32([9] * 6)))
    assert o["status"].tolist() == [0, api.STATUS_BAD_LENGTH, api.STATUS_BAD_SLOT, api.STATUS_BAD_LENGTH, api.STATUS_BAD_SLOT,
                                    api.STATUS_BAD_SLOT]  # (the last: nothing to read is a state of zeros, but there is none to write)
    ref.check_state(pool[0], r.want(0, r.pool[0])[1], 128, n, PIECES)
    assert torch.equal(pool[1:].cpu(), r.pool[1:])
    assert not out[1:].any()
    ref.check_out(out[0], r.want(0, r.pool[0])[0], 128, n, BF, PIECES)


@pytest.mark.parametrize("n", [20, 200])
def test_later_rows_have_no_part(api, n):
    """Infinities and NaN in the rows of a token, or behind a request's count, leave the rows before as they are."""
    r = Rows(2, n, 1, 1, 128, 128, BF, 12)
    args = r.gpu("q", "k", "v", "g")
    clean = api.spec_state_forward(*args, r.pool.cuda(), write=False)["out"]
    for at in (1, 14, n // 2 + 3, n - 1):
        for x in (args[2], args[1], args[0]):
            spoilt = [y.clone() for y in args]
            i = [j for j in range(3) if args[j] is x][0]
            spoilt[i][0, at, 0, 5], spoilt[i][0, at, 0, 9] = float("inf"), float("nan")
            got = api.spec_state_forward(*spoilt, r.pool.cuda(), write=False)["out"]
            outs = r.want(0, r.pool[0], list(range(at)))[0]
            ref.check_out(got[0, :at], outs, 128, n, BF, PIECES)
            assert torch.equal(got[1], clean[1])
            assert bool(got[0, at].isnan().any())
        for y in spoilt[:3]:
            y[0, at:] = float("nan")
        spoilt[3][0, at:] = float("nan")
        pool = r.pool.cuda()
        got = api.spec_state_forward(*spoilt, pool, counts=i32([at, n]))["out"]
        outs, last = r.want(0, r.pool[0], list(range(at)))
        ref.check_out(got[0, :at], outs, 128, n, BF, PIECES)
        ref.check_state(pool[0], last, 128, n, PIECES)
        assert not got[0, at:].any()


@pytest.mark.parametrize("n", [9, 150])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_decays_at_their_ends(api, n, dtype):
    """Nothing forgotten, everything forgotten (-inf, and sums far below the least float), and growth."""
    r = Rows(1, n, 5, 1, 128, 128, dtype, 13)
    r.g[..., 0] = 0.0
    r.g[..., 1] = -300.0
    r.g[..., 2] = torch.where(torch.arange(n) % 5 == 2, -float("inf"), r.g[0, :, 2])
    r.g[..., 3] = torch.where(torch.arange(n) % 7 == 3, -1e30, -1e-3)
    r.g[..., 4] = 0.02
    pool = r.pool.cuda()
    o = api.spec_state_forward(*r.gpu("q", "k", "v", "g"), pool)
    outs, last = r.want(0, r.pool[0])
    ref.check_out(o["out"][0], outs, 128, n, dtype, PIECES)
    ref.check_state(pool[0], last, 128, n, PIECES)


@pytest.mark.parametrize("size", [1e-6, 1e4])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_values_of_every_size(api, size, dtype):
    """Heads whose keys, values and states lie far from 1, rows of very different sizes among them."""
    n = 140
    r = Rows(1, n, 2, 1, 128, 128, dtype, 14)
    top = 6e4 if dtype == HF else 1e30
    r.k = (r.k.float() * size * torch.exp(2 * torch.randn(1, n, 2, 1, generator=torch.Generator().manual_seed(1)))).clamp(-top, top).to(dtype)
    r.v = (r.v.float() * torch.exp(2 * torch.randn(1, n, 2, 1, generator=torch.Generator().manual_seed(2)))).to(dtype)
    r.pool *= size
    pool = r.pool.cuda()
    scale = 1e-5 if size > 1 else 1.0
    o = api.spec_state_forward(*r.gpu("q", "k", "v", "g"), pool, scale=scale)
    outs, last = r.want(0, r.pool[0], scale=scale)
    ref.check_out(o["out"][0], outs, 128, n, dtype, PIECES)
    ref.check_state(pool[0], last, 128, n, PIECES)


def test_nothing_to_do(api):
    r = Rows(2, 4, 1, 1, 64, 64, BF, 15)
    q, k, v, g = r.gpu("q", "k", "v", "g")
    pool, dst = r.pool.cuda(), torch.zeros(2, 1, 64, 64, device="cuda")
    o = api.spec_state_forward(q[:, :0], k[:, :0], v[:, :0], g[:, :0], pool, dst=dst)  # no tokens: the states as they are
    assert o["out"].shape == (2, 0, 1, 64) and o["status"].tolist() == [0, 0] and torch.equal(dst, pool)
    dst.zero_()
    o = api.spec_state_forward(q, k, v, g, pool, dst=dst, counts=i32([0, 0]))
    assert not o["out"].any() and torch.equal(dst, pool)
    dst.zero_()
    api.spec_state_commit(k, v, g, pool, dst=dst, counts=i32([0, 0]))
    assert torch.equal(dst, pool)
    o = api.spec_state_attend(q, k, v, g, pool, n_query=i32([0, 0]))
    assert not o["out"].any() and o["status"].tolist() == [0, 0]
    o = api.spec_state_attend(q[:0], k[:0], v[:0], g[:0], pool)
    assert o["out"].shape == (0, 4, 1, 64)


@pytest.mark.parametrize("Dk,Dv,Hk,G,dtype", [(128, 128, 8, 3, BF), (64, 64, 20, 1, HF), (112, 48, 10, 2, BF), (16, 128, 10, 1, HF), (128, 80, 7, 2, HF)])
@pytest.mark.parametrize("n", [1, 5, 16])
def test_many_requests(api, Dk, Dv, Hk, G, dtype, n):
    """Enough (request, head)s that a CTA takes several: ragged, wrong ones among them, slots in any order, in place and not."""
    B = 64
    r = Rows(B, n, Hk, G, Dk, Dv, dtype, 500 + n, slots=B + 3)
    g = torch.Generator().manual_seed(n)
    slots = torch.randperm(B + 3, generator=g)[:B].tolist()
    counts = torch.randint(0, n + 1, (B,), generator=g).tolist()
    slots[7], slots[20], counts[30] = -1, B + 3, n + 1
    pool, dst = r.pool.cuda(), torch.full((B, r.H, Dk, Dv), 3.0, device="cuda")
    out = torch.full(r.v.shape, 5.0, dtype=dtype, device="cuda")
    o = api.spec_state_forward(*r.gpu("q", "k", "v", "g"), pool, slots=i32(slots), dst=dst, counts=i32(counts), out=dict(out=out, status=i32([9] * B)))
    bad = {20: api.STATUS_BAD_SLOT, 30: api.STATUS_BAD_LENGTH}
    assert o["status"].tolist() == [bad.get(b, 0) for b in range(B)]
    d = api.spec_state_attend(*r.gpu("q", "k", "v", "g"), pool, slots=i32(slots), n_query=i32(counts))
    assert d["status"].tolist() == o["status"].tolist()  # (which may be another kernel's work: the same to their bounds)
    for b in list(range(0, B, 9)) + [7, 20, 30, B - 1]:
        if b in bad:
            assert not out[b].any() and not d["out"][b].any() and bool((dst[b] == 3).all())
            continue
        outs, last = r.want(b, r.pool[slots[b]] if slots[b] >= 0 else r.zeros(), list(range(counts[b])))
        ref.check_out(d["out"][b, :counts[b]], outs, Dk, n, dtype, PIECES)
        assert not d["out"][b, counts[b]:].any()
        ref.check_out(out[b, :counts[b]], outs, Dk, n, dtype)
        assert not out[b, counts[b]:].any()
        ref.check_state(dst[b], last, Dk, n)
    rows = max(1, n - 1)
    index = torch.stack([torch.randperm(n, generator=g)[:rows].sort().values for _ in range(B)]).to(torch.int32)
    counts = torch.randint(0, rows + 1, (B,), generator=g).tolist()
    slots[7], slots[20], counts[9] = next(s for s in range(B + 3) if s not in slots), next(s for s in range(B + 2, -1, -1) if s not in slots), rows
    index[9, 0] = n
    was = pool.clone()
    o = api.spec_state_commit(*r.gpu("k", "v", "g"), pool, slots=i32(slots), counts=i32(counts), index=index.cuda())
    assert o["status"].tolist() == [api.STATUS_BAD_INDEX if b == 9 else 0 for b in range(B)]
    assert torch.equal(pool[slots[9]], was[slots[9]])
    for b in list(range(0, B, 8)) + [7, 20]:
        ref.check_state(pool[slots[b]], r.want(b, r.pool[slots[b]], index[b, :counts[b]].tolist())[1], Dk, n)
    for s in set(range(B + 3)) - set(slots):
        assert torch.equal(pool[s], was[s])


@pytest.mark.parametrize("n", [3, 90])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-38, 3e30])
def test_scales(api, n, scale):
    """Scales that are zero, negative, or far from 1 (the values so that the outputs stay within their type)."""
    r = Rows(1, n, 1, 2, 64, 64, BF, 35)
    if scale > 1:
        r.q = (r.q.float() * 1e-30).to(BF)
    o = api.spec_state_forward(*r.gpu("q", "k", "v", "g"), r.pool.cuda(), write=False, scale=scale)
    ref.check_out(o["out"][0], [x if i == 0 else x.abs() for i, x in enumerate(r.want(0, r.pool[0], scale=scale)[0])], 64, n, BF, PIECES)


def test_very_many_requests(api):
    """More requests than are put in order of their lengths."""
    B, n = 4100, 40
    r = Rows(1, n, 1, 1, 16, 16, BF, 36)
    q, k, v, g = (x.cuda().expand(B, *x.shape[1:]).contiguous() for x in (r.q, r.k, r.v, r.g))
    counts = torch.arange(B) % (n + 1)
    pool = torch.zeros(B, 1, 16, 16, device="cuda")
    o = api.spec_state_forward(q, k, v, g, None, dst=pool, counts=counts.int().cuda())
    outs, _ = r.want(0, r.zeros())
    for b in (0, 1, 40, 41, 2000, B - 1):
        m = int(counts[b])
        ref.check_out(o["out"][b, :m], [x[:m] for x in outs], 16, n, BF, PIECES)
        ref.check_state(pool[b], r.want(0, r.zeros(), list(range(m)))[1], 16, n, PIECES)
        assert not o["out"][b, m:].any()
    assert not o["status"].any()


# ------------------------------------------------------------------ drafted rows

def random_tree(n, seed, reach=10, depth=64):
    g = torch.Generator().manual_seed(seed)
    parents, d = [-1], [0]
    for i in range(1, n):
        may = [j for j in range(max(0, i - reach), i) if d[j] < depth] or [0]
        parents.append(may[int(torch.randint(len(may), (1,), generator=g))])
        d.append(d[parents[-1]] + 1)
    return parents


@pytest.mark.parametrize("Dk,Dv,Hk,G,dtype", SHAPES)
@pytest.mark.parametrize("n,rows", [(1, None), (9, [9, 1, 0]), (33, None), (60, [60, 17, 41]), (64, None), (100, [100, 65, 64])])
@pytest.mark.parametrize("tree", [False, True])
def test_attend(api, Dk, Dv, Hk, G, dtype, n, rows, tree):
    r = Rows(3, n, Hk, G, Dk, Dv, dtype, 200 + n, slots=4)
    slots = [3, 0, -1]
    pool = r.pool.cuda()
    trees = [random_tree(n, 300 + b) for b in range(3)]
    par = None
    if tree:
        par = i32(trees)
        for b in range(3):
            par[b, n if rows is None else rows[b]:] = -7  # not read
    o = api.spec_state_attend(*r.gpu("q", "k", "v", "g"), pool, slots=i32(slots), parents=par, n_query=None if rows is None else i32(rows))
    assert o["status"].tolist() == [0, 0, 0] and torch.equal(pool.cpu(), r.pool)
    for b in range(3):
        m = n if rows is None else rows[b]
        outs = r.want(b, r.pool[slots[b]] if slots[b] >= 0 else r.zeros(), list(range(m)), trees[b][:m] if tree else None)[0]
        ref.check_out(o["out"][b, :m], outs, Dk, n, dtype, PIECES)
        assert not o["out"][b, m:].any()


@pytest.mark.parametrize("n", [60, 130])
def test_attend_wrong_trees(api, n):
    r = Rows(6, n, 1, 1, 128, 128, BF, 16)
    trees = [random_tree(n, b) for b in range(6)]
    trees[1][0] = 0
    trees[2][5] = 5
    trees[3][7] = -1
    trees[4] = ref.chain(n) if n > 65 else trees[4][:9] + [n + 3] + trees[4][10:]  # too deep; a parent that does not exist
    o = api.spec_state_attend(*r.gpu("q", "k", "v", "g"), r.pool.cuda(), parents=i32(trees))
    assert o["status"].tolist() == [0] + [api.STATUS_BAD_TREE] * 4 + [0]
    assert not o["out"][1:5].any()
    for b in (0, 5):
        ref.check_out(o["out"][b], r.want(b, r.pool[b], parents=trees[b])[0], 128, n, BF, PIECES)


def test_attend_deepest_tree_and_spoilt_nodes(api):
    """A path of 64 edges; infinities and NaN in a node leave the nodes that do not follow it as they are."""
    n = 64
    r = Rows(1, n, 2, 2, 128, 128, BF, 17)
    q, k, v, g = r.gpu("q", "k", "v", "g")
    pool = r.pool.cuda()
    o = api.spec_state_attend(q, k, v, g, pool, parents=i32([ref.chain(n)]))
    ref.check_out(o["out"][0], r.want(0, r.pool[0])[0], 128, n, BF, PIECES)
    parents = random_tree(n, 5)
    par = i32([parents])
    for x in (k, v):
        keep = x[0, 20].clone()
        x[0, 20, 0, 3], x[0, 20, 0, 8] = float("nan"), float("inf")
        o = api.spec_state_attend(q, k, v, g, pool, parents=par)
        x[0, 20] = keep
        below = {20}
        for i in range(21, n):
            if parents[i] in below:
                below.add(i)
        clear = [i for i in range(n) if i not in below]
        outs = r.want(0, r.pool[0], parents=parents)[0]
        ref.check_out(o["out"][0, clear], [y[clear] for y in outs], 128, n, BF, PIECES)
        assert bool(o["out"][0, 20].isnan().any())


# ------------------------------------------------------------------ accepted rows

@pytest.mark.parametrize("Dk,Dv,Hk,G,dtype", SHAPES)
@pytest.mark.parametrize("n,rows", [(5, None), (9, 9), (60, 7), (60, 60)])
def test_commit(api, Dk, Dv, Hk, G, dtype, n, rows):
    r = Rows(3, n, Hk, G, Dk, Dv, dtype, 400 + n, slots=4)
    g = torch.Generator().manual_seed(n)
    index = None if rows is None else torch.stack([torch.randperm(n, generator=g)[:rows].sort().values for _ in range(3)]).to(torch.int32)
    counts = [rows or n, 0, 1]
    pool, dst = r.pool.cuda(), torch.zeros(3, r.H, Dk, Dv, device="cuda")
    if index is not None:
        index[2, 1:] = -1  # the padding of path_nodes
    o = api.spec_state_commit(*r.gpu("k", "v", "g"), pool, slots=i32([2, 0, 3]), dst=dst, counts=i32(counts),
                              index=None if index is None else index.cuda())
    assert o["status"].tolist() == [0, 0, 0]
    for b, s in enumerate((2, 0, 3)):
        at = list(range(counts[b])) if index is None else index[b, :counts[b]].tolist()
        ref.check_state(dst[b], r.want(b, r.pool[s], at)[1], Dk, n)
    api.spec_state_commit(*r.gpu("k", "v", "g"), pool, slots=i32([2, 0, 3]), counts=i32(counts), index=None if index is None else index.cuda())
    assert torch.equal(pool[[2, 0, 3]], dst) and torch.equal(pool[1].cpu(), r.pool[1])


def test_commit_wrong_requests(api):
    r = Rows(5, 12, 1, 1, 64, 128, BF, 18)
    pool = r.pool.cuda()
    index = i32([[0, 3, 5]] * 5)
    index[1, 1], index[2, 2], index[3, 2] = 12, -1, -1
    o = api.spec_state_commit(*r.gpu("k", "v", "g"), pool, counts=i32([3, 3, 3, 2, 4]), index=index)
    assert o["status"].tolist() == [0, api.STATUS_BAD_INDEX, api.STATUS_BAD_INDEX, 0, api.STATUS_BAD_LENGTH]
    for b in (1, 2, 4):
        assert torch.equal(pool[b].cpu(), r.pool[b])
    for b, m in ((0, 3), (3, 2)):
        ref.check_state(pool[b], r.want(b, r.pool[b], [0, 3, 5][:m])[1], 64, 12)


# ------------------------------------------------------------------ as they are used

def test_a_round_of_each(api):
    """A prompt, then rounds of drafting: the tree's rows over the state, the accepted path committed; the outputs and the state
    are those of the accepted tokens alone, one after another."""
    B, n, N, Hk, G, D = 2, 70, 20, 2, 2, 128
    p = Rows(B, n, Hk, G, D, D, BF, 19)
    pool = api.spec_state_new(B, Hk * G, D, D)
    api.spec_state_forward(*p.gpu("q", "k", "v", "g"), None, dst=pool)
    rows = [[[x[b]] for x in (p.q, p.k, p.v, p.g)] for b in range(B)]  # all accepted rows of a request
    for turn in range(3):
        d = Rows(B, N, Hk, G, D, D, BF, 20 + turn)
        trees = [random_tree(N, 40 + turn + b, reach=4) for b in range(B)]
        o = api.spec_state_attend(*d.gpu("q", "k", "v", "g"), pool, parents=i32(trees))
        path = torch.full((B, N + 1), -1, dtype=torch.int32)
        counts = []
        for b in range(B):
            nodes, at = [], N - 1 - b
            while at >= 0:
                nodes.append(at)
                at = trees[b][at]
            nodes = nodes[::-1]
            path[b, :len(nodes)] = torch.tensor(nodes)
            counts.append(len(nodes))
            for x, y in zip(rows[b], (d.q, d.k, d.v, d.g)):
                x.append(y[b, nodes])
            every = [torch.cat(x) for x in rows[b]]
            outs, _ = ref.walk(*every, torch.zeros(Hk * G, D, D), ref.chain(len(every[0])), D ** -0.5)
            ref.check_out(o["out"][b, nodes], [y[-len(nodes):] for y in outs], D, len(every[0]), BF, PIECES)
        api.spec_state_commit(*d.gpu("k", "v", "g"), pool, counts=i32(counts), index=path.cuda())
    for b in range(B):
        every = [torch.cat(x) for x in rows[b]]
        _, last = ref.walk(*every, torch.zeros(Hk * G, D, D), ref.chain(len(every[0])), D ** -0.5)
        ref.check_state(pool[b], last, D, len(every[0]), PIECES)


@pytest.mark.parametrize("keep", [12, 40])
def test_with_the_verify_step(api, keep):
    """The layer of a verify step between its tree's rerank and its verdict: sel_parents in, path_nodes and n_emit out."""
    B, N, V, Hk, G, D = 3, 48, 512, 2, 2, 128
    g = torch.Generator().manual_seed(keep)
    trees = torch.tensor([random_tree(N, 60 + b, reach=6, depth=6) for b in range(B)], dtype=torch.int32)
    conf = torch.rand(B, N, generator=g)
    tok = torch.randint(0, V, (B, N), generator=g, dtype=torch.int32)
    tree = api.spec_tree_rerank(trees.cuda(), conf.cuda(), keep, node_tok=tok.cuda())
    d = Rows(B, keep, Hk, G, D, D, BF, 37)
    pool = d.pool.cuda()
    o = api.spec_state_attend(*d.gpu("q", "k", "v", "g"), pool, parents=tree["sel_parents"], n_query=tree["n_sel"])
    assert o["status"].tolist() == [0] * B
    for b in range(B):
        m = int(tree["n_sel"][b])
        ref.check_out(o["out"][b, :m], d.want(b, d.pool[b], list(range(m)), tree["sel_parents"][b, :m].tolist())[0], D, keep, BF, PIECES)
    target = torch.randn(B, keep, V, generator=g)
    for b in range(B):  # a target that wants some path of the tree
        at = keep - 1 - b
        while at > 0:
            p = int(tree["sel_parents"][b, at])
            target[b, p, int(tree["sel_tok"][b, at])] = 50.0
            at = p
    verdict = api.spec_verify_tree(target.cuda(), None, tree["sel_parents"], tree["sel_tok"], torch.zeros(B, keep + 1, device="cuda"), 0.0, 64)
    assert verdict["status"].tolist() == [0] * B and bool((verdict["n_emit"] > 1).any())
    c = api.spec_state_commit(*d.gpu("k", "v", "g"), pool, index=verdict["path_nodes"], counts=verdict["n_emit"])
    assert c["status"].tolist() == [0] * B
    for b in range(B):
        ref.check_state(pool[b], d.want(b, d.pool[b], verdict["path_nodes"][b, :int(verdict["n_emit"][b])].tolist())[1], D, keep)


def test_workspace(api):
    """A call that needs a workspace is refused one that is too small or badly placed, and gives the same with its own."""
    r = Rows(2, 200, 2, 1, 128, 128, BF, 38)
    x = r.gpu("q", "k", "v", "g", "pool")
    want = api.spec_state_forward(*x, write=False)["out"]
    need = api.lib().spec_state_workspace_size(api.OP_STATE_FORWARD, api._state_struct(x[4], None, 2, tuple(x[4].shape[1:]), x[4].device, "s"), 2, 200)
    assert need > 0
    n0 = api.launch_count()
    room = torch.empty(need + 512, dtype=torch.uint8, device="cuda")
    for bad in (room[:need - 256], room[16:]):
        with pytest.raises(api.SpecError, match="workspace"):
            api.spec_state_forward(*x, write=False, ws=bad)
    assert api.launch_count() == n0
    guard = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    assert torch.equal(api.spec_state_forward(*x, write=False, ws=guard[:need])["out"], want)
    assert bool((guard[need:] == 77).all())


@pytest.mark.parametrize("n", [1, 20, 300, 900])
def test_captured_and_replayed(api, n):
    """Two captured calls of different sizes on one stream, replayed in turn over new inputs, against calls outside a graph."""
    a, b = Rows(2, n, 2, 1, 128, 128, BF, 30), Rows(1, n + 130, 2, 1, 128, 128, BF, 31)
    sets = []
    for r in (a, b):
        x = r.gpu("q", "k", "v", "g", "pool")
        dst = torch.zeros_like(x[4])
        o = dict(out=torch.empty_like(x[2]), status=i32([0] * r.B))
        sets.append((x, dst, o))
        ws = torch.empty(max(256, api.lib().spec_state_workspace_size(
            api.OP_STATE_FORWARD, api._state_struct(x[4], None, r.B, tuple(x[4].shape[1:]), x[4].device, "state"), r.B, r.n)),
            dtype=torch.uint8, device="cuda")
        sets[-1] += (ws,)
    graphs = []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for x, dst, o, ws in sets:
        with torch.cuda.stream(s):
            api.spec_state_forward(*x, dst=dst, out=o, ws=ws)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                api.spec_state_forward(*x, dst=dst, out=o, ws=ws)
            graphs.append(g)
    for turn in range(3):
        for (x, dst, o, ws), g, r in zip(sets, graphs, (a, b)):
            fresh = Rows(r.B, r.n, 2, 1, 128, 128, BF, 50 + turn)
            for t, u in zip(x, (fresh.q, fresh.k, fresh.v, fresh.g, fresh.pool)):
                t.copy_(u)
            g.replay()
            torch.cuda.synchronize()
            other = torch.zeros_like(dst)
            w = api.spec_state_forward(*x, dst=other)
            assert torch.equal(w["out"], o["out"]) and torch.equal(other, dst)


def test_on_another_stream(api):
    r = Rows(2, 150, 2, 1, 128, 128, BF, 32)
    args, pool = r.gpu("q", "k", "v", "g"), r.pool.cuda()
    want_pool = pool.clone()
    want = api.spec_state_forward(*args, want_pool)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o = api.spec_state_forward(*args, pool, stream=s)
    d = api.spec_state_attend(*[x[:, :60] for x in args], pool, stream=s)
    c = api.spec_state_commit(*[x[:, :9] for x in args[1:]], pool, stream=s)
    s.synchronize()
    assert torch.equal(o["out"], want["out"])
    d2 = api.spec_state_attend(*[x[:, :60] for x in args], want_pool)
    api.spec_state_commit(*[x[:, :9] for x in args[1:]], want_pool)
    assert torch.equal(d["out"], d2["out"]) and torch.equal(pool, want_pool) and c["status"].tolist() == [0, 0]


def test_same_results_again(api):
    """A call gives the same bits every time, alone and among others, and under spec_trace_repeat (in place too)."""
    r = Rows(3, 333, 2, 2, 128, 128, BF, 33)
    args, pool = r.gpu("q", "k", "v", "g"), r.pool.cuda()
    first = None
    for _ in range(4):
        p = pool.clone()
        o = api.spec_state_forward(*args, p, counts=i32([333, 20, 0]))
        first = first or (o["out"].clone(), p.clone())
        assert torch.equal(o["out"], first[0]) and torch.equal(p, first[1])
    api.trace_enable(True)
    api.trace_repeat(3)
    try:
        p = pool.clone()
        o = api.spec_state_forward(*args, p, counts=i32([333, 20, 0]))
        c = pool.clone()
        api.spec_state_commit(*[x[:, :9] for x in args[1:]], c)
        assert api.trace_collect()
    finally:
        api.trace_repeat(1)
        api.trace_enable(False)
    assert torch.equal(o["out"], first[0]) and torch.equal(p, first[1])
    api.spec_state_commit(*[x[:, :9] for x in args[1:]], pool)
    assert torch.equal(c, pool)


def test_binding_refuses(api):
    r = Rows(2, 4, 1, 2, 64, 64, BF, 34)
    q, k, v, g, pool = r.gpu("q", "k", "v", "g", "pool")
    n0 = api.launch_count()
    for bad in (dict(q=q.float()), dict(k=k.half()), dict(v=v[:, :3]), dict(g=g.double()), dict(g=g[:, :, :1]), dict(q=q[:, :, :, :32]),
                dict(pool=pool[:, :1]), dict(pool=pool.double()), dict(pool=pool.cpu()), dict(v=v.transpose(2, 3))):
        a = dict(q=q, k=k, v=v, g=g, pool=pool)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            api.spec_state_forward(a["q"], a["k"], a["v"], a["g"], a["pool"])
        if "q" not in bad:
            with pytest.raises((TypeError, ValueError)):
                api.spec_state_commit(a["k"], a["v"], a["g"], a["pool"])
    for kw in (dict(slots=torch.zeros(2, dtype=torch.int64, device="cuda")), dict(slots=i32([0])), dict(counts=i32([1])),
               dict(out=dict(out=torch.empty(2, 4, 2, 32, dtype=BF, device="cuda"))), dict(out=dict(out=torch.empty_like(v, dtype=HF))),
               dict(out=dict(out=torch.empty_like(v), status=torch.zeros(2, device="cuda"))), dict(dst=pool[:, :1])):
        with pytest.raises((TypeError, ValueError)):
            api.spec_state_forward(q, k, v, g, pool, **kw)
    for par in (torch.zeros(2, 4, dtype=torch.int64, device="cuda"), i32([[-1, 0, 0]] * 2), i32([[-1] * 2] * 4).T):
        with pytest.raises((TypeError, ValueError)):
            api.spec_state_attend(q, k, v, g, pool, parents=par)
    with pytest.raises(api.SpecError):
        api.spec_state_forward(q, k, v, g, pool, scale=float("nan"))
    assert api.launch_count() == n0


def test_two_host_threads(api):
    """Two host threads on one stream, whose calls share its workspace, and on streams of their own."""
    import threading
    sets = [Rows(2, n, 2, 1, 128, 128, BF, 70 + n).gpu("q", "k", "v", "g", "pool") for n in (130, 700)]
    want = [api.spec_state_forward(*x, write=False)["out"] for x in sets]
    torch.cuda.synchronize()
    for streams in ([torch.cuda.current_stream()] * 2, [torch.cuda.Stream(), torch.cuda.Stream()]):
        got, failed = [[], []], []

        def work(i):
            try:
                for _ in range(20):
                    got[i].append(api.spec_state_forward(*sets[i], write=False, stream=streams[i])["out"])
            except Exception as e:  # noqa: BLE001 (told to the test's own thread)
                failed.append(e)

        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert not failed
        for i in range(2):
            assert len(got[i]) == 20 and all(torch.equal(x, want[i]) for x in got[i])
