"""The 8-bit cache's operators where rows, keys or buffers are of the odd kind: against their 64-bit definitions."""
import math

import pytest
import torch

import cache_oracle as ref
from test_gpu_cache import BF, HF, api, check_attend, gen, rand_cache, rand_table  # noqa: F401

pytestmark = pytest.mark.gpu

NAN_CODE = 0x7f


def nan_key(cache, table, b, t, P):
    """A NaN in one component of every head's key at position t of request b."""
    cache[0].view(torch.uint8)[int(table[b, t // P]), :, t % P, 3] = NAN_CODE


def check_weights(got, cache, table, q, lse, lens, counts, index, cap, prev):
    want, tol = ref.weights(ref.Cache64(cache, table), q, lse, lens, counts, index, q.shape[3] ** -0.5, cap, prev)
    got = got.cpu().double()
    assert torch.equal(got.isnan(), want.isnan())
    off = (got - want).abs() / tol
    some = ~want.isnan()
    assert bool((off[some] <= 1).all()), float(off[some].max())
    return want


# ------------------------------------------------------------------ rows that add nothing

@pytest.mark.parametrize("D", [64, 80, 128])
@pytest.mark.parametrize("dtype,cap", [(BF, 0.0), (HF, 0.0), (BF, 20.0)])
@pytest.mark.parametrize("N,G", [(5, 2), (40, 4)])
def test_rows_of_no_weight_hold_anything(api, D, dtype, cap, N, G):  # noqa: F811
    """A row whose lse is -inf adds nothing, whatever its q: NaN, infinities, the largest numbers."""
    B, H, P = 3, 2, 32
    lens = [0, 130, 300]
    W = -(-(max(lens) + N) // P)
    cache = rand_cache(api, B * W, H, P, D, 200)
    table = rand_table(B, W, B * W, 201)
    g = gen(202)
    q = torch.randn(B, N, H * G, D, generator=g).to(dtype).cuda()
    lse = (torch.rand(B, N, H * G, generator=g) * 3 + 3).cuda()
    prev = torch.rand(B, H, W * P, generator=g).cuda()
    for row, what in ((1, math.nan), (2, math.inf), (3, -math.inf), (N - 1, torch.finfo(dtype).max)):
        q[:, row, ::2] = what
        lse[:, row, ::2] = -math.inf
    q[1, 0, 1, 7] = math.nan  # one element of one head's row
    lse[1, 0, 1] = -math.inf
    o = api.spec_cache_weights(q, lse, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), prev=prev, softcap=cap)
    assert o["status"].tolist() == [0] * B
    want = check_weights(o["weights"], cache, table, q, lse, lens, [N] * B, None, cap, prev)
    assert not bool(want.isnan().any())


@pytest.mark.parametrize("D", [64, 80, 128])
@pytest.mark.parametrize("dtype,cap", [(BF, 0.0), (HF, 0.0), (HF, 20.0)])
@pytest.mark.parametrize("picked", [False, True])
def test_keys_of_nan_reach_the_rows_that_see_them(api, D, dtype, cap, picked):  # noqa: F811
    """A NaN key: NaN where a row that counts sees it, nothing where none does -- all of lse -inf, or every one before it."""
    B, N, H, G, P = 4, 6, 2, 3, 32
    lens = [70, 200, 33, 270]
    W = -(-(max(lens) + N) // P)
    cache = rand_cache(api, B * W, H, P, D, 203)
    table = rand_table(B, W, B * W, 204)
    g = gen(205)
    q = torch.randn(B, N, H * G, D, generator=g).to(dtype).cuda()
    lse = (torch.rand(B, N, H * G, generator=g) * 3 + 3).cuda()
    prev = torch.rand(B, H, W * P, generator=g).cuda()
    counts, index = [6, 4, 0, 6], None
    if picked:
        index = torch.stack([torch.randperm(N, generator=g) for _ in range(B)]).to(torch.int32).cuda()
    at = torch.arange(N).expand(B, N) if index is None else index.cpu().long()
    nan_key(cache, table, 0, 5, P)  # in the context, seen by rows that count
    nan_key(cache, table, 1, 7, P)
    lse[1] = -math.inf              # ... by none that does
    nan_key(cache, table, 2, 20, P)  # ... by no row at all
    nan_key(cache, table, 3, lens[3] + 2, P)  # a drafted one: rows 2 and later see it and do not count
    for i in range(2, N):
        lse[3, at[3, i]] = -math.inf
    o = api.spec_cache_weights(q, lse, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), prev=prev, softcap=cap, index=index,
                               counts=torch.tensor(counts, dtype=torch.int32, device="cuda"))
    assert o["status"].tolist() == [0] * B
    want = check_weights(o["weights"], cache, table, q, lse, lens, counts, index, cap, prev)
    assert int(want.isnan().sum()) == H and bool(want[0, :, 5].isnan().all())
    for b in (1, 2):  # what was there, to the bit
        T = lens[b] + counts[b]
        assert torch.equal(o["weights"][b, :, :T], prev[b, :, :T])


def test_weights_after_an_attention_of_fewer_rows(api):  # noqa: F811
    """Rows past n_query have lse -inf from the attention, and a q that nothing wrote."""
    B, N, H, G, D, P = 2, 6, 2, 4, 128, 64
    lens, rows = [700, 420], [6, 2]
    W = 12
    cache = rand_cache(api, B * W, H, P, D, 206)
    table = rand_table(B, W, B * W, 207)
    q = torch.randn(B, N, H * G, D, generator=gen(208)).to(BF).cuda()
    q[1, 2:] = math.nan
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    prev = torch.zeros(B, H, W * P, device="cuda")
    lse = ref.attend(ref.Cache64(cache, table), q.nan_to_num(nan=0.0), lens, rows, None, D ** -0.5, 0.0)[1].float().cuda()
    w = api.spec_cache_weights(q, lse, cache, table, ln, prev=prev)
    check_weights(w["weights"], cache, table, q, lse, lens, [N] * B, None, 0.0, prev)
    total = w["weights"].double().sum(2)
    assert bool(((total - torch.tensor(rows, device="cuda")[:, None] * G).abs() < 0.01).all())


# ------------------------------------------------------------------ many short units

@pytest.mark.parametrize("N,G,D,dtype", [(3, 4, 128, BF), (9, 4, 128, HF), (16, 4, 64, BF), (40, 4, 64, HF)])
def test_units_of_a_tile_or_two_keep_their_own_factors(api, N, G, D, dtype):  # noqa: F811
    """Requests of up to two tiles, many to a CTA, whose rows of q differ in magnitude: four copies, two and one of the rows."""
    B, H, P = 320, 2, 16
    g = gen(210)
    lens = torch.randint(0, 250 - N, (B,), generator=g).tolist()
    W = -(-250 // P)
    cache = rand_cache(api, B * W, H, P, D, 211)
    table = rand_table(B, W, B * W, 212)
    size = torch.exp2(-3.0 * torch.randint(0, 4, (B, N, 1, 1), generator=g))
    q = (torch.randn(B, N, H * G, D, generator=g) * 4 * size).to(dtype).cuda()
    check_attend(api, q, cache, table, lens)


# ------------------------------------------------------------------ status

@pytest.mark.parametrize("B", [3, 300])
@pytest.mark.parametrize("D", [64, 80, 128])
def test_a_status_from_before_does_not_stay(api, B, D):  # noqa: F811
    """Whatever the caller's status held, each request gets its own of this call: good ones, empty ones, and every kind of bad one."""
    N, H, G, P, W = 4, 2, 2, 16, 4
    cache = rand_cache(api, 64, H, P, D, 220)
    table = torch.randint(0, 64, (B, W), generator=gen(221)).to(torch.int32).cuda()
    lens = torch.randint(0, W * P - N, (B,), generator=gen(222)).to(torch.int32).cuda()
    index = torch.arange(N, dtype=torch.int32, device="cuda").repeat(B, 1).contiguous()
    counts = torch.full((B,), N, dtype=torch.int32, device="cuda")
    q = torch.randn(B, N, H * G, D, generator=gen(223)).to(BF).cuda()
    lse = torch.full((B, N, H * G), 4.0, device="cuda")
    prev = torch.rand(B, H, W * P, generator=gen(224)).cuda()
    want = [0] * B
    for b, kind in zip((1, B - 1, B // 2, B // 3, 2 * B // 3), ("page", "length", "index", "count", "empty")):
        want[b] = {"page": api.STATUS_BAD_PAGE, "index": api.STATUS_BAD_INDEX, "empty": 0}.get(kind, api.STATUS_BAD_LENGTH)
        lens[b], counts[b], index[b], table[b] = 20, N, torch.arange(N), torch.arange(W)
        if kind == "page":
            table[b, 1] = 64
        elif kind == "length":
            lens[b] = W * P
        elif kind == "index":
            index[b, 2] = N
        elif kind == "count":
            counts[b] = N + 1
        else:
            lens[b], counts[b] = 0, 0
    for before in (-5, 0, api.STATUS_TIMEOUT, 1 << 30):
        o = dict(weights=prev.clone(), status=torch.full((B,), before, dtype=torch.int32, device="cuda"))
        api.spec_cache_weights(q, lse, cache, table, lens, prev=prev, counts=counts, index=index, out=o)
        assert o["status"].tolist() == want
        for b in range(B):
            if want[b]:
                assert torch.equal(o["weights"][b], prev[b])


# ------------------------------------------------------------------ tracing

@pytest.mark.parametrize("D", [64, 80, 128])
def test_repeats_of_a_traced_call_change_nothing(api, D):  # noqa: F811
    """Every operator under spec_trace_repeat gives the bits of an untraced call; weights in place as well."""
    B, N, H, G, P, W = 2, 5, 2, 3, 32, 8
    lens = torch.tensor([200, 37], dtype=torch.int32, device="cuda")
    q = torch.randn(B, N, H * G, D, generator=gen(230)).to(BF).cuda()
    k, v = (torch.randn(B, N, H, D, generator=gen(s)).to(BF).cuda() * 9 for s in (231, 232))
    prev = torch.rand(B, H, W * P, generator=gen(233)).cuda()

    def step():
        cache = rand_cache(api, B * W + B * 2, H, P, D, 234)
        every = torch.randperm(B * W + B * 2, generator=gen(235)).to(torch.int32).cuda()
        table, dst = every[:B * W].reshape(B, W).contiguous(), every[B * W:].reshape(B, 2).contiguous()
        a = api.spec_cache_append(cache, table, lens, k, v)
        o = api.spec_cache_attend(q, cache, table, lens)
        w = api.spec_cache_weights(q, o["lse"], cache, table, lens, prev=prev)
        room = prev.clone()
        i = api.spec_cache_weights(q, o["lse"], cache, table, lens, prev=room, out=dict(weights=room))
        e = api.spec_cache_evict(cache, table, a["new_len"], i["weights"], 50, 5, dst)
        return [t.clone() for x in (a, o, w, i, e) for t in x.values()] + [x.view(torch.uint8) for x in cache[:2]] + cache[2:], w, i

    want, w, i = step()
    assert torch.equal(w["weights"], i["weights"])
    api.trace_enable(True)
    api.trace_repeat(3)
    try:
        got = step()[0]
        torch.cuda.synchronize()
        times = api.trace_collect(32)
    finally:
        api.trace_repeat(1)
        api.trace_enable(False)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    assert all(ms > 0 for ms, _ in times.values()) and len(times) >= 5


# ------------------------------------------------------------------ host threads

def test_threads_on_one_stream_get_their_own_answers(api):  # noqa: F811
    """Attention of two shapes, each from a thread of its own, over the workspace of the stream that they share."""
    import threading

    jobs = []
    for seed, (B, N, H, G, D, W) in ((240, (2, 9, 2, 4, 128, 40)), (241, (24, 20, 2, 4, 64, 12))):
        cache = rand_cache(api, B * W, H, 64, D, seed)
        table = rand_table(B, W, B * W, seed)
        lens = torch.randint(0, W * 64 - N, (B,), generator=gen(seed)).to(torch.int32).cuda()
        q = torch.randn(B, N, H * G, D, generator=gen(seed)).to(BF).cuda()
        jobs.append((q, cache, table, lens))
    want = [api.spec_cache_attend(*j) for j in jobs]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        for _ in range(200):
            got[i].append(api.spec_cache_attend(*jobs[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in (0, 1):
        assert len(got[i]) == 200
        for o in got[i]:
            for name in ("out", "lse", "status"):
                assert torch.equal(o[name], want[i][name]), (i, name)


@pytest.mark.parametrize("name", ["append", "attend", "few", "weights", "evict"])
def test_a_threads_first_call(api, name):  # noqa: F811
    """An operator as the first thing that a host thread does with the GPU."""
    import threading

    B, N, H, G, P, D, W = 2, 9, 2, 4, 64, 128, 40
    cache = rand_cache(api, B * W, H, P, D, 250)
    table = rand_table(B, W, B * W, 251)
    lens = torch.tensor([2500, 1200], dtype=torch.int32, device="cuda")
    q = torch.randn(B, N, H * G, D, generator=gen(252)).to(BF).cuda()
    lse = torch.full((B, N, H * G), 4.0, device="cuda")
    w = torch.rand(B, H, W * P, generator=gen(253)).cuda()
    one = q[:, :1, :2].contiguous()
    dst = api.spec_cache_new(B, H, P, D)
    to = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    call = {"append": lambda: api.spec_cache_append(cache, table, lens, q[:, :, :H], q[:, :, H:2 * H]),
            "attend": lambda: api.spec_cache_attend(q, cache, table, lens),
            "few": lambda: api.spec_cache_attend(one, cache, table, lens),
            "weights": lambda: api.spec_cache_weights(q, lse, cache, table, lens, prev=w),
            "evict": lambda: api.spec_cache_evict(cache, table, lens, w, 50, 5, to, dst_cache=dst)}[name]
    want = call()
    torch.cuda.synchronize()
    got = []
    thread = threading.Thread(target=lambda: got.append(call()))
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert got and all(torch.equal(got[0][x], want[x]) for x in want)


# ------------------------------------------------------------------ no rows at all

@pytest.mark.parametrize("D", [64, 80, 128])
def test_calls_without_rows_say_what_is_wrong(api, D):  # noqa: F811
    """N = 0: nothing to write but the status (and the new length), which tell good requests from bad ones as ever."""
    B, H, G, P, W = 4, 2, 2, 16, 4
    cache = rand_cache(api, 16, H, P, D, 260)
    table = torch.arange(16, dtype=torch.int32, device="cuda").reshape(B, W)
    table[2, 1] = 99
    lens = torch.tensor([30, W * P + 1, 40, 0], dtype=torch.int32, device="cuda")
    q = torch.empty(B, 0, H * G, D, dtype=BF, device="cuda")
    k = torch.empty(B, 0, H, D, dtype=BF, device="cuda")
    prev = torch.rand(B, H, W * P, generator=gen(261)).cuda()
    want = [0, api.STATUS_BAD_LENGTH, api.STATUS_BAD_PAGE, 0]
    for before in (-3, 77):
        status = torch.full((B,), before, dtype=torch.int32, device="cuda")
        out = dict(out=torch.empty_like(q), lse=torch.empty(B, 0, H * G, device="cuda"), status=status)
        assert api.spec_cache_attend(q, cache, table, lens, out=out)["status"].tolist() == want
        status.fill_(before)
        mask = torch.ones(B, 0, 0, dtype=torch.uint8, device="cuda")
        assert api.spec_cache_attend(q, cache, table, lens, mask=mask, lse=False, out=dict(out=out["out"], status=status))["status"].tolist() == want
        status.fill_(before)
        w = api.spec_cache_weights(q, out["lse"], cache, table, lens, prev=prev, out=dict(weights=prev.clone(), status=status))
        assert w["status"].tolist() == want and torch.equal(w["weights"], prev)
        new = torch.full((B,), before, dtype=torch.int32, device="cuda")
        status.fill_(before)
        a = api.spec_cache_append(cache, table, lens, k, k, out=dict(new_len=new, status=status))
        # (no page is written, so none is looked at)
        assert a["status"].tolist() == [0, api.STATUS_BAD_LENGTH, 0, 0] and a["new_len"].tolist() == lens.tolist()


@pytest.mark.parametrize("D", [64, 80])
def test_empty_contexts_with_room_for_nothing(api, D):  # noqa: F811
    """Weights of no positions at all (an empty tensor has no address): nothing is kept, and a longer request is told so."""
    B, H, G, P = 3, 2, 2, 16
    cache = rand_cache(api, 8, H, P, D, 270)
    none = torch.empty(B, H, 0, device="cuda")
    table = torch.arange(3, dtype=torch.int32, device="cuda")[:, None].contiguous()
    lens = torch.tensor([0, 2, 0], dtype=torch.int32, device="cuda")
    want = [0, api.STATUS_BAD_LENGTH, 0]
    e = api.spec_cache_evict(cache, table, lens, none, 4, 1, table + 3)
    assert e["status"].tolist() == want and e["new_len"].tolist() == [0, 0, 0] and bool((e["kept"] == -1).all())
    q = torch.randn(B, 1, H * G, D, generator=gen(271)).to(BF).cuda()
    lse = torch.zeros(B, 1, H * G, device="cuda")
    counts = torch.zeros(B, dtype=torch.int32, device="cuda")
    for prev in (None, none):
        w = api.spec_cache_weights(q, lse, cache, table, lens, prev=prev, counts=counts,
                                   out=dict(weights=none, status=torch.full((B,), 9, dtype=torch.int32, device="cuda")))
        assert w["status"].tolist() == want
    # a table of no pages
    w = api.spec_cache_weights(q, lse, cache, table[:, :0].contiguous(), counts, counts=counts)
    assert w["status"].tolist() == [0, 0, 0] and w["weights"].shape == (B, H, 0)


# ------------------------------------------------------------------ scales that are no powers of two

def e4m3_values():
    """Every positive number of e4m3 and the points half way between neighbours."""
    x = torch.arange(1, 127, dtype=torch.uint8).view(ref.F8).double()
    return x, (x[1:] + x[:-1]) / 2


def near_ties(limit):
    """(a, half, s): s the float32 nearest half / a, so that the product a s is the half-way point `half` in float32 but not exactly; s < 1."""
    values, halves = e4m3_values()
    found = []
    for a in values.tolist():
        for half in halves.tolist():
            if not 0.5 < half / a < 1:
                continue
            s = float(torch.tensor(half / a, dtype=torch.float64).float())
            if a * s != half and float(torch.tensor(a).float() * torch.tensor(s).float()) == half:
                found.append((a, half, s))
    return found[::max(1, len(found) // limit)][:limit]


def codes(x):
    return torch.tensor(x, dtype=torch.float64).float().to(ref.F8).view(torch.uint8)


def same_cells(cache, table, want):
    got = ref.Cache64(cache, table)
    for w in (0, 1):
        assert torch.equal(got.scale[w], want.scale[w])
        assert torch.equal(got.val[w], want.val[w])


@pytest.mark.parametrize("D", [64, 80, 128])
@pytest.mark.parametrize("s", [0.7, 1.0 / 3, 0.013])
def test_append_rounds_a_quotient_once(api, D, s):  # noqa: F811
    """New rows behind a token whose block keeps a scale of the caller's own: values whose quotient is half way in float32, not in truth."""
    P, H = 16, 1
    _, halves = e4m3_values()
    s = float(torch.tensor(s).float())
    reach = 448 * 2.0 ** math.floor(math.log2(s))  # what asks for no scale above s
    x = (halves * s).float()
    x = x[x < reach]
    x = torch.cat([x, -x, x.nextafter(torch.tensor(math.inf)), x.nextafter(torch.tensor(0.0))])
    x = torch.nn.functional.pad(x, (0, -len(x) % D)).reshape(1, -1, H, D)
    x = x[:, :P - 1] if x.shape[1] >= P else x
    cache = rand_cache(api, 1, H, P, D, 280)
    for i in (2, 3):
        cache[i].fill_(s)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    want = ref.Cache64(cache, table)
    want.append(0, 1, x[0], x[0])
    assert float(want.scale[0]) == s
    api.spec_cache_append(cache, table, torch.ones(1, dtype=torch.int32, device="cuda"), x.cuda(), x.cuda())
    same_cells(cache, table, want)


@pytest.mark.parametrize("D", [64, 128])
def test_append_rounds_old_tokens_once(api, D):  # noqa: F811
    """A block whose scale of the caller's own grows to a power of two: old values half way in float32, not in truth."""
    ties = near_ties(60)
    P, H, B = 16, 1, len(ties)
    cache = rand_cache(api, B, H, P, D, 281)
    for b, (a, _, s) in enumerate(ties):
        for w in (0, 1):
            cache[w].view(torch.uint8)[b, 0, :3] = codes([a, -a])[torch.arange(3 * D) % 2].reshape(3, D).cuda()
            cache[2 + w][b] = s
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    x = torch.full((B, 1, H, D), 448.0).to(BF)  # asks for a scale of 1
    want = ref.Cache64(cache, table)
    for b in range(B):
        want.append(b, 3, x[b], x[b])
    assert bool((want.scale[0] == 1).all())
    api.spec_cache_append(cache, table, torch.full((B,), 3, dtype=torch.int32, device="cuda"), x.cuda(), x.cuda())
    same_cells(cache, table, want)


@pytest.mark.parametrize("D", [64, 80, 128])
def test_evict_rounds_once(api, D):  # noqa: F811
    """Kept rows of a block with a scale of the caller's own: values half way in float32, and largest ones just above a scale's reach."""
    ties = near_ties(60)
    values, _ = e4m3_values()
    for a in values.tolist():  # a s is 448 in float32 and more in truth: the scale has to be 2
        s = float(torch.tensor(448.0 / a, dtype=torch.float64).float())
        if a < 448 and a * s > 448 and float(torch.tensor(a).float() * torch.tensor(s).float()) == 448:
            ties.append((a, None, s))
    assert ties[-1][1] is None
    P, H, B = 16, 1, len(ties)
    cache = rand_cache(api, B, H, P, D, 282)
    pool = rand_cache(api, B, H, P, D, 283)
    for b, (a, half, s) in enumerate(ties):
        for w in (0, 1):
            x = codes([a, -a])[torch.arange(5 * D) % 2].reshape(5, D)
            if half is not None:
                x[4, 7] = codes([448.0])[0]  # scale 1
            cache[w].view(torch.uint8)[b, 0, :5] = x.cuda()
            cache[2 + w][b] = s
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    before, want = ref.Cache64(cache, table), ref.Cache64(pool, table)
    lens = torch.full((B,), 5, dtype=torch.int32, device="cuda")
    api.spec_cache_evict(cache, table, lens, torch.ones(B, H, P, device="cuda"), 5, 0, table, dst_cache=pool)
    for b, (_, half, _) in enumerate(ties):
        for w in (0, 1):
            rows = before.rows(w, b, 5)[0]
            scale = ref.block_scale(rows)
            assert scale == (2 if half is None else 1)
            want.scale[w][b, 0] = scale
            want.val[w][b, 0, :5] = ref.e4m3(rows / scale)
    same_cells(pool, table, want)


# ------------------------------------------------------------------ wrong requests on the tensor cores

@pytest.mark.parametrize("N,G,D", [(5, 4, 128), (16, 4, 64), (40, 4, 128)])
@pytest.mark.parametrize("kind", ["page", "page below", "length", "negative", "count"])
def test_wrong_requests_among_long_ones(api, kind, N, G, D):  # noqa: F811
    """Requests cut over several CTAs, every third of them wrong: those give zeros and their status, the others the bits they had."""
    B, H, P = 9, 2, 64
    lens = torch.tensor([3000, 2100, 900, 64, 5000, 1, 700, 4000, 2500], dtype=torch.int32, device="cuda")
    W = -(-(5000 + N) // P)
    cache = rand_cache(api, B * W, H, P, D, 290)
    table = rand_table(B, W, B * W, 291)
    q = torch.randn(B, N, H * G, D, generator=gen(292)).to(BF).cuda()
    n = torch.full((B,), N, dtype=torch.int32, device="cuda")
    lse = torch.full((B, N, H * G), 5.0, device="cuda")
    prev = torch.rand(B, H, W * P, generator=gen(293)).cuda()

    def both():
        return (api.spec_cache_attend(q, cache, table, lens, n_query=n),
                api.spec_cache_weights(q, lse, cache, table, lens, prev=prev, counts=n))

    good = both()
    wrong = [1, 4, 7]
    for b in wrong:
        if kind == "page":
            table[b, int(lens[b]) // P] = B * W
        elif kind == "page below":
            table[b, 0] = -7
        elif kind == "length":
            lens[b] = W * P
        elif kind == "negative":
            lens[b] = -(1 << 31)
        else:
            n[b] = N + 1
    status = api.STATUS_BAD_PAGE if "page" in kind else api.STATUS_BAD_LENGTH
    o, w = both()
    for x in (o, w):
        assert x["status"].tolist() == [status if b in wrong else 0 for b in range(B)]
    for b in range(B):
        if b in wrong:
            assert bool((o["out"][b] == 0).all()) and bool((o["lse"][b] == -math.inf).all()) and torch.equal(w["weights"][b], prev[b])
        else:
            assert torch.equal(w["weights"][b], good[1]["weights"][b])
            if "page" in kind:  # (a request without a length moves the cuts, and with them the order of sums)
                assert torch.equal(o["out"][b], good[0]["out"][b]) and torch.equal(o["lse"][b], good[0]["lse"][b])
    check_attend_of_good(o, q, cache, table, lens, n, wrong)


def check_attend_of_good(o, q, cache, table, lens, n, wrong):
    lens, n = lens.tolist(), n.tolist()
    for b in wrong:
        lens[b], n[b] = 0, 0
    out, lse, t_out, t_lse = ref.attend(ref.Cache64(cache, table), q, lens, n, None, q.shape[3] ** -0.5, 0.0)
    for b in range(len(lens)):
        if b not in wrong:
            assert bool(((o["out"][b].cpu().double() - out[b]).abs() <= t_out[b]).all())
            assert bool(((o["lse"][b].cpu().double() - lse[b]).abs() <= t_lse[b]).all())
