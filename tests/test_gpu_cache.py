"""The 8-bit cache's operators on the GPU against their 64-bit definitions."""
import math

import pytest
import torch

import cache_oracle as ref

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def api():
    from speculative_decoding_verification_02_gb300 import api, build
    build.build()
    torch.cuda.set_device(0)
    return api


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rand_cache(api, pages, H, P, D, seed, spread=3, page_gap=0):
    """A pool of random codes (NaN among none) whose blocks differ in scale; page_gap: bytes between pages."""
    g = gen(seed)
    parts = []
    for _ in range(2):
        room = torch.zeros(pages, H * P * D + page_gap, dtype=torch.uint8)
        x = (torch.randn(pages, H * P * D, generator=g) * 40).clamp(-448, 448).to(ref.F8)
        room[:, :H * P * D] = x.view(torch.uint8)
        room = room.cuda()
        parts.append(torch.as_strided(room, (pages, H, P, D), (H * P * D + page_gap, P * D, D, 1)).view(ref.F8))
    scales = [torch.exp2(torch.randint(-6 - spread, -5, (pages, H), generator=g).float()).cuda() for _ in range(2)]
    return [parts[0], parts[1], scales[0], scales[1]]


def rand_table(B, W, pages, seed):
    return torch.randperm(pages, generator=gen(seed))[:B * W].reshape(B, W).to(torch.int32).cuda()


def tree_mask(B, n, seed):
    g = gen(seed)
    m = torch.zeros(B, n, n, dtype=torch.uint8)
    for b in range(B):
        for i in range(n):
            if i:
                m[b, i] = m[b, int(torch.randint(0, i, (1,), generator=g))]
            m[b, i, i] = 1
    return m.cuda()


def check_attend(api, q, cache, table, lens, n_query=None, mask=None, scale=None, cap=0.0, **kw):
    B, N = q.shape[:2]
    dev_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    nq = None if n_query is None else torch.tensor(n_query, dtype=torch.int32, device="cuda")
    o = api.spec_cache_attend(q, cache, table, dev_lens, n_query=nq, mask=mask, scale=scale, softcap=cap, **kw)
    torch.cuda.synchronize()
    s = q.shape[3] ** -0.5 if scale is None else scale
    out, lse, t_out, t_lse = ref.attend(ref.Cache64(cache, table), q, lens, n_query or [N] * B, mask, s, cap)
    assert o["status"].tolist() == [0] * B
    got, got_lse = o["out"].cpu().double(), o["lse"].cpu().double()
    empty = lse == -math.inf
    assert torch.equal(got_lse == -math.inf, empty)
    assert bool((got[empty] == 0).all())
    worst = ((got - out).abs() / t_out.clamp(min=1e-300))[~empty]
    assert bool((worst <= 1).all()), float(worst.max())
    worst = ((got_lse - lse).abs() / t_lse)[~empty]
    assert bool((worst <= 1).all()), float(worst.max())
    return o


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("D,P,H,dtype", [(128, 64, 2, BF), (64, 16, 3, HF), (128, 128, 1, torch.float32), (80, 32, 2, BF), (256, 256, 1, HF),
                                         (16, 16, 5, BF)])
@pytest.mark.parametrize("lens,counts", [([0, 5, 63], [1, 9, 9]), ([16, 127, 31], [0, 40, 33]), ([255, 0, 1], [41, 0, 2])])
def test_append(api, D, P, H, dtype, lens, counts):
    B, n = 3, 41
    W = -(-(max(lens) + n) // P)
    cache = rand_cache(api, B * W + 2, H, P, D, 1)
    table = rand_table(B, W, B * W + 2, 2)
    g = gen(3)
    k = (torch.randn(B, n, H, D, generator=g) * torch.exp(2 * torch.randn(B, n, 1, 1, generator=g))).to(dtype).cuda()
    v = (torch.randn(B, n, H, D, generator=g) * 3).to(dtype).cuda()
    want = ref.Cache64(cache, table)
    for b in range(B):
        want.append(b, lens[b], k[b, :counts[b]].cpu(), v[b, :counts[b]].cpu())
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o = api.spec_cache_append(cache, table, ln, k, v, counts=torch.tensor(counts, dtype=torch.int32, device="cuda"))
    assert o["status"].tolist() == [0] * B and o["new_len"].tolist() == [a + c for a, c in zip(lens, counts)]
    got = ref.Cache64(cache, table)
    for w in (0, 1):
        assert torch.equal(got.val[w], want.val[w])  # the untouched pages and slots among them
        assert torch.equal(got.scale[w], want.scale[w])


def test_append_path_strides_and_dtype_of_layout(api):
    """Rows picked by index, keys and values as slices of one [B, H, n, 3, D] projection, pages apart from one another."""
    B, n, H, D, P = 2, 12, 2, 128, 16
    cache = rand_cache(api, 9, H, P, D, 4, page_gap=48)
    table = rand_table(B, 3, 9, 5)
    x = torch.randn(B, H, n, 3, D, generator=gen(6)).to(BF).cuda()
    k, v = x[:, :, :, 1].transpose(1, 2), x[:, :, :, 2].transpose(1, 2)
    index = torch.tensor([[0, 3, 4, 11, -1], [0, 1, 7, 9, 10]], dtype=torch.int32, device="cuda")
    counts = torch.tensor([4, 5], dtype=torch.int32, device="cuda")
    lens = [14, 0]
    want = ref.Cache64(cache, table)
    for b in range(B):
        at = index[b, :int(counts[b])].long()
        want.append(b, lens[b], k[b][at].cpu(), v[b][at].cpu())
    o = api.spec_cache_append(cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), k, v, counts=counts, index=index)
    assert o["new_len"].tolist() == [18, 5] and o["status"].tolist() == [0, 0]
    got = ref.Cache64(cache, table)
    for w in (0, 1):
        assert torch.equal(got.val[w], want.val[w]) and torch.equal(got.scale[w], want.scale[w])


@pytest.mark.parametrize("offset", [1, 3])
def test_append_unaligned_rows(api, offset):
    B, n, H, D, P = 1, 5, 2, 64, 16
    cache = rand_cache(api, 2, H, P, D, 7)
    table = rand_table(B, 2, 2, 8)
    flat = torch.randn(2 * B * n * H * D + 8, generator=gen(9)).to(BF).cuda()
    k = flat[offset:offset + B * n * H * D].view(B, n, H, D)
    v = flat[offset + B * n * H * D:][:B * n * H * D].view(B, n, H, D)
    want = ref.Cache64(cache, table)
    want.append(0, 13, k[0].cpu(), v[0].cpu())
    api.spec_cache_append(cache, table, torch.tensor([13], dtype=torch.int32, device="cuda"), k, v)
    got = ref.Cache64(cache, table)
    for w in (0, 1):
        assert torch.equal(got.val[w], want.val[w]) and torch.equal(got.scale[w], want.scale[w])


def test_append_extremes(api):
    """Zeros, tiny and huge values, infinities and NaN, and a scale that grows over a block of small values."""
    H, D, P = 1, 32, 16
    rows = torch.zeros(1, 8, H, D)
    rows[0, 1] = 1e-30
    rows[0, 2] = 3e38
    rows[0, 3, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 1.0])
    rows[0, 4] = torch.linspace(-500, 500, D)
    rows[0, 5] = 2.0 ** -70
    rows[0, 6] = 448.0 * 2.0 ** 60
    rows[0, 7] = 449.0
    x = rows.cuda()
    for order in ([0, 4, 7], [1, 5, 0], [4, 2], [3, 4], [0, 3], [6, 4], [1, 4, 2]):
        cache = rand_cache(api, 1, H, P, D, 10)
        table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
        want = ref.Cache64(cache, table)
        n = 0
        for t in order:  # one row a call
            want.append(0, n, rows[0, t:t + 1], rows[0, t:t + 1])
            api.spec_cache_append(cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), x[:, t:t + 1], x[:, t:t + 1])
            n += 1
        got = ref.Cache64(cache, table)
        for w in (0, 1):
            assert torch.equal(got.scale[w], want.scale[w]), order
            assert torch.equal(got.val[w][0, 0, :n].nan_to_num(nan=1e9), want.val[w][0, 0, :n].nan_to_num(nan=1e9)), order


# ------------------------------------------------------------------ attend

SHAPES = [  # B, N, H, G, D, P, lens
    (1, 1, 1, 1, 128, 64, [0]),
    (1, 1, 2, 4, 128, 64, [1]),
    (2, 1, 2, 8, 64, 16, [15, 16]),
    (3, 5, 2, 4, 128, 64, [127, 128, 129]),
    (2, 9, 1, 4, 128, 32, [500, 3]),
    (1, 17, 2, 3, 64, 128, [300]),
    (2, 33, 1, 2, 128, 16, [77, 1000]),
    (1, 60, 2, 4, 128, 64, [411]),
    (2, 64, 1, 8, 64, 256, [255, 600]),
    (1, 150, 1, 2, 128, 64, [64]),
    (2, 7, 3, 1, 80, 32, [65, 40]),
    (1, 3, 1, 2, 256, 16, [200]),
]


@pytest.mark.parametrize("B,N,H,G,D,P,lens", SHAPES)
@pytest.mark.parametrize("dtype,cap", [(BF, 0.0), (HF, 0.0), (BF, 30.0)])
@pytest.mark.parametrize("tree", [False, True])
def test_attend(api, B, N, H, G, D, P, lens, dtype, cap, tree):
    W = -(-(max(lens) + N) // P)
    cache = rand_cache(api, B * W + 1, H, P, D, 11)
    table = rand_table(B, W, B * W + 1, 12)
    q = (torch.randn(B, N, H * G, D, generator=gen(13)) * 2).to(dtype).cuda()
    check_attend(api, q, cache, table, lens, mask=tree_mask(B, N, 14) if tree else None, cap=cap)


@pytest.mark.parametrize("D,G,N,dtype,cap", [(64, 1, 1, BF, 0.0), (128, 1, 1, HF, 0.0), (64, 2, 1, HF, 25.0), (128, 4, 1, BF, 25.0), (128, 1, 3, BF, 0.0),
                                             (64, 1, 4, BF, 0.0), (96, 3, 2, HF, 0.0), (240, 1, 2, BF, 10.0)])
@pytest.mark.parametrize("tree", [False, True])
def test_attend_few_rows(api, D, G, N, dtype, cap, tree):
    """One to six rows: the scalar kernel, its clusters, requests without positions and shares that are empty."""
    B, H, P = 5, 2, 16
    lens = [0, 1, 130, 1025, 3000]
    W = -(-(max(lens) + N) // P)
    cache = rand_cache(api, B * W, H, P, D, 111)
    table = rand_table(B, W, B * W, 112)
    q = (torch.randn(B, N, H * G, D, generator=gen(113)) * 2).to(dtype).cuda()
    check_attend(api, q, cache, table, lens, n_query=[N, N, max(N - 1, 0), N, N], mask=tree_mask(B, N, 114) if tree else None, cap=cap)


@pytest.mark.parametrize("N,G,D", [(1, 1, 128), (9, 4, 128), (40, 4, 64)])
def test_scales_that_are_no_powers_of_two(api, N, G, D):
    """A cache that another program wrote: any positive scale is served by the operators that read it."""
    B, H, P, W = 2, 2, 32, 12
    lens = [300, 65]
    cache = rand_cache(api, B * W, H, P, D, 115)
    for i in (2, 3):
        cache[i] *= 1 + 0.7 * torch.rand(cache[i].shape, generator=gen(116)).cuda()
    table = rand_table(B, W, B * W, 117)
    q = torch.randn(B, N, H * G, D, generator=gen(118)).to(BF).cuda()
    o = check_attend(api, q, cache, table, lens)
    w = api.spec_cache_weights(q, o["lse"], cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    want, tol = ref.weights(ref.Cache64(cache, table), q, o["lse"], lens, [N] * B, None, D ** -0.5, 0.0, torch.zeros_like(w["weights"]))
    assert bool(((w["weights"].cpu().double() - want).abs() <= tol).all())


def test_attend_long_and_ragged(api):
    lens = [20000, 0, 777, 4095, 1, 9000]
    B, N, H, G, D, P = 6, 5, 2, 4, 128, 128
    W = -(-(max(lens) + N) // P)
    cache = rand_cache(api, B * W, H, P, D, 15)
    table = rand_table(B, W, B * W, 16)
    q = torch.randn(B, N, H * G, D, generator=gen(17)).to(BF).cuda()
    check_attend(api, q, cache, table, lens, n_query=[5, 5, 0, 3, 1, 4])


def test_attend_sharp_and_flat_scores(api):
    """A far token that holds almost all of the weight, and a context of equal scores."""
    B, N, H, G, D, P = 2, 2, 1, 4, 128, 64
    lens = [3000, 5000]
    W = -(-(max(lens) + N) // P)
    cache = rand_cache(api, B * W, H, P, D, 18)
    table = rand_table(B, W, B * W, 19)
    q = (torch.randn(B, N, H * G, D, generator=gen(20)) * 30).to(BF).cuda()
    q[1] = 0
    check_attend(api, q, cache, table, lens)
    check_attend(api, q, cache, table, lens, scale=0.0)
    check_attend(api, q, cache, table, lens, scale=-0.05)


def test_attend_scales_far_apart(api):
    """Blocks whose values differ by 2^40, and the largest scale's block first, last and between."""
    B, N, H, G, D, P = 3, 3, 1, 2, 128, 16
    lens = [200, 150, 129]
    W = -(-(max(lens) + N) // P)
    cache = rand_cache(api, B * W, H, P, D, 21)
    table = torch.arange(B * W, dtype=torch.int32, device="cuda").reshape(B, W)
    cache[3][:] = torch.exp2(torch.randint(-40, 1, (B * W, H), generator=gen(22)).float()).cuda()
    cache[3][0] = 1.0
    cache[3][W + 9] = 2.0 ** 30
    cache[3][2 * W + 3] = 2.0 ** -60
    q = torch.randn(B, N, H * G, D, generator=gen(23)).to(BF).cuda()
    check_attend(api, q, cache, table, lens)


def test_attend_masked_places_hold_anything(api):
    """NaN in slots behind the context, in pages' unused ends and in rows that a row does not see changes nothing."""
    B, N, H, G, D, P = 2, 6, 2, 2, 128, 64
    lens = [70, 0]
    cache = rand_cache(api, 8, H, P, D, 24)
    table = rand_table(B, 2, 8, 25)
    mask = tree_mask(B, N, 26)
    mask[1, 2] = 0  # a row that sees nothing
    mask[:, :, 4] = 0
    mask[:, 4, 4] = 1  # only itself sees row 4
    q = torch.randn(B, N, H * G, D, generator=gen(27)).to(BF).cuda()
    clean = check_attend(api, q, cache, table, lens, mask=mask)
    nan = torch.full((1,), math.nan).to(ref.F8).view(torch.uint8).item()
    for pool in cache[:2]:
        raw = pool.view(torch.uint8)
        for b in range(B):
            T = lens[b] + N
            for t in range(T, 2 * P):
                raw[int(table[b, t // P]), :, t % P] = nan
            t = lens[b] + 4
            raw[int(table[b, t // P]), :, t % P] = nan
    o = api.spec_cache_attend(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), mask=mask)
    for i in range(N):
        if i == 4:
            assert bool(o["out"][:, 4].isnan().all())
        else:
            assert torch.equal(o["out"][:, i], clean["out"][:, i]) and torch.equal(o["lse"][:, i], clean["lse"][:, i])
    assert bool((o["out"][1, 2] == 0).all()) and bool((o["lse"][1, 2] == -math.inf).all())


def test_attend_nan_in_the_context_shows(api):
    cache = rand_cache(api, 4, 1, 64, 128, 28)
    table = rand_table(1, 4, 4, 29)
    q = torch.randn(1, 2, 4, 128, generator=gen(30)).to(BF).cuda()
    ln = torch.tensor([190], dtype=torch.int32, device="cuda")
    cache[1].view(torch.uint8)[int(table[0, 1]), 0, 7, 5] = 0x7f
    o = api.spec_cache_attend(q, cache, table, ln)
    assert bool(o["out"][..., 5].isnan().all())
    cache[0].view(torch.uint8)[int(table[0, 1]), 0, 7, 5] = 0x7f
    o = api.spec_cache_attend(q, cache, table, ln)
    assert bool(o["out"].isnan().all())


def test_attend_strides(api):
    """q as a transposed slice of a fused projection, out likewise, pages apart, offsets that are not of 16 bytes."""
    B, N, H, G, D, P = 2, 7, 2, 4, 128, 32
    lens = [100, 33]
    cache = rand_cache(api, 9, H, P, D, 31, page_gap=64)
    table = rand_table(B, 4, 9, 32)
    x = torch.randn(B, H * G, N, D + 3, generator=gen(33)).to(BF).cuda()
    q = x[..., 1:D + 1].transpose(1, 2)
    y = torch.full((B, H * G, N, D + 5), 7.0, dtype=BF, device="cuda")
    out = dict(out=y[..., 3:D + 3].transpose(1, 2), lse=torch.empty(B, N, H * G, device="cuda"),
               status=torch.empty(B, dtype=torch.int32, device="cuda"))
    check_attend(api, q, cache, table, lens, out=out)
    assert bool((y[..., :3] == 7).all()) and bool((y[..., D + 3:] == 7).all())


@pytest.fixture
def roomy(monkeypatch):
    """Page tables with room for thousands of further positions, their entries not yet given: short contexts, but the choice of the
    kernel goes by the room, so more than four rows are the tensor cores' here and the scalar kernel's without."""
    narrow = rand_table
    monkeypatch.setitem(globals(), "rand_table",
                        lambda *a: torch.nn.functional.pad(narrow(*a), (0, 200), value=-1).contiguous())


@pytest.mark.parametrize("B,N,H,G,D,P,lens", SHAPES)
@pytest.mark.parametrize("dtype,cap", [(BF, 0.0), (HF, 0.0), (BF, 30.0), (HF, 5.0)])
@pytest.mark.parametrize("tree", [False, True])
def test_attend_with_room_to_grow(api, roomy, B, N, H, G, D, P, lens, dtype, cap, tree):
    test_attend(api, B, N, H, G, D, P, lens, dtype, cap, tree)


@pytest.mark.parametrize("test", [test_attend_masked_places_hold_anything, test_attend_nan_in_the_context_shows, test_attend_strides,
                                  test_attend_scales_far_apart, test_attend_sharp_and_flat_scores])
def test_attend_cases_with_room_to_grow(api, roomy, test):
    test(api)


@pytest.mark.parametrize("D,G,N,cap", [(64, 8, 1, 0.0), (128, 3, 3, 30.0), (64, 1, 60, 0.0), (128, 4, 9, 0.0)])
@pytest.mark.parametrize("tree", [False, True])
def test_attend_more_rows_over_short_contexts(api, D, G, N, cap, tree):
    """Chunks of four rows over whole contexts, one of them the last and ragged, in clusters and alone."""
    B, H, P = 5, 2, 16
    lens = [0, 1, 130, 270, 64]
    W = -(-(max(lens) + N) // P)
    cache = rand_cache(api, B * W, H, P, D, 121)
    table = rand_table(B, W, B * W, 122)
    q = (torch.randn(B, N, H * G, D, generator=gen(123)) * 2).to(BF).cuda()
    check_attend(api, q, cache, table, lens, n_query=[N, N, max(N - 1, 0), N, 0], mask=tree_mask(B, N, 124) if tree else None, cap=cap)


def test_attend_pool_past_two_gigabytes(api):
    H, P, D = 1, 256, 128
    pages = (1 << 31) // (H * P * D) + 3
    pool = [torch.zeros(pages, H, P, D, dtype=torch.uint8, device="cuda").view(ref.F8) for _ in range(2)]
    cache = pool + [torch.full((pages, H), 2.0 ** -6, device="cuda") for _ in range(2)]
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    few = rand_cache(api, 3, H, P, D, 34)
    for to, frm in zip(cache, few):
        to.view(torch.uint8)[table[0].long()] = frm.view(torch.uint8) if to.dtype == ref.F8 else frm.view(torch.uint8)
    q = torch.randn(1, 4, 2, D, generator=gen(35)).to(BF).cuda()
    small = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    a = api.spec_cache_attend(q, cache, table, torch.tensor([700], dtype=torch.int32, device="cuda"))
    b = api.spec_cache_attend(q, few, small, torch.tensor([700], dtype=torch.int32, device="cuda"))
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    k = torch.randn(1, 9, H, D, generator=gen(36)).to(BF).cuda()
    ln = torch.tensor([250], dtype=torch.int32, device="cuda")
    api.spec_cache_append(cache, table, ln, k, k)
    api.spec_cache_append(few, small, ln, k, k)
    for x, y in zip(cache, few):
        assert torch.equal(x.view(torch.uint8)[table[0].long()], y.view(torch.uint8))


def test_attend_is_the_same_on_every_run_and_stream(api):
    B, N, H, G, D, P = 4, 9, 2, 4, 128, 64
    W = 40
    cache = rand_cache(api, B * W, H, P, D, 37)
    table = rand_table(B, W, B * W, 38)
    ln = torch.tensor([2500, 17, 900, 1300], dtype=torch.int32, device="cuda")
    q = torch.randn(B, N, H * G, D, generator=gen(39)).to(BF).cuda()
    first = api.spec_cache_attend(q, cache, table, ln)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            again = api.spec_cache_attend(q, cache, table, ln)
        side.synchronize()
        assert torch.equal(first["out"], again["out"]) and torch.equal(first["lse"], again["lse"])


def test_all_in_a_graph(api):
    """The four operators captured and replayed on new data of the same shapes."""
    B, N, H, G, D, P, W = 2, 5, 2, 2, 64, 16, 8
    cache = rand_cache(api, B * W + B * 2, H, P, D, 40)
    every = torch.randperm(B * W + B * 2, generator=gen(41)).to(torch.int32).cuda()
    table, dst = every[:B * W].reshape(B, W), every[B * W:].reshape(B, 2)
    ln = torch.tensor([40, 61], dtype=torch.int32, device="cuda")
    k, v, q = (torch.randn(B, N, h, D, generator=gen(42 + h)).to(BF).cuda() for h in (H, H, H * G))
    prev = torch.zeros(B, H, W * P, device="cuda")

    def step():
        a = api.spec_cache_append(cache, table, ln, k, v)
        o = api.spec_cache_attend(q, cache, table, ln)
        w = api.spec_cache_weights(q, o["lse"], cache, table, ln, prev=prev)
        e = api.spec_cache_evict(cache, table, a["new_len"], w["weights"], 20, 5, dst)
        return a, o, w, e

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    k.copy_(torch.randn(B, N, H, D, generator=gen(50)))
    q.copy_(torch.randn(B, N, H * G, D, generator=gen(51)))
    ln += 3
    graph.replay()
    torch.cuda.synchronize()
    kept = [{n: t.clone() for n, t in x.items()} for x in captured]
    eager = step()
    for x, y in zip(kept, eager):
        for name in x:
            assert torch.equal(x[name], y[name]), name


# ------------------------------------------------------------------ weights

@pytest.mark.parametrize("B,N,H,G,D,P,lens", [(1, 1, 1, 1, 128, 64, [0]), (2, 1, 2, 4, 128, 64, [63, 700]), (3, 5, 1, 8, 64, 16, [0, 15, 1000]),
                                              (1, 40, 2, 4, 128, 128, [333]), (2, 3, 2, 2, 80, 32, [31, 64]), (1, 70, 1, 8, 128, 64, [129])])
@pytest.mark.parametrize("dtype,cap,path", [(BF, 0.0, False), (HF, 0.0, True), (BF, 20.0, True)])
def test_weights(api, B, N, H, G, D, P, lens, dtype, cap, path):
    W = -(-(max(lens) + N) // P)
    cache = rand_cache(api, B * W, H, P, D, 60)
    table = rand_table(B, W, B * W, 61)
    g = gen(62)
    q = torch.randn(B, N, H * G, D, generator=g).to(dtype).cuda()
    lse = (torch.rand(B, N, H * G, generator=g) * 3 + 3).cuda()
    lse[0, 0, 0] = -math.inf
    prev = torch.rand(B, H, W * P, generator=g).cuda()
    index = counts = None
    cnt = [N] * B
    if path:
        index = torch.stack([torch.randperm(N, generator=g).sort().values for _ in range(B)]).to(torch.int32).cuda()
        cnt = [int(torch.randint(0, N + 1, (1,), generator=g)) for _ in range(B)]
        counts = torch.tensor(cnt, dtype=torch.int32, device="cuda")
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o = api.spec_cache_weights(q, lse, cache, table, ln, prev=prev, counts=counts, index=index, softcap=cap)
    want, tol = ref.weights(ref.Cache64(cache, table), q, lse, lens, cnt, index, D ** -0.5, cap, prev)
    got = o["weights"].cpu().double()
    assert o["status"].tolist() == [0] * B
    worst = (got - want).abs() / tol
    assert bool((worst <= 1).all()), float(worst.max())
    for b in range(B):
        assert torch.equal(o["weights"][b, :, lens[b] + cnt[b]:], prev[b, :, lens[b] + cnt[b]:])  # not written
    again = api.spec_cache_weights(q, lse, cache, table, ln, prev=prev, counts=counts, index=index, softcap=cap, out=dict(weights=prev))
    assert torch.equal(again["weights"], o["weights"])  # in place
    fresh = api.spec_cache_weights(q, lse, cache, table, ln, counts=counts, index=index, softcap=cap)
    assert fresh["weights"].shape == prev.shape


@pytest.mark.parametrize("D", [64, 80, 128])
def test_weights_of_normalisers_in_any_strides(api, D):
    """Heads outermost, a slice of wider rows, one request's for all: the same bits as of a contiguous copy."""
    B, N, H, G, P, W = 3, 5, 2, 3, 32, 9
    cache = rand_cache(api, B * W, H, P, D, 110)
    table = rand_table(B, W, B * W, 111)
    g = gen(112)
    q = torch.randn(B, N, H * G, D, generator=g).to(BF).cuda()
    ln = torch.tensor([0, 100, 283], dtype=torch.int32, device="cuda")
    wide = (torch.rand(H * G + 1, N, 2 * B, generator=g) * 3 + 3).cuda()
    for lse in (wide[1:, :, ::2].permute(2, 1, 0), wide.reshape(2 * B, N, H * G + 1)[1:B + 1, :, 1:], wide[:-1, :, 1].T.expand(B, N, H * G)):
        assert lse.shape == (B, N, H * G) and not lse.is_contiguous()
        got = api.spec_cache_weights(q, lse, cache, table, ln)
        want = api.spec_cache_weights(q, lse.contiguous(), cache, table, ln)
        assert got["status"].tolist() == [0] * B and torch.equal(got["weights"], want["weights"])
        assert bool((got["weights"].sum(-1) > 0).all())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,rows", [(64, 1), (64, 9), (80, 1), (128, 2), (128, 40)])
def test_small_capped_scores_keep_their_digits(api, D, rows, dtype):
    """Scores of one product each, so known exactly, far below the cap and around half of it: their weights to a few roundings."""
    T, P, cap, scale = 256, 128, 30.0, 2.0 ** -4
    codes = torch.zeros(2, 1, P, D, dtype=torch.uint8)
    codes[..., 0] = torch.cat([torch.arange(0, 0x7f), torch.arange(0x80, 0xff), torch.zeros(2)]).reshape(2, 1, P).to(torch.uint8)
    k = codes.cuda().view(ref.F8)
    one = torch.ones(2, 1, device="cuda")
    cache = [k, k.clone(), one, one.clone()]
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    q = torch.zeros(1, rows, 1, D, dtype=dtype, device="cuda")
    q[..., 0] = 1.0
    # all rows see the context alone: no tokens of their own among the positions
    lens = torch.tensor([T - rows], dtype=torch.int32, device="cuda")
    lse = torch.full((1, rows, 1), 2.0, device="cuda")
    w = api.spec_cache_weights(q, lse, cache, table, lens, scale=scale, softcap=cap)["weights"][0, 0].cpu().double()
    x = k.reshape(T, D)[:, 0].cpu().double() * scale
    s = cap * torch.tanh(x / cap)
    seen = torch.tensor([rows if j < T - rows else T - j for j in range(T)]).double()
    want = seen * torch.exp(s - 2.0)
    # a score: the polynomial, 8 roundings, and past half the cap a quotient of exponentials to 2^-20 of the cap; the weight: the
    # exponent's roundings and the exponential's
    off = s.abs() * (3e-8 + 8 * 2.0 ** -24) + torch.where(x.abs() > 14.9, cap * 2.0 ** -20, 0.0)
    off += (s.abs() + 2.0) * 1.4427 * 2.0 ** -22 + 2.0 ** -21 + rows * 2.0 ** -24
    worst = ((w - want).abs() / (want * off)).max()
    assert worst <= 1, float(worst)
    o = api.spec_cache_attend(q[:, :1].contiguous(), cache, table, torch.tensor([T - 1], dtype=torch.int32, device="cuda"), scale=scale, softcap=cap)
    # the largest scores rule the sum: at 448 / 16 those are past half the cap
    assert abs(float(o["lse"]) - float(torch.logsumexp(s, 0))) <= cap * 2.0 ** -20 + 30 * 2.0 ** -22


@pytest.mark.parametrize("N,D", [(1, 64), (3, 64), (1, 128), (9, 128), (20, 128)])
def test_normalisers_of_small_capped_scores(api, N, D):
    """Two positions or so, scores near zero: the normaliser is off by a few roundings of 1."""
    G, P, cap = 4, 16, 30.0
    codes = torch.zeros(2, 1, P, D, dtype=torch.uint8)
    codes[..., 0] = torch.randint(0, 0x38, (2, 1, P), generator=gen(120)).to(torch.uint8)
    k = codes.cuda().view(ref.F8)
    one = torch.ones(2, 1, device="cuda")
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    q = torch.zeros(1, N, G, D, dtype=BF, device="cuda")
    q[..., 0] = torch.rand(1, N, G, generator=gen(121)).to(BF).cuda()
    o = api.spec_cache_attend(q, [k, k.clone(), one, one.clone()], table, torch.tensor([1], dtype=torch.int32, device="cuda"), scale=1.0, softcap=cap)
    x = q[0, ..., 0].cpu().double()[..., None] * k.flip(0).reshape(2 * P, D)[:, 0].cpu().double()
    s = cap * torch.tanh(x / cap)
    for i in range(N):
        want = torch.logsumexp(s[i, :, :i + 2], -1)
        # (scores up to 1, sums up to 21 e: roundings of the score, the exponentials, the sum and the logarithm)
        assert bool(((o["lse"][0, i].cpu().double() - want).abs() <= 3e-8 + 16 * 2.0 ** -24 + 2.0 ** -21 + want.abs() * 2.0 ** -22).all())


def test_weights_of_an_attention_sum_to_its_rows(api):
    """Every row's weights sum to 1: the operators agree on what a score is."""
    B, N, H, G, D, P, W = 2, 4, 2, 3, 128, 64, 5
    cache = rand_cache(api, B * W, H, P, D, 63)
    table = rand_table(B, W, B * W, 64)
    ln = torch.tensor([200, 31], dtype=torch.int32, device="cuda")
    q = torch.randn(B, N, H * G, D, generator=gen(65)).to(BF).cuda()
    o = api.spec_cache_attend(q, cache, table, ln, softcap=15.0)
    w = api.spec_cache_weights(q, o["lse"], cache, table, ln, softcap=15.0)
    # the two kernels' scores differ by at most what the attention's q is rounded by (2^-18 of a row's largest, 4096 by 128 terms)
    assert bool(((w["weights"].double().sum(2) - N * G).abs() < N * G * 2.0 ** -9).all())


# ------------------------------------------------------------------ evict

def check_evict(api, B, H, D, P, lens, keep, recent, weights, seed=70, **kw):
    W = max(1, -(-max(lens) // P))
    Wd = -(-keep // P)
    cache = rand_cache(api, B * (W + Wd), H, P, D, seed)
    every = torch.randperm(B * (W + Wd), generator=gen(seed + 1)).to(torch.int32).cuda()
    table, dst = every[:B * W].reshape(B, W).contiguous(), every[B * W:].reshape(B, Wd).contiguous()
    before, after = ref.Cache64(cache, table), ref.Cache64(cache, dst)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o = api.spec_cache_evict(cache, table, ln, weights, keep, recent, dst, **kw)
    got = ref.Cache64(cache, dst)
    assert o["status"].tolist() == [0] * B
    host = weights.cpu()
    for b in range(B):
        n = min(keep, lens[b])
        assert int(o["new_len"][b]) == n
        kept = ref.evict(before, host, b, lens[b], keep, recent)
        for h in range(H):
            assert o["kept"][b, h].tolist() == kept[h] + [-1] * (keep - n)
            assert torch.equal(o["weights"][b, h, :n].cpu(), host[b, h][kept[h]]) or bool(host[b, h][kept[h]].isnan().any())
            assert bool((o["weights"][b, h, n:] == 0).all())
        for which in (0, 1):
            rows = before.rows(which, b, lens[b])
            for w in range(-(-n // P)):
                page, m = int(dst[b, w]), min(P, n - w * P)
                for h in range(H):
                    part = rows[h][kept[h][w * P:w * P + m]]
                    s = ref.block_scale(part)
                    after.scale[which][page, h] = s
                    after.val[which][page, h, :m] = ref.e4m3(part / s)
    for which in (0, 1):
        assert torch.equal(got.val[which], after.val[which]) and torch.equal(got.scale[which], after.scale[which])
    return o


@pytest.mark.parametrize("D,P,H", [(128, 64, 2), (64, 16, 3), (80, 32, 1), (256, 256, 1)])
@pytest.mark.parametrize("lens,keep,recent", [([100, 1, 0], 33, 5), ([257, 64, 65], 64, 64), ([31, 400, 300], 1, 0), ([500, 499, 7], 600, 3),
                                              ([90, 91, 92], 90, 0)])
def test_evict(api, D, P, H, lens, keep, recent):
    w = torch.rand(3, H, max(lens), generator=gen(71)).cuda()
    check_evict(api, 3, H, D, P, lens, keep, recent, w)


@pytest.mark.parametrize("kind", ["equal", "few", "signs", "nan", "tiny"])
def test_evict_ties_and_odd_weights(api, kind):
    B, H, T = 2, 2, 1500
    g = gen(72)
    w = {"equal": torch.ones(B, H, T), "few": torch.randint(0, 3, (B, H, T), generator=g).float(),
         "signs": torch.randn(B, H, T, generator=g).round(), "nan": torch.rand(B, H, T, generator=g),
         "tiny": torch.rand(B, H, T, generator=g) * 1e-42}[kind]
    if kind == "nan":
        w[:, :, ::3] = math.nan
        w[:, :, 1] = math.inf
        w[:, :, 2] = -math.inf
    if kind == "signs":
        w[:, :, ::2] = -0.0
    check_evict(api, B, H, 64, 32, [T, T - 100], 1200, 7, w.cuda())


def test_evict_long(api):
    T = 70001
    w = torch.exp(torch.randn(1, 2, T + 13, generator=gen(73))).cuda()
    check_evict(api, 1, 2, 64, 256, [T], 4097, 100, w)


def test_evict_to_another_pool_and_strided_weights(api):
    B, H, D, P, T, keep = 2, 2, 64, 16, 50, 20
    cache = rand_cache(api, 8, H, P, D, 74)
    pool = api.spec_cache_new(4, H, P, D)
    table, dst = rand_table(B, 4, 8, 75), rand_table(B, 2, 4, 76)
    room = torch.rand(B, T + 3, H, generator=gen(77)).cuda().transpose(1, 2).contiguous()
    big = torch.zeros(B, 2 * H, T + 9, device="cuda")
    big[:, ::2, :T + 3] = room
    w = big[:, ::2, :T + 3]
    ln = torch.tensor([T, 9], dtype=torch.int32, device="cuda")
    o = api.spec_cache_evict(cache, table, ln, w, keep, 4, dst, dst_cache=pool)
    before, got = ref.Cache64(cache, table), ref.Cache64(pool, dst)
    for b, n in ((0, T), (1, 9)):
        for h, kept in enumerate(ref.evict(before, w.cpu(), b, n, keep, 4)):
            assert o["kept"][b, h, :len(kept)].tolist() == kept
            for which in (0, 1):
                part = before.rows(which, b, n)[h][kept]
                want = [ref.e4m3(x / ref.block_scale(x)) * ref.block_scale(x) for x in part.split(P)]
                assert torch.equal(got.rows(which, b, len(kept))[h], torch.cat(want))


# ------------------------------------------------------------------ requests that are wrong

def wrong_requests(api):
    """Three requests, the second in turn wrong in each way: (lens, counts or rows, table change, index change, status)."""
    return [("length", api.STATUS_BAD_LENGTH), ("negative", api.STATUS_BAD_LENGTH), ("count", api.STATUS_BAD_LENGTH),
            ("page", api.STATUS_BAD_PAGE), ("page below", api.STATUS_BAD_PAGE), ("index", api.STATUS_BAD_INDEX)]


@pytest.mark.parametrize("kind", ["length", "negative", "count", "page", "page below", "index"])
def test_wrong_requests_leave_the_others_alone(api, kind):
    status = dict(wrong_requests(api))[kind]
    B, N, H, G, D, P, W = 3, 6, 2, 2, 128, 16, 6
    clean = rand_cache(api, B * W + B, H, P, D, 80)
    every = torch.randperm(B * W + B, generator=gen(81)).to(torch.int32).cuda()
    table, dst = every[:B * W].reshape(B, W).contiguous(), every[B * W:].reshape(B, 1).contiguous()
    lens = torch.tensor([50, 60, 70], dtype=torch.int32, device="cuda")
    counts = torch.tensor([6, 5, 4], dtype=torch.int32, device="cuda")
    index = torch.arange(N, dtype=torch.int32, device="cuda").repeat(B, 1).contiguous()
    k = torch.randn(B, N, H, D, generator=gen(82)).to(BF).cuda()
    q = torch.randn(B, N, H * G, D, generator=gen(83)).to(BF).cuda()
    w = torch.rand(B, H, W * P, generator=gen(84)).cuda()
    lse = torch.full((B, N, H * G), 4.0, device="cuda")

    def all_four(lens, counts, table, index):
        cache = [x.clone() for x in clean]
        a = api.spec_cache_append(cache, table, lens, k, k, counts=counts, index=index)
        o = api.spec_cache_attend(q, cache, table, lens, n_query=counts)
        s = api.spec_cache_weights(q, lse, cache, table, lens, prev=w, counts=counts, index=index)
        e = api.spec_cache_evict(cache, table, lens, w, 12, 3, dst)
        return cache, a, o, s, e

    good = all_four(lens, counts, table, index)
    if kind == "length":
        lens = lens.clone()
        lens[1] = W * P + 1
    elif kind == "negative":
        lens = lens.clone()
        lens[1] = -1
    elif kind == "count":
        counts = counts.clone()
        counts[1] = N + 1
    elif kind == "index":
        index = index.clone()
        index[1, 2] = N
    else:
        table = table.clone()
        table[1, 3] = -1 if kind == "page below" else B * W + B
    bad = all_four(lens, counts, table, index)
    _, a, o, s, e = bad
    assert a["status"].tolist() == [0, status, 0] and int(a["new_len"][1]) == int(lens[1])
    assert s["status"].tolist() == [0, status, 0] and torch.equal(s["weights"][1], w[1])
    if kind != "index":
        assert o["status"].tolist() == [0, status, 0]
        assert bool((o["out"][1] == 0).all()) and bool((o["lse"][1] == -math.inf).all())
    if kind not in ("index", "count"):
        assert e["status"].tolist() == [0, status, 0] and int(e["new_len"][1]) == 0 and bool((e["kept"][1] == -1).all())
    for i in (0, 2):
        for x, y in zip(good[1:], bad[1:]):
            for name in x:
                assert torch.equal(x[name][i], y[name][i]), (kind, name)


def test_bindings_refuse(api):
    cache = rand_cache(api, 4, 2, 16, 64, 90)
    table = rand_table(2, 2, 4, 91)
    ln = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = torch.zeros(2, 3, 4, 64, dtype=BF, device="cuda")
    with pytest.raises(TypeError):
        api.spec_cache_attend(q.float(), cache, table, ln)
    with pytest.raises(ValueError):
        api.spec_cache_attend(q[..., :32], cache, table, ln)
    with pytest.raises(TypeError):
        api.spec_cache_attend(q, cache, table.long(), ln)
    with pytest.raises(TypeError):
        api.spec_cache_attend(q, cache, table, ln, mask=torch.ones(2, 3, 2, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        api.spec_cache_attend(q, [cache[0].transpose(1, 2), *cache[1:]], table, ln)
    with pytest.raises(api.SpecError):
        api.spec_cache_attend(q[:, :, :3], cache, table, ln)  # 3 query heads over 2
    with pytest.raises(ValueError):
        api.spec_cache_append(cache, table, ln, q, q[:, :, :2])
    with pytest.raises(api.SpecError):
        api.spec_cache_evict(cache, table, ln, torch.zeros(2, 2, 32, device="cuda"), 0, 0, table)
    with pytest.raises(TypeError):
        api.spec_cache_evict(cache, table, ln, torch.zeros(2, 3, 32, device="cuda"), 4, 0, table)


@pytest.mark.parametrize("name", ["new_len", "status", "kept", "weights", "lse", "out"])
def test_bindings_refuse_outputs_that_do_not_fit(api, name):
    cache = rand_cache(api, 4, 2, 16, 64, 92)
    table = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    ln = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    q = torch.zeros(2, 3, 4, 64, dtype=BF, device="cuda")
    w = torch.zeros(2, 2, 16, device="cuda")
    a = api.spec_cache_append(cache, table, ln, q[:, :, :2], q[:, :, 2:])
    o = api.spec_cache_attend(q, cache, table, ln)
    s = api.spec_cache_weights(q, o["lse"], cache, table, ln, prev=w)
    e = api.spec_cache_evict(cache, table, ln, w, 4, 0, table + 2)
    calls = [(a, lambda x: api.spec_cache_append(cache, table, ln, q[:, :, :2], q[:, :, 2:], out=x)),
             (o, lambda x: api.spec_cache_attend(q, cache, table, ln, out=x)),
             (s, lambda x: api.spec_cache_weights(q, o["lse"], cache, table, ln, prev=w, out=x)),
             (e, lambda x: api.spec_cache_evict(cache, table, ln, w, 4, 0, table + 2, out=x))]
    tried = 0
    for good, call in calls:
        call(good)
        if name not in good:
            continue
        for bad in (good[name][:1], good[name].double(), good[name].cpu()):
            tried += 1
            with pytest.raises((TypeError, ValueError)):
                call(dict(good, **{name: bad}))
    assert tried >= 3


def test_workspace_of_the_caller_and_of_a_stream(api):
    """Too small a workspace of the caller's is refused; a stream's own grows."""
    B, N, H, G, P, D, W = 2, 9, 2, 4, 64, 128, 40
    cache = rand_cache(api, B * W, H, P, D, 99)
    table = rand_table(B, W, B * W, 100)
    ln = torch.tensor([2500, 1200], dtype=torch.int32, device="cuda")
    q = torch.randn(B, N, H * G, D, generator=gen(101)).to(BF).cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    few = api.spec_cache_attend(q[:, :1].contiguous(), cache, table, ln, stream=side)
    got = api.spec_cache_attend(q, cache, table, ln, stream=side)
    side.synchronize()
    cs = api._cache_struct(cache, table, B, q.device)[0]
    need = api.lib().spec_cache_workspace_size(api.OP_CACHE_ATTEND, cs, B, N, H * G)
    assert need > 0 and few["status"].tolist() == [0, 0]
    with pytest.raises(api.SpecError):
        api.spec_cache_attend(q, cache, table, ln, ws=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    own = api.spec_cache_attend(q, cache, table, ln, ws=torch.empty(need, dtype=torch.uint8, device="cuda"))
    for x in ("out", "lse", "status"):
        assert torch.equal(got[x], own[x]), x


def test_a_call_belongs_to_its_stream(api):
    """What a call copies or fills first is done on the stream it is given, whatever the current one is busy with."""
    B, N, H, G, P, D, W = 2, 4, 2, 2, 32, 64, 5
    cache = rand_cache(api, B * W, H, P, D, 93)
    table = rand_table(B, W, B * W, 94)
    ln = torch.tensor([100, 37], dtype=torch.int32, device="cuda")
    q = torch.randn(B, N, H * G, D, generator=gen(95)).to(BF).cuda()
    mask = tree_mask(B, N, 96).transpose(1, 2).contiguous().cuda().transpose(1, 2)  # a copy is taken of it
    prev = torch.rand(B, H, W * P, generator=gen(97)).cuda()

    def calls(**kw):
        o = api.spec_cache_attend(q, cache, table, ln, mask=mask, **kw)
        yield o
        yield api.spec_cache_weights(q, want["lse"], cache, table, ln, prev=prev, **kw)
        yield api.spec_cache_weights(q, want["lse"], cache, table, ln, **kw)
        yield api.spec_cache_evict(cache, table, ln, prev, 20, 4, dst, dst_cache=other, **kw)
        yield api.spec_cache_append(other, table, ln, q[:, :, :2], q[:, :, 2:], **kw)

    other = rand_cache(api, B * W, H, P, D, 98)
    dst = table[:, :1].contiguous()
    want = api.spec_cache_attend(q, cache, table, ln, mask=mask)
    first = list(calls())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    second = list(calls(stream=side))
    side.synchronize()
    with torch.cuda.stream(side):
        got = [{k: t.cpu() for k, t in o.items()} for o in second]
    torch.cuda.synchronize()
    for x, y, z in zip(first, got, second):
        for k in x:
            assert torch.equal(x[k].cpu(), y[k]) and torch.equal(x[k], z[k]), k


def test_weights_without_rows_copies_prev(api):
    """counts of 0: out is prev over the context, whatever out held."""
    cache = rand_cache(api, 8, 2, 64, 128, 66)
    table = rand_table(2, 4, 8, 67)
    ln = torch.tensor([150, 0], dtype=torch.int32, device="cuda")
    q = torch.randn(2, 3, 4, 128, generator=gen(68)).to(BF).cuda()
    lse = torch.zeros(2, 3, 4, device="cuda")
    prev = torch.rand(2, 2, 256, generator=gen(69)).cuda()
    out = torch.full((2, 2, 256), -7.0, device="cuda")
    api.spec_cache_weights(q, lse, cache, table, ln, prev=prev, counts=torch.zeros(2, dtype=torch.int32, device="cuda"), out=dict(weights=out))
    assert torch.equal(out[0, :, :150], prev[0, :, :150]) and bool((out[0, :, 150:] == -7).all()) and bool((out[1] == -7).all())


@pytest.mark.parametrize("N,G,D,dtype", [(1, 1, 128, BF), (40, 8, 64, HF), (7, 3, 128, HF)])
def test_weights_many_requests(api, N, G, D, dtype):
    """More requests than a launch takes, most of them short, some without rows."""
    B, H, P = 300, 1, 16
    g = gen(95)
    lens = torch.randint(0, 60, (B,), generator=g).tolist()
    lens[7] = 700
    cnt = torch.randint(0, N + 1, (B,), generator=g).tolist()
    W = -(-(700 + N) // P)
    cache = rand_cache(api, B * W, H, P, D, 96)
    table = rand_table(B, W, B * W, 97)
    q = torch.randn(B, N, H * G, D, generator=g).to(dtype).cuda()
    lse = (torch.rand(B, N, H * G, generator=g) * 3 + 3).cuda()
    prev = torch.rand(B, H, W * P, generator=g).cuda()
    o = api.spec_cache_weights(q, lse, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), prev=prev,
                               counts=torch.tensor(cnt, dtype=torch.int32, device="cuda"))
    want, tol = ref.weights(ref.Cache64(cache, table), q, lse, lens, cnt, None, D ** -0.5, 0.0, prev)
    assert bool(((o["weights"].cpu().double() - want).abs() <= tol).all())


@pytest.mark.parametrize("N,G,D,dtype", [(1, 1, 128, BF), (3, 16, 64, HF), (9, 4, 128, BF), (70, 2, 64, BF)])
def test_attend_many_requests(api, N, G, D, dtype):
    """More requests than a launch takes, most of them of a tile or two, so that a CTA goes through many units."""
    B, H, P = 300, 2, 16
    g = gen(98)
    lens = torch.randint(0, 200, (B,), generator=g).tolist()
    lens[3] = 900
    nq = torch.randint(0, N + 1, (B,), generator=g).tolist()
    W = -(-(900 + N) // P)
    cache = rand_cache(api, B * W, H, P, D, 99)
    table = rand_table(B, W, B * W, 100)
    q = torch.randn(B, N, H * G, D, generator=g).to(dtype).cuda()
    check_attend(api, q, cache, table, lens, n_query=nq)


def test_the_whole_step(api):
    """The example's step: what is committed, weighed and kept is what the definitions give on its own inputs."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "cached_tree_step.py")
    spec = importlib.util.spec_from_file_location("cached_tree_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    r = example.step(context=300, keep=90, recent=20, page=64, seed=3)
    torch.cuda.synchronize()
    n_emit = r["verdict"]["n_emit"]
    assert torch.equal(r["committed"]["new_len"], r["length"] + n_emit)
    for name in ("attended", "committed", "weights", "kept", "drafted"):
        assert r[name]["status"].tolist() == [0] * 4
    # committed rows are the path's, rounded at their block's scale
    c64 = ref.Cache64(r["cache"], r["table"])
    for b in range(4):
        n, base = int(n_emit[b]), int(r["length"][b])
        nodes = r["verdict"]["path_nodes"][b, :n].long()
        for which, x in ((0, r["k"]), (1, r["v"])):
            got = c64.rows(which, b, base + n)[:, base:]
            want = x[b, nodes].cpu().double().transpose(0, 1)
            scale = torch.stack([c64.scale[which][c64.table[b, (base + i) // 64]] for i in range(n)], 1)[:, :, None]
            assert torch.equal(got, ref.e4m3(want / scale) * scale)
    # weights of the accepted rows sum to their number; what is kept are the definition's positions
    G = r["q"].shape[2] // r["k"].shape[2]
    total = r["weights"]["weights"].double().sum(2)
    assert bool(((total - n_emit[:, None].double() * G).abs() < 0.02 * G * n_emit[:, None].double()).all())
    w = r["weights"]["weights"].cpu()
    for b in range(4):
        T = int(r["committed"]["new_len"][b])
        for h, kept in enumerate(ref.evict(c64, w, b, T, 90, 20)):
            assert r["kept"]["kept"][b, h, :len(kept)].tolist() == kept
    out, lse, t_out, t_lse = ref.attend(ref.Cache64(r["cache"], r["small_table"]), r["q1"], r["kept"]["new_len"].tolist(), [1] * 4, None,
                                        128 ** -0.5, 0.0)
    assert bool(((r["drafted"]["out"].cpu().double() - out).abs() <= t_out).all())
