"""The paged 8-bit cache: its plan (equal to the oracle's), the write of new tokens (equal byte for byte)
and one-token attention over it (within bounds that follow from the kernel's arithmetic)."""
import numpy as np
import pytest
import torch

from oracle import attention as oa
from tests import attn_bounds as ab

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.init()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def pages_of(lens, page):
    return [-(-int(x) // page) for x in lens]


def table_of(lens, page, width, seed, spare=3):
    """A block table of shuffled pages for `lens` tokens, and the pages left over."""
    order = np.random.RandomState(seed).permutation(sum(pages_of(lens, page)) + spare)
    table, at = np.full((len(lens), width), -1), 0
    for r, n in enumerate(pages_of(lens, page)):
        table[r, :n] = order[at:at + n]
        at += n
    return table, order[at:]


def filled_cache(P, Hk, page, d, seed):
    """Random finite bytes with power-of-two scales."""
    r = np.random.RandomState(seed)
    c = r.randint(0, 127, (P, Hk, page, d)) | (r.randint(0, 2, (P, Hk, page, d)) << 7)
    return c.astype(np.uint8), 2.0 ** r.randint(-9, -5, (P, Hk))


# ---- plan ----------------------------------------------------------------------------------------

def plan_both(lens, added, table, free, head, page, rows):
    import linear_attention_sequence_rule_b200 as gdn
    t = i32(table)
    p = gdn.cache_plan(i32(lens), i32(added), t, i32(free), i32([head]), page, rows)
    torch.cuda.synchronize()
    want = oa.plan(lens, added, table, free, head, page, rows)
    got = dict(p._asdict(), table=t)
    for name, w in want.items():
        assert np.array_equal(got[name].cpu().numpy().ravel(), np.asarray(w).ravel()), name
    return p


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("n,hi,new", [(1, 0, 1), (1, 100, 1), (7, 300, 1), (256, 500, 1), (33, 0, 700), (9, 200, 300),
                                      (1500, 90, 3)])
def test_plan(n, hi, new, page):
    r = np.random.RandomState(n + page)
    lens, added = r.randint(0, hi + 1, n), r.randint(0, new + 1, n)
    width = (hi + new) // page + 2
    table, left = table_of(lens, page, width, seed=n, spare=sum(pages_of(lens + added, page)))
    plan_both(lens, added, table, np.concatenate([[77], left]), 1, page, int(added.sum()) + n % 3)


def test_plan_of_the_longest_batch():
    r = np.random.RandomState(0)
    n, page = 16384, 16
    lens, added = r.randint(0, 40, n), r.randint(0, 4, n)
    table, left = table_of(lens, page, 4, seed=1, spare=n)
    plan_both(lens, added, table, left, 0, page, int(added.sum()) + 5)


@pytest.mark.parametrize("case", ["pages", "row", "negative", "rows", "head", "huge"])
def test_plan_refuses_as_a_whole(case):
    lens, added, page, rows, head = [3, 20, 0], [14, 1, 40], 16, 60, 0
    table, left = table_of(lens, page, 4, seed=2, spare=5)
    free = left[:3 if case == "pages" else 5]
    if case == "row":
        added = [14, 50, 40]
    if case == "negative":
        lens = [3, -1, 0]
    if case == "rows":
        rows = 54
    if case == "head":
        head = 6
    if case == "huge":
        added = [14, 2 ** 31 - 1, 2 ** 31 - 1]
    p = plan_both(lens, added, table, free, head, page, rows)
    assert p.status[0].item() != 0


def test_plan_in_place_and_empty():
    import linear_attention_sequence_rule_b200 as gdn
    lens, head = i32([3, 16, 0]), i32([0])
    table, left = table_of([3, 16, 0], 16, 3, seed=3, spare=9)
    t = i32(table)
    for _ in range(40):  # lens and free_head updated in place, one token a step
        p = gdn.cache_plan(lens, i32([1, 0, 0]), t, i32(left), head, 16, 4, lens_out=lens, free_head_out=head)
    assert lens.tolist() == [43, 16, 0] and head.tolist() == [2] and p.positions.tolist() == [42, -1, -1, -1]
    few = i32([7, 0, 9, 8, 7])  # the single numbers may lie anywhere
    p = gdn.cache_plan(lens, i32([0, 0, 0]), t, i32(left), few[1:2], 16, 0, free_head_out=few[1:2], status=few[2:4])
    assert few.tolist() == [7, 0, 0, 0, 7]
    p = gdn.cache_plan(lens, i32([0, 0, 0]), t, i32([]), i32([0]), 16, 0)
    assert p.status.tolist() == [0, 0] and p.slots.numel() == 0 and p.cu_seqlens.tolist() == [0] * 4


# ---- append --------------------------------------------------------------------------------------

def append_both(x, y, slots, kc, ks, vc, vs, dtype):
    import linear_attention_sequence_rule_b200 as gdn
    dev = [torch.from_numpy(c).cuda().view(torch.float8_e4m3fn) for c in (kc, vc)]
    sc = [torch.from_numpy(s).float().cuda() for s in (ks, vs)]
    gdn.cache_append(x.cuda(), y.cuda(), i32(slots), dev[0], dev[1], sc[0], sc[1])
    torch.cuda.synchronize()
    for rows, c, s, gc, gs in ((x, kc, ks, dev[0], sc[0]), (y, vc, vs, dev[1], sc[1])):
        wc, ws = oa.append(rows, slots, c, s)
        assert np.array_equal(gs.double().cpu().numpy(), ws)
        gb, nan = gc.view(torch.uint8).cpu().numpy(), (wc & 127) == 127
        assert np.array_equal(gb[~nan], wc[~nan]) and ((gb[nan] & 127) == 127).all()
    return dev, sc


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page,Hk", [(64, 16, 3), (64, 128, 1), (128, 32, 2), (128, 64, 2), (64, 64, 1)])
@pytest.mark.parametrize("kind", ["step", "prompts", "mixed"])
def test_append(kind, d, page, Hk, dtype):
    r = np.random.RandomState(page + d)
    n = 40 if kind == "step" else 6
    lens = np.zeros(n, int) if kind == "prompts" else r.randint(0, 3 * page, n)
    added = np.ones(n, int) if kind == "step" else r.randint(0, 3 * page + 5, n)
    width = max(pages_of(lens + added, page)) + 1
    table, left = table_of(lens, page, width, seed=5, spare=sum(pages_of(added, page)) + n)
    p = oa.plan(lens, added, table, left, 0, page, int(added.sum()) + 2)
    P = int(max(p["table"].max(), left.max())) + 1
    kc, ks = filled_cache(P, Hk, page, d, 6)
    vc, vs = filled_cache(P, Hk, page, d, 7)
    g = torch.Generator().manual_seed(8)
    rows = len(p["slots"])
    mag = torch.exp2(torch.randint(-6, 8, (rows, Hk, 1), generator=g).float())
    x, y = ((torch.randn(rows, Hk, d, generator=g) * mag).to(DT[dtype]) for _ in range(2))
    append_both(x, y, p["slots"], kc, ks, vc, vs, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_extremes(dtype):
    """Zeros, the smallest and largest values, infinities and NaN; growth of the scale over all of e4m3."""
    d, page = 64, 16
    x = torch.zeros(12, 1, d)
    x[1, 0, :3] = torch.tensor([1e-30, 1e-12, -1e-18])
    x[2, 0, 5] = float("nan")
    x[3, 0, :2] = torch.tensor([float("inf"), 1.0])
    x[5, 0] = torch.linspace(-449, 449, d)
    x[6, 0, 0] = 3e38
    x[8, 0, 1] = 2.0 ** -120
    x[9:] = torch.randn(3, 1, d, generator=torch.Generator().manual_seed(1))
    # pages 0..6: runs of 1, 2, 1, ... rows, some behind tokens that are held
    slots = [0, 17, 18, 35, 48, 49, 66, 80, 96, 7, 8, 9]
    slots[9:] = [112 + 3, 112 + 4, 112 + 5]
    kc, ks = filled_cache(9, 1, page, d, 9)
    ks[7] = 2.0 ** -40
    append_both(x.to(DT[dtype]), x.flip(2).to(DT[dtype]), slots, kc, ks, kc.copy(), ks.copy(), dtype)


def test_append_leaves_rows_without_a_slot():
    d, page = 64, 16
    kc, ks = filled_cache(4, 2, page, d, 10)
    x = torch.randn(6, 2, d, generator=torch.Generator().manual_seed(2)).bfloat16()
    slots = [-1, 64, 2 ** 31 - 1, -2 ** 31, 3, -5]  # four pages: slots 0 .. 63
    append_both(x, x, slots, kc, ks, kc.copy(), ks.copy(), "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page,Hk", [(64, 16, 2), (64, 32, 1), (128, 64, 1), (64, 128, 1), (128, 128, 2), (128, 16, 12),
                                       (128, 32, 12), (64, 16, 12), (64, 64, 12), (128, 64, 12)])
def test_append_many_rows(d, page, Hk, dtype):
    """More than 2048 rows: runs of every length up to several pages, in any order, some behind held tokens."""
    r = np.random.RandomState(page + d + 1)
    added = np.concatenate([np.arange(0, 9), r.randint(1, 3 * page, 24), [5 * page + 3], np.ones(90, int)])
    while added.sum() < 2200:
        added = np.append(added, r.randint(1, 4 * page))
    r.shuffle(added)
    lens = r.randint(0, 2 * page, len(added))
    width = max(pages_of(lens + added, page)) + 1
    table, left = table_of(lens, page, width, seed=40, spare=sum(pages_of(added, page)) + len(added))
    p = oa.plan(lens, added, table, left, 0, page, int(added.sum()) + 5)
    P = int(max(p["table"].max(), left.max())) + 1
    kc, ks = filled_cache(P, Hk, page, d, 41)
    vc, vs = filled_cache(P, Hk, page, d, 42)
    g = torch.Generator().manual_seed(43)
    rows = len(p["slots"])
    mag = torch.exp2(torch.randint(-6, 8, (rows, Hk, 1), generator=g).float())
    x, y = ((torch.randn(rows, Hk, d, generator=g) * mag).to(DT[dtype]) for _ in range(2))
    append_both(x, y, p["slots"], kc, ks, vc, vs, dtype)


@pytest.mark.parametrize("rows", [40, 2400])
def test_append_rows_out_of_order_on_a_page_are_not_written(rows):
    """Behind a row without the next slot, and behind a slot given twice, a page's rows are left out."""
    d, page, P = 64, 16, 160
    slots = np.full(rows, -1)
    slots[:9] = [3, 4, 4, 5, 6, 20, 22, 23, 40]
    slots[20:25] = [64, 65, 66, 64, 65]
    if rows > 100:
        slots[62:67] = [100, 101, 102, 101, 102]  # across two blocks of rows
        slots[2390:2396] = 130 + np.arange(6)
    kept = slots.copy()
    for i in (2, 3, 4, 6, 7, 23, 24, 65, 66):
        if i < rows:
            kept[i] = -1
    kc, ks = filled_cache(P, 1, page, d, 44)
    x = torch.randn(rows, 1, d, generator=torch.Generator().manual_seed(45)).bfloat16()
    import linear_attention_sequence_rule_b200 as gdn
    dev, sc = [torch.from_numpy(kc).cuda() for _ in range(2)], [torch.from_numpy(ks).float().cuda() for _ in range(2)]
    gdn.cache_append(x.cuda(), x.cuda(), i32(slots), *dev, *sc)
    wc, ws = oa.append(x, kept, kc, ks)
    for c, s in zip(dev, sc):
        assert np.array_equal(c.cpu().numpy(), wc) and np.array_equal(s.double().cpu().numpy(), ws)


# ---- one-token attention ---------------------------------------------------------------------------

def decode_both(q, kc, vc, ks, vs, table, lens, dtype, scale=None):
    import linear_attention_sequence_rule_b200 as gdn
    dev = [torch.from_numpy(c).cuda() for c in (kc, vc)]
    sc = [torch.from_numpy(s).float().cuda() for s in (ks, vs)]
    out = gdn.attn_decode(q.cuda(), dev[0], dev[1], sc[0], sc[1], i32(table), i32(lens), scale=scale)
    gdn.device_status()
    want, pv, s_abs = oa.decode(q, kc, vc, ks, vs, table, lens, scale=scale)
    n = max(1, int(max(lens)))
    # weights below 2^-14 of the largest: 2^-25 of it each; pv bounds the largest weight's share
    ab.check("out", oa.f64(out), want, ab.decode(want, pv, s_abs, dtype, q.shape[-1], n) + tiny(vc, vs, n))
    return out


def tiny(vc, vs, n):
    """fp16's absolute error of a weight, 2^-25 of the largest, on n values of at most 448 x scale."""
    return n * 2.0 ** -25 * 448 * float(vs.max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_decode_lengths(page, d, dtype):
    lens = [1, 0, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 300, 511, 900]
    table, _ = table_of(lens, page, 900 // page + 2, seed=11)
    P = int(table.max()) + 3
    kc, ks = filled_cache(P, 2, page, d, 12)
    vc, vs = filled_cache(P, 2, page, d, 13)
    q = torch.randn(len(lens), 6, d, generator=torch.Generator().manual_seed(14)).to(DT[dtype])
    out = decode_both(q, kc, vc, ks, vs, table, lens, dtype, scale=0.02)
    assert not out[1].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (2, 2), (7, 1), (8, 1), (9, 1), (16, 1), (17, 1), (40, 1), (24, 2)])
def test_decode_shared_heads(Hq, Hk, dtype):
    lens, page, d = [70, 333], 64, 128
    table, _ = table_of(lens, page, 6, seed=15)
    kc, ks = filled_cache(int(table.max()) + 1, Hk, page, d, 16)
    vc, vs = filled_cache(int(table.max()) + 1, Hk, page, d, 17)
    q = torch.randn(2, Hq, d, generator=torch.Generator().manual_seed(18)).to(DT[dtype])
    decode_both(q, kc, vc, ks, vs, table, lens, dtype, scale=0.01)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 64])
def test_decode_long_context_is_split(page, dtype):
    import linear_attention_sequence_rule_b200 as gdn
    lens, d = [9000, 5], 64
    width = 9000 // page + 40
    assert gdn.gdn_attn_decode_workspace_bytes(2, 2, 1, d, page, width, 1) > 0
    table, _ = table_of(lens, page, width, seed=19)
    kc, ks = filled_cache(int(table.max()) + 1, 1, page, d, 20)
    vc, vs = filled_cache(int(table.max()) + 1, 1, page, d, 21)
    q = torch.randn(2, 2, d, generator=torch.Generator().manual_seed(22)).to(DT[dtype])
    decode_both(q, kc, vc, ks, vs, table, lens, dtype, scale=0.02)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 32, 128])
def test_decode_never_reads_past_the_length(page, dtype):
    """NaN bytes behind a request's length, in spare pages, and table entries out of range."""
    lens, d = [page + 3, 5, 3 * page, 2 * page - 1], 64
    table, _ = table_of(lens, page, 6, seed=23)
    P = int(table.max()) + 3
    kc, ks = filled_cache(P, 2, page, d, 24)
    vc, vs = filled_cache(P, 2, page, d, 25)
    used = np.zeros((P, page), bool)
    for r, L in enumerate(lens):
        for j in range(L):
            used[table[r, j // page], j % page] = True
    for c in (kc, vc):
        c.transpose(0, 2, 1, 3)[~used] = 0x7f
    table[2, 1] = P + 5     # a page out of range in the middle: its tokens are left out
    table[3, 0] = -7
    q = torch.randn(4, 4, d, generator=torch.Generator().manual_seed(26)).to(DT[dtype])
    decode_both(q, kc, vc, ks, vs, table, lens, dtype, scale=0.02)
    # lengths beyond the table row are cut there, negative ones are empty
    long = [6 * page + 9, -3, 0, 1]
    table[0] = table[0, 0]
    kc[table[0, 0]], vc[table[0, 0]] = 0x38, 0x38
    out = decode_both(q, kc, vc, ks, vs, table, long, dtype, scale=0.02)
    assert not out[1].any() and not out[2].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_large_and_small_magnitudes(dtype):
    """Blocks of values 2^40 apart, queries of 1e-3 and 1e3: the frame of the weights carries them."""
    lens, page, d = [150], 32, 64
    table, _ = table_of(lens, page, 6, seed=27)
    P = int(table.max()) + 1
    kc, ks = filled_cache(P, 1, page, d, 28)
    vc, vs = filled_cache(P, 1, page, d, 29)
    vs = vs * 2.0 ** np.linspace(-20, 20, P).round()[:, None]
    ks = ks * 2.0 ** np.linspace(6, -6, P).round()[:, None]
    q = torch.randn(1, 4, d, generator=torch.Generator().manual_seed(30))
    q = q * torch.tensor([1e-3, 1.0, 30.0, 1e3]).view(1, 4, 1)
    decode_both(q.to(DT[dtype]), kc, vc, ks, vs, table, lens, dtype, scale=1e-4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 64])
def test_decode_many_requests_some_long(page, dtype):
    """Contexts that are not split and span more than 32 tiles a warp."""
    import linear_attention_sequence_rule_b200 as gdn
    d, n = 64, 1100
    lens = np.random.RandomState(46).randint(0, 60, n)
    lens[[3, 500, 1099]] = [4097, 9000, 8191]
    width = 9100 // page
    assert gdn.gdn_attn_decode_workspace_bytes(n, 2, 1, d, page, width, gdn._DT[DT[dtype]]) == 0
    table, _ = table_of(lens, page, width, seed=47)
    kc, ks = filled_cache(int(table.max()) + 1, 1, page, d, 48)
    vc, vs = filled_cache(int(table.max()) + 1, 1, page, d, 49)
    q = torch.randn(n, 2, d, generator=torch.Generator().manual_seed(50)).to(DT[dtype])
    decode_both(q, kc, vc, ks, vs, table, lens, dtype, scale=0.02)


@pytest.mark.parametrize("lens", ["any", "equal", "empty", "one", "classes"])
@pytest.mark.parametrize("n", [2, 31, 129, 512, 513])
def test_decode_order_of_the_requests(n, lens):
    """More CTAs than places: every request is worked on once, in whatever order its length gives."""
    page, d, Hk = 64, 64, 8 if n > 31 else 40
    r = np.random.RandomState(n)
    lengths = dict(any=r.randint(0, 1100, n), equal=np.full(n, 70), empty=np.zeros(n, int), one=np.ones(n, int),
                   classes=2 ** r.randint(0, 11, n) + r.randint(-1, 2, n))[lens].copy()
    if lens == "any":
        lengths[[0, n - 1]] = -3, 1100
    table, _ = table_of(np.maximum(lengths, 0), page, 18, seed=60)
    P = max(int(table.max()) + 1, 1)
    kc, ks = filled_cache(P, Hk, page, d, 61)
    vc, vs = filled_cache(P, Hk, page, d, 62)
    q = torch.randn(n, Hk, d, generator=torch.Generator().manual_seed(63)).bfloat16()
    decode_both(q, kc, vc, ks, vs, table, lengths, "bf16", scale=0.02)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_heads_do_not_touch_one_another(dtype):
    """A head's result does not depend on what the heads beside it hold: huge, tiny, infinite or NaN."""
    import linear_attention_sequence_rule_b200 as gdn
    lens, page, d = [100, 40], 32, 128
    table, _ = table_of(lens, page, 4, seed=51)
    P = int(table.max()) + 1
    dev = [torch.from_numpy(filled_cache(P, 1, page, d, x)[0]).cuda() for x in (52, 53)]
    sc = [torch.from_numpy(filled_cache(P, 1, page, d, x)[1]).float().cuda() for x in (52, 53)]
    q = torch.randn(2, 12, d, generator=torch.Generator().manual_seed(54)).to(DT[dtype]).cuda()
    f = lambda x: gdn.attn_decode(x, *dev, *sc, i32(table), i32(lens), scale=0.02)
    want = f(q)
    for h, bad in ((0, 2.0 ** 60), (5, 2.0 ** -60), (9, float("inf")), (11, float("nan"))):
        y = q.clone()
        y[:, h] *= bad
        rest = [i for i in range(12) if i != h]
        assert torch.equal(f(y)[:, rest], want[:, rest]), (h, bad)
    gdn.device_status()


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, give what each gives alone."""
    import linear_attention_sequence_rule_b200 as gdn
    page, d, n = 64, 128, 5
    g = torch.Generator("cuda").manual_seed(55)
    cases = []
    for ctx in (3000, 700):
        width = -(-ctx // page)
        table = torch.randperm(n * width, generator=g, device="cuda").to(torch.int32).view(n, width)
        cache = [torch.randint(0, 120, (n * width, 2, page, d), generator=g, device="cuda").to(torch.uint8) for _ in range(2)]
        sc = [torch.full((n * width, 2), 2.0 ** -7, device="cuda") for _ in range(2)]
        q = torch.randn(n, 8, d, generator=g, device="cuda").bfloat16()
        cases.append((q, *cache, *sc, table, i32([ctx - 7 * i for i in range(n)])))
    want = [gdn.attn_decode(*c, scale=0.01) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(20):
        for i, (c, st) in enumerate(zip(cases, streams)):
            got[i].append(gdn.attn_decode(*c, scale=0.01, stream=st))
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for xs, w in zip(got, want) for x in xs)
    gdn.device_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nothing_is_written_outside_the_arrays(dtype):
    """Outputs and workspaces that lie between marked bytes, at odd sizes."""
    import linear_attention_sequence_rule_b200 as gdn
    held = []

    def guarded(*shape, dtype):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        raw = torch.full((n + 1024 + 512,), 0x5a, dtype=torch.uint8, device="cuda")
        at = 512 + (-(raw.data_ptr() + 512)) % 256
        held.append((raw, at, n))
        return raw[at:at + n].view(dtype).view(*shape)

    dt, lengths, Hq, Hk, d, page = DT[dtype], [129, 1, 70, 0, 33], 6, 2, 64, 32
    T, N, code = sum(lengths) + 3, len(lengths), gdn._DT[DT[dtype]]
    g = torch.Generator().manual_seed(56)
    q, do = (torch.randn(T, Hq, d, generator=g).to(dt).cuda() for _ in range(2))
    k, v = (torch.randn(T, Hk, d, generator=g).to(dt).cuda() for _ in range(2))
    table = guarded(N, 6, dtype=torch.int32).fill_(-1)
    plan = gdn.cache_plan(i32([0] * N), i32(lengths), table, i32(range(20)), i32([0]), page, T,
                          *(guarded(m, dtype=torch.int32) for m in (N + 1, T, T, N, 1, 2)))
    assert plan.status.tolist() == [0, 0]
    cache = [guarded(20, Hk, page, d, dtype=torch.uint8).zero_() for _ in range(2)]
    sc = [guarded(20, Hk, dtype=torch.float32).zero_() for _ in range(2)]
    gdn.cache_append(k, v, plan.slots, *cache, *sc)
    out, lse = guarded(T, Hq, d, dtype=dt), guarded(T, Hq, dtype=torch.float32)
    gdn.attn_fwd(q, k, v, cu_seqlens=plan.cu_seqlens, out=out, lse=lse)
    grads = [guarded(T, h, d, dtype=dt) for h in (Hq, Hk, Hk)]
    ws = guarded(gdn.gdn_attn_bwd_workspace_bytes(N, T, Hq, Hk, d, 1, code), dtype=torch.uint8)
    gdn.attn_bwd(q, k, v, out, lse, do, plan.cu_seqlens, None, *grads, workspace=ws)
    ws = guarded(gdn.gdn_attn_decode_workspace_bytes(N, Hq, Hk, d, page, 6, code), dtype=torch.uint8)
    gdn.attn_decode(q[:N], *cache, *sc, table, plan.lens, out=guarded(N, Hq, d, dtype=dt), workspace=ws)
    gdn.device_status()
    for raw, at, n in held:
        assert bool((raw[:at] == 0x5a).all()) and bool((raw[at + n:] == 0x5a).all())


# ---- together --------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_then_generation_steps(dtype):
    """As a serving step runs them: prompts planned, attended to and cached, then one-token steps."""
    import linear_attention_sequence_rule_b200 as gdn
    page, d, Hq, Hk, P, width = 32, 64, 6, 2, 40, 8
    prompts = [70, 1, 0, 128, 33]
    n = len(prompts)
    free = np.random.RandomState(31).permutation(P)
    lens, head, table = i32([0] * n), i32([0]), torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    cache = [torch.zeros(P, Hk, page, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.zeros(P, Hk, device="cuda") for _ in range(2)]
    ref = [(c.cpu().numpy(), s.double().cpu().numpy()) for c, s in zip(cache, sc)]
    state = dict(lens=[0] * n, free_head=0, table=table.cpu().numpy())
    g = torch.Generator().manual_seed(32)
    rnd = lambda rows, h: torch.randn(rows, h, d, generator=g).to(DT[dtype])
    for step, added in enumerate([prompts] + [[1] * n, [1, 0, 1, 1, 1], [0, 3, 1, 1, 0], [1] * n]):
        rows = sum(added) + 2
        p = gdn.cache_plan(lens, i32(added), table, i32(free), head, page, rows, lens_out=lens, free_head_out=head)
        state = oa.plan(state["lens"], added, state["table"], free, state["free_head"], page, rows)
        assert state["status"] == [0, 0] and p.slots.tolist() == state["slots"]
        k, v = rnd(rows, Hk), rnd(rows, Hk)
        gdn.cache_append(k.cuda(), v.cuda(), p.slots, *cache, *sc)
        ref = [oa.append(x, state["slots"], c, s) for x, (c, s) in zip((k, v), ref)]
        if step == 0:  # the prompts themselves, packed by the plan's offsets
            q = rnd(rows, Hq)
            out, _ = gdn.attn_fwd(q.cuda(), k.cuda(), v.cuda(), cu_seqlens=p.cu_seqlens)
            m = sum(added)
            r = oa.prompt(q[:m], k[:m], v[:m], cu=p.cu_seqlens.cpu())
            ab.check("prefill", oa.f64(out)[:m], r["out"], ab.forward(r, dtype, d, max(added))[0])
        q = rnd(n, Hq)
        out = gdn.attn_decode(q.cuda(), *cache, *sc, table, lens)
        for (c, s), gc, gs in zip(ref, cache, sc):
            assert np.array_equal(gc.cpu().numpy(), c) and np.array_equal(gs.double().cpu().numpy(), s)
        want, pv, s_abs = oa.decode(q, ref[0][0], ref[1][0], ref[0][1], ref[1][1], state["table"], state["lens"])
        ab.check("step", oa.f64(out), want,
                 ab.decode(want, pv, s_abs, dtype, d, 200) + tiny(ref[1][0], ref[1][1], 200))
    assert lens.tolist() == state["lens"] and head.item() == state["free_head"]
    gdn.device_status()


def test_generation_step_replayed_from_a_graph():
    """A captured step (plan in place, append, attention) replayed gives what eager steps give; two graphs
    with workspaces of their own run on the same cache in turn."""
    import linear_attention_sequence_rule_b200 as gdn
    page, d, Hq, Hk, n, width, P = 64, 128, 8, 2, 3, 40, 130
    r = torch.Generator("cuda").manual_seed(33)
    free, one = torch.randperm(P, generator=r, device="cuda").to(torch.int32), i32([1] * n)
    k, v = (torch.randn(n, Hk, d, generator=r, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(n, Hq, d, generator=r, device="cuda").bfloat16()

    def fresh():
        lens, head, table = i32([0] * n), i32([0]), torch.full((n, width), -1, dtype=torch.int32, device="cuda")
        cache = [torch.zeros(P, Hk, page, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
        sc = [torch.zeros(P, Hk, device="cuda") for _ in range(2)]
        # a prompt of 1000 tokens each
        p = gdn.cache_plan(lens, i32([1000] * n), table, free, head, page, 3000, lens_out=lens, free_head_out=head)
        x = torch.randn(3000, Hk, d, generator=torch.Generator("cuda").manual_seed(34), device="cuda").bfloat16()
        gdn.cache_append(x, x, p.slots, *cache, *sc)
        return lens, head, table, cache, sc

    def step(st, out):
        lens, head, table, cache, sc = st
        p = gdn.cache_plan(lens, one, table, free, head, page, n, lens_out=lens, free_head_out=head)
        gdn.cache_append(k, v, p.slots, *cache, *sc)
        gdn.attn_decode(q, *cache, *sc, table, lens, out=out)

    eager, a, b = fresh(), torch.empty_like(q), torch.empty_like(q)
    outs = []
    for _ in range(4):
        step(eager, a)
        outs.append(a.clone())
    held = fresh()
    start = [x.clone() for x in (held[0], held[1], held[2], *held[3], *held[4])]
    graphs = []
    for o in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(held, o)
        graphs.append((g, o))
    for x, y in zip((held[0], held[1], held[2], *held[3], *held[4]), start):
        x.copy_(y)
    for i in range(4):
        g, o = graphs[i % 2]
        g.replay()
        assert torch.equal(o, outs[i])
    assert torch.equal(held[0], eager[0]) and all(torch.equal(x, y) for x, y in zip(held[3] + held[4], eager[3] + eager[4]))
    gdn.device_status()
