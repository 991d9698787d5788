"""The paged cache on the GPU against plain references in 64 bits
(``paged_reference.py``): plan, append, page means, selection, top-k and the
attention of one token, alone and together over several steps.  What the cache
holds behind the sequences' ends is NaN throughout."""
import random

import pytest

import paged_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_sparse_attention_queries_b200 as ab  # noqa: E402

BF16, I32 = torch.bfloat16, torch.int32
CAPACITY = 4


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.fail("no CUDA device")
    from block_sparse_attention_queries_b200 import build as abbuild
    abbuild.build()
    ab.lib()
    return torch.device("cuda:0")


@pytest.fixture(autouse=True)
def _clean(dev):
    ab.device_error(dev)
    yield
    assert ab.device_error(dev) == 0


def ints(v, dev):
    return torch.tensor(v, dtype=I32, device=dev)


# -------------------------------------------------------------------- plan
def _plan_case(S, page, seed, max_new, spare):
    r = random.Random(seed)
    max_pages = ref.cdiv(4 * max_new + 70, page) + 1
    lens = [r.choice([0, 0, 1, page - 1, page, page + 1, r.randint(0, max_pages * page - max_new)]) for _ in range(S)]
    lens = [min(n, max_pages * page) for n in lens]
    n_new = [r.choice([-1, 0, 1, 1, r.randint(0, max_new)]) for _ in range(S)]
    pages = [ref.cdiv(n, page) for n in lens]
    num_pages = sum(pages) + spare
    ids = list(range(num_pages))
    r.shuffle(ids)
    table = [[ids.pop() if j < k else -9 for j in range(max_pages)] for k in pages]
    free = ids + [-5] * (num_pages - len(ids))
    return n_new, lens, table, free, len(ids), page, max_pages, num_pages


def _run_plan(case, T, dev, in_place=False):
    n_new, lens, table, free, count, page, max_pages, num_pages = case
    pp = ab.PagedParams(len(lens), 1, 1, 64, page, num_pages, max_pages)
    t = dict(n_new=ints(n_new, dev), lens=ints(lens, dev), table=ints(table, dev), free_pages=ints(free, dev),
             free_count=ints([count], dev))
    kw = {} if in_place else dict(lens_out=torch.full_like(t["lens"], -3), free_count_out=torch.full_like(t["free_count"], -3))
    out = ab.ab_paged_plan(pp, T=T, **t, **kw)
    lens_out, count_out = kw.get("lens_out", t["lens"]), kw.get("free_count_out", t["free_count"])
    return [x.tolist() for x in (lens_out, t["table"], t["free_pages"], count_out, *out)]


@pytest.mark.parametrize("S,page,max_new,seed", [(1, 16, 1, 0), (1, 64, 500, 1), (7, 32, 40, 2), (256, 16, 1, 3), (33, 16, 700, 4),
                                                (1024, 64, 9, 5), (1500, 16, 30, 6), (8192, 16, 3, 7)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(dev, S, page, max_new, seed, in_place):
    case = _plan_case(S, page, seed, max_new, spare=S * (max_new // page + 2))
    n_new, lens, table, free, count, page, max_pages, num_pages = case
    T = sum(max(n, 0) for n in n_new) + 5
    want = ref.plan(n_new, lens, table, free, count, page, max_pages, T)
    got = _run_plan(case, T, dev, in_place)
    assert not want[-1] and ab.device_error(dev) == 0
    for g, w in zip(got, (want[0], want[1], want[2], [want[3]], *want[4:7])):
        assert g == w
    assert _run_plan(case, T, dev) == got  # and again


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("short", ["pages", "more pages", "slots", "row", "bad"])
def test_plan_does_not_fit(dev, seed, short):
    case = list(_plan_case(40 + 700 * (seed % 3), 16, 100 + seed, 50, spare={"pages": 60, "more pages": 2}.get(short, 20000)))
    n_new, lens = case[0], case[1]
    total = sum(max(n, 0) for n in n_new)
    T = total // 2 if short == "slots" else total + 50 * len(lens)
    if short == "more pages":  # nothing is given back
        n_new[:] = [50 if n == -1 else n for n in n_new]
    if short == "row":
        n_new[7], n_new[11] = case[6] * case[5] + 1 - lens[7], 2 ** 24
    if short == "bad":
        n_new[5] = -2
    want = ref.plan(*case[:5], case[5], case[6], T)
    got = _run_plan(case, T, dev)
    # 60 pages more than are in use can be enough, with those given back
    assert want[-1] or short == "pages"
    assert ab.device_error(dev) == (CAPACITY if want[-1] else 0)
    for g, w in zip(got, (want[0], want[1], want[2], [want[3]], *want[4:7])):
        assert g == w


def test_plan_only_releases(dev):
    case = _plan_case(5, 16, 9, 40, 3)
    case = ([-1] * 5, *case[1:])
    want = ref.plan(*case[:5], case[5], case[6], 0)
    got = _run_plan(case, 0, dev)
    assert got[:4] == [want[0], want[1], want[2], [want[3]]] and got[4] == [0] * 6


def test_plan_refuses_bad_state(dev):
    # a count or a length out of range, a free list with an unknown page: no
    # access out of range, the error is raised, the slots are -1
    pp = ab.PagedParams(2, 1, 1, 64, 16, 8, 4)
    for count, lens, free in ((99, [1, 0], range(8)), (4, [70, 0], range(8)), (4, [-3, 0], range(8)), (4, [0, 0], [100] * 8)):
        cu, slots, pos = ab.ab_paged_plan(pp, ints([0, 5], dev), ints(lens, dev), ints([[0, 0, 0, 0]] * 2, dev),
                                          ints(list(free), dev), ints([count], dev), T=5)
        assert ab.device_error(dev) == CAPACITY
        if list(free) == [100] * 8:
            assert slots.tolist() == [-1] * 5
        else:
            assert all(0 <= x < 8 * 16 for x in slots.tolist())


# ------------------------------------------------------- append and means
def _rope(norm, Hq, Hk, d, n_pos, interleaved, seed, dev, rotate=True):
    g = torch.Generator().manual_seed(seed)
    shape = {"none": None, "head": lambda H: (d,), "token": lambda H: (H, d)}[norm]
    wq, wk = (None, None) if shape is None else (1 + 0.3 * torch.randn(shape(H), generator=g) for H in (Hq, Hk))
    a = torch.rand(n_pos, d // 2, generator=g) * 20
    cos, sin = (a.cos(), a.sin()) if rotate else (None, None)
    up = lambda t: None if t is None else t.to(dev)  # noqa: E731
    return (wq, wk, cos, sin), ab.NormRope(norm, interleaved, 1e-6, up(wq), up(wk), up(cos), up(sin))


@pytest.mark.parametrize("Hq,Hkv,d,page", [(1, 1, 64, 16), (8, 2, 128, 16), (40, 40, 128, 64), (16, 1, 64, 32), (5, 5, 128, 32)])
@pytest.mark.parametrize("norm,interleaved", [("none", True), ("head", False), ("token", True), ("head", True)])
def test_append(dev, Hq, Hkv, d, page, norm, interleaved):
    g = torch.Generator().manual_seed(3)
    lens = [0, 5, page - 1, page, 3 * page + 7, 2]
    new = [3 * page + 1, 1, 1, 2, 0, page - 2]
    T, pad = sum(new), 4
    c = ref.Cache([n + m for n, m in zip(lens, new)], Hkv, d, page, 5)
    n_pos = max(n + m for n, m in zip(lens, new))
    (wq, wk, cos, sin), nr = _rope(norm, Hq, Hkv, d, n_pos, interleaved, 6, dev)
    slots, pos = [], []
    for s, (n, m) in enumerate(zip(lens, new)):
        for i in range(n, n + m):
            slots.append(int(c.table[s, i // page]) * page + i % page)
            pos.append(i)
    x = torch.randn(T + pad, Hq + 2 * Hkv, d, generator=g).to(BF16)
    xd = x.to(dev)
    pp = ab.PagedParams(len(lens), Hq, Hkv, d, page, c.num_pages, c.max_pages)
    K, V, ksum = c.K.to(dev), c.V.to(dev), c.ksum.to(dev)
    Q0 = torch.full((T + pad, Hq, d), 7.0, dtype=BF16, device=dev)
    Q = ab.ab_paged_append(pp, nr, xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], ints(slots + [-1] * pad, dev),
                           ints(pos + [0] * pad, dev), K, V, ksum=ksum, out=Q0)
    assert (Q[T:] == 7.0).all()
    at = torch.tensor(pos)
    q, size = ref.norm_rotate(x[:T, :Hq], norm, wq, cos, sin, at, interleaved, 1e-6)
    ref.assert_norm_rotate(Q[:T].cpu(), q, size, norm, Hq * d)
    k, size = ref.norm_rotate(x[:T, Hq:Hq + Hkv], norm, wk, cos, sin, at, interleaved, 1e-6)
    Kc, Vc, sc = K.cpu(), V.cpu(), ksum.cpu()
    sl = torch.tensor(slots)
    ref.assert_norm_rotate(Kc[sl // page, :, sl % page], k, size, norm, Hkv * d)
    assert torch.equal(Vc[sl // page, :, sl % page], x[:T, Hq + Hkv:])
    # everything else is as it was
    mask = torch.zeros(c.num_pages, page, dtype=torch.bool)
    mask[sl // page, sl % page] = True
    for new_t, old_t in ((Kc, c.K), (Vc, c.V)):
        a, b = new_t.transpose(1, 2)[~mask], old_t.transpose(1, 2)[~mask]
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    fill = {}
    for z in slots:
        fill[z // page] = max(fill.get(z // page, 0), z % page + 1)
    for p in range(c.num_pages):
        if p in fill:
            n = fill[p]
            keys = Kc[p, :, :n].double()
            off = (sc[p].double() - keys.mean(1)).abs() - (ref.HALF * keys.mean(1).abs() + (n + 2) * ref.U * 1.01 * keys.abs().mean(1))
            assert off.max() <= 0
        else:
            assert torch.equal(sc[p].view(torch.int16), c.ksum[p].view(torch.int16))


@pytest.mark.parametrize("Hq,Hkv,d", [(32, 8, 128), (40, 4, 128), (72, 9, 64), (160, 10, 128), (48, 3, 64)])
def test_append_many_tokens_of_few_key_heads(dev, Hq, Hkv, d):
    g = torch.Generator().manual_seed(7)
    page, T = 16, 1500
    (wq, wk, cos, sin), nr = _rope("token", Hq, Hkv, d, T, True, 8, dev)
    num_pages = ref.cdiv(T, page) + 1
    pp = ab.PagedParams(1, Hq, Hkv, d, page, num_pages, num_pages)
    x = torch.randn(T, Hq + 2 * Hkv, d, generator=g).to(BF16)
    xd, at = x.to(dev), torch.arange(T)
    slots = at + page
    slots[700] = -1                                              # a token that is skipped
    K, V = (torch.zeros(num_pages, Hkv, page, d, dtype=BF16, device=dev) for _ in range(2))
    Q = ab.ab_paged_append(pp, nr, xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], ints(slots.tolist(), dev), ints(at.tolist(), dev),
                           K, V, out=torch.full((T, Hq, d), 7.0, dtype=BF16, device=dev)).cpu()
    assert (Q[700] == 7.0).all()
    kept = at != 700
    q, size = ref.norm_rotate(x[:, :Hq], "token", wq, cos, sin, at, True, 1e-6)
    ref.assert_norm_rotate(Q[kept], q[kept], size[kept], "token", Hq * d)
    k, size = ref.norm_rotate(x[:, Hq:Hq + Hkv], "token", wk, cos, sin, at, True, 1e-6)
    sl = slots[kept]
    ref.assert_norm_rotate(K.cpu()[sl // page, :, sl % page], k[kept], size[kept], "token", Hkv * d)
    assert torch.equal(V.cpu()[sl // page, :, sl % page], x[kept, Hq + Hkv:])
    left = 700 + page
    assert (K[left // page, :, left % page] == 0).all() and (V[left // page, :, left % page] == 0).all()


def test_append_bad_slots_and_positions(dev):
    # reported, and nothing is written for them
    _, nr = _rope("head", 2, 2, 64, 10, True, 1, dev)
    pp = ab.PagedParams(1, 2, 2, 64, 16, 4, 4)
    x = torch.randn(3, 2, 64, device=dev).to(BF16)
    K = torch.zeros(4, 2, 16, 64, dtype=BF16, device=dev)
    V, ksum = torch.zeros_like(K), torch.zeros(4, 2, 64, dtype=BF16, device=dev)
    Q = torch.zeros(3, 2, 64, dtype=BF16, device=dev)
    ab.ab_paged_append(pp, nr, x, x, x, ints([64, -1, 2 ** 31 - 1], dev), ints([0, 0, 0], dev), K, V, ksum=ksum, out=Q)
    assert ab.device_error(dev) == CAPACITY
    assert not any(t.any() for t in (K, V, ksum, Q))
    ab.ab_paged_append(pp, nr, x, x, x, ints([0, 1, 2], dev), ints([10, -1, 3], dev), K, V, out=Q)
    assert ab.device_error(dev) == CAPACITY
    assert not Q[:2].any() and Q[2].any() and not K[0, :, :2].any() and K[0, :, 2].any()


# ------------------------------------------------------- select and top-k
@pytest.mark.parametrize("Hq,Hkv,d,page", [(1, 1, 64, 16), (12, 12, 128, 32), (32, 8, 128, 16), (16, 1, 64, 64), (9, 1, 128, 16)])
@pytest.mark.parametrize("lens", [[1], [16 * 128, 16 * 128 + 1, 0, 5], [40000, 77, 3000], [700] * 70 + [9000, 13000],
                                  [0, 20000, 1, 0, 16384, 0]])
def test_select(dev, Hq, Hkv, d, page, lens):
    g = torch.Generator().manual_seed(11)
    c = ref.Cache(lens, Hkv, d, page, 12)
    q = (1.3 * torch.randn(len(lens), Hq, d, generator=g)).to(BF16)
    pp = ab.PagedParams(len(lens), Hq, Hkv, d, page, c.num_pages, c.max_pages)
    P = torch.full((len(lens), Hkv, c.max_pages), -1.0, device=dev)
    got = ab.ab_paged_select(pp, q.to(dev), c.ksum.to(dev), c.table.to(dev), ints(lens, dev), out=P).cpu()
    G = Hq // Hkv
    for s, n in enumerate(lens):
        k = ref.cdiv(n, page)
        assert (got[s, :, k:] == -1).all()
        for h in range(Hkv if k else 0):
            p, eps = ref.select(q[s, h * G:(h + 1) * G], c.ksum[c.table[s, :k].long(), h], n, page, d)
            x = got[s, h, :k].double()
            # exponentials 2^-21 each, a row's sum of k terms in 32 lanes' parts, G terms
            rel = 2 * eps + 2.0 ** -20 + (k / 32 + 60) * ref.U * 2
            assert ((x - p).abs() <= rel * p + 1e-37).all(), ((x - p).abs() / p).max()


@pytest.mark.parametrize("keep", [0.05, 0.11, 0.5, 1.0])
@pytest.mark.parametrize("recent", [0, 1, 5, 10000])
def test_topk(dev, keep, recent):
    r = torch.Generator().manual_seed(4)
    page, Hkv = 16, 3
    pages = [1, 2, 7, 255, 256, 257, 1023, 1025, 5000, 0]
    lens = [n * page - (n % 3 if n else 0) for n in pages]
    S, most = len(lens), max(pages) + 2
    P = torch.rand(S, Hkv, most, generator=r) ** 4
    P[:, 1] = (P[:, 1] * 8).round() / 8        # many ties, many zeros
    P[:, 2] = 0.25                             # all equal
    P[4, 0, ::3], P[5, 0, ::5] = float("nan"), -1.0
    pp = ab.PagedParams(S, Hkv, Hkv, 64, page, 4, most, keep_ratio=keep, recent=recent)
    idx = torch.full((S, Hkv, most), -4, dtype=I32, device=dev)
    idx, count = ab.ab_paged_topk(pp, P.to(dev), ints(lens, dev), out=(idx, torch.zeros(S, Hkv, dtype=I32, device=dev)))
    idx, count = idx.cpu(), count.cpu()
    for s, n in enumerate(pages):
        for h in range(Hkv):
            want = ref.topk(P[s, h], n, keep, recent)
            assert count[s, h] == len(want) and idx[s, h, :len(want)].tolist() == want
            assert (idx[s, h, len(want):] == -4).all()


@pytest.mark.parametrize("most", [300, 2000, 6000, 9000])
def test_topk_widths(dev, most):
    # tables of several widths, rows around the lengths where the method changes
    g = torch.Generator().manual_seed(most)
    pages = sorted({1, 3, 31, 32, 33, 255, 256, 257, most - 1, most} & set(range(most + 1)))
    P = torch.rand(len(pages), 2, most, generator=g)
    P[:, 1] = (P[:, 1] * 5).floor() / 5
    for keep, recent in ((0.07, 0), (0.5, 2)):
        pp = ab.PagedParams(len(pages), 2, 2, 64, 16, 4, most, keep_ratio=keep, recent=recent)
        idx, count = ab.ab_paged_topk(pp, P.to(dev), ints([n * 16 for n in pages], dev))
        for s, n in enumerate(pages):
            for h in range(2):
                want = ref.topk(P[s, h], n, keep, recent)
                assert count[s, h] == len(want) and idx[s, h, :len(want)].tolist() == want


@pytest.mark.parametrize("same", [1, 2, 255, 256, 257, 700])
@pytest.mark.parametrize("levels", [1, 3, 10 ** 6])
def test_topk_close_values(dev, same, levels):
    # `same` values of one octave's eighth, of `levels` different values, around the last that is kept
    g = torch.Generator().manual_seed(same + levels)
    n, Hkv = 1000, 8
    P = torch.zeros(1, Hkv, n + 3)
    for h in range(Hkv):
        x = torch.rand(n, generator=g) * 0.1
        x[:150] = 0.6 + 0.3 * torch.rand(150, generator=g)
        x[150:150 + same] = 0.25 * (1 + (torch.rand(same, generator=g) * levels).floor() / levels * 0.124)
        P[0, h, :n] = x[torch.randperm(n, generator=g)]
    for kept in (149, 150, 151, 150 + same // 2, 150 + same, min(n, 151 + same)):
        pp = ab.PagedParams(1, Hkv, Hkv, 64, 16, 4, n + 3, keep_ratio=kept / n, recent=0)
        idx, count = ab.ab_paged_topk(pp, P.to(dev), ints([n * 16], dev))
        for h in range(Hkv):
            want = ref.topk(P[0, h], n, kept / n, 0)
            assert len(want) == kept
            assert count[0, h] == len(want) and idx[0, h, :len(want)].tolist() == want


def test_topk_rows_beyond_shared_memory(dev):
    n, most = 24577, 30000
    P = torch.rand(2, 1, most, generator=torch.Generator().manual_seed(14))
    P[1] = (P[1] * 50).round() / 50
    pp = ab.PagedParams(2, 1, 1, 64, 16, 4, most, keep_ratio=0.3, recent=2)
    idx, count = ab.ab_paged_topk(pp, P.to(dev), ints([n * 16, most * 16 - 5], dev))
    for s, k in enumerate((n, most)):
        want = ref.topk(P[s, 0], k, 0.3, 2)
        assert count[s, 0] == len(want) and idx[s, 0, :len(want)].tolist() == want


# --------------------------------------------------------------- attention
def _check_attention(O, q, c, lists=None, rows=None):
    G = q.shape[1] // c.Hkv
    for s, n in enumerate(c.lens):
        row = s if rows is None else rows[s]
        if row is None:
            continue
        for h in range(c.Hkv):
            got = O[s, h * G:(h + 1) * G]
            keys, values = c.keys[s][:, h], c.values[s][:, h]
            if lists is not None:
                at = [i for j in lists[s][h] for i in range(j * c.page, min((j + 1) * c.page, n))]
                keys, values = keys[at], values[at]
            if not len(keys):
                assert (got == 0).all()
                continue
            o, size, eps = ref.attention(q[row, h * G:(h + 1) * G], keys, values, c.d)
            ref.assert_attention(got, o, size, eps, len(keys))


HEADS = [(1, 1, 64, 16), (12, 12, 128, 16), (8, 2, 128, 32), (32, 4, 128, 64), (7, 1, 64, 64), (16, 1, 128, 16), (10, 1, 64, 32)]


@pytest.mark.parametrize("Hq,Hkv,d,page", HEADS)
@pytest.mark.parametrize("lens", [[1], [777], [0, 64, 1, 0, 63, 65, 128, 15, 0], [5000, 3, 0, 12345]])
def test_attention_all_pages(dev, Hq, Hkv, d, page, lens):
    g = torch.Generator().manual_seed(21)
    c = ref.Cache(lens, Hkv, d, page, 22, kscale=1.5)
    q = torch.randn(len(lens), Hq, d, generator=g).to(BF16)
    pp = ab.PagedParams(len(lens), Hq, Hkv, d, page, c.num_pages, c.max_pages)
    O = torch.full((len(lens), Hq, d), 9.0, dtype=BF16, device=dev)
    args = [t.to(dev) for t in (q, c.K, c.V, c.table)] + [ints(lens, dev)]
    ab.ab_attention_paged(pp, *args, out=O)
    _check_attention(O.cpu(), q, c)
    O2 = ab.ab_attention_paged(pp, *args)
    assert torch.equal(O, O2)


@pytest.mark.parametrize("Hq,Hkv,d,page", HEADS)
def test_attention_lists(dev, Hq, Hkv, d, page):
    # any order, repeated pages, empty rows, the partial last page anywhere
    r = random.Random(5)
    g = torch.Generator().manual_seed(31)
    lens = [1, 700, 0, 3000, 64]
    c = ref.Cache(lens, Hkv, d, page, 32, kscale=1.5)
    S = len(lens)
    lists = []
    for n in lens:
        k = ref.cdiv(n, page)
        row = []
        for h in range(Hkv):
            m = r.choice([0, 1, 3, k]) if k else 0
            row.append([r.randrange(k) for _ in range(min(m, c.max_pages))] if h % 2 else r.sample(range(k), min(m, k)))
        lists.append(row)
    idx = torch.full((S, Hkv, c.max_pages), 10 ** 6, dtype=I32)
    for s in range(S):
        for h in range(Hkv):
            idx[s, h, :len(lists[s][h])] = torch.tensor(lists[s][h], dtype=I32)
    count = torch.tensor([[len(x) for x in row] for row in lists], dtype=I32)
    q = torch.randn(S, Hq, d, generator=g).to(BF16)
    pp = ab.PagedParams(S, Hq, Hkv, d, page, c.num_pages, c.max_pages)
    O = ab.ab_attention_paged(pp, *(t.to(dev) for t in (q, c.K, c.V, c.table)), ints(lens, dev), idx=idx.to(dev),
                              count=count.to(dev), out=torch.full((S, Hq, d), 9.0, dtype=BF16, device=dev))
    _check_attention(O.cpu(), q, c, lists)


def test_attention_many_short_rows(dev):
    # more rows than CTAs, most sequences empty
    lens = [0] * 1000
    r = random.Random(8)
    for s in r.sample(range(1000), 90):
        lens[s] = r.randint(1, 200)
    c = ref.Cache(lens, 5, 64, 16, 42)
    g = torch.Generator().manual_seed(41)
    q = torch.randn(1000, 10, 64, generator=g).to(BF16)
    pp = ab.PagedParams(1000, 10, 5, 64, 16, c.num_pages, c.max_pages)
    O = ab.ab_attention_paged(pp, *(t.to(dev) for t in (q, c.K, c.V, c.table)), ints(lens, dev),
                              out=torch.full((1000, 10, 64), 9.0, dtype=BF16, device=dev))
    _check_attention(O.cpu(), q, c)


@pytest.mark.parametrize("Hq,Hkv,d,page,keys", [(8, 2, 128, 16, 256), (8, 2, 128, 16, 272), (3, 3, 64, 64, 512), (16, 1, 64, 32, 544), (40, 40, 128, 64, 64)])
@pytest.mark.parametrize("S", [1, 3, 149, 400])
def test_attention_short_tables(dev, Hq, Hkv, d, page, keys, S):
    # tables around the length up to which no row is divided
    g = torch.Generator().manual_seed(S)
    lens = torch.randint(0, keys + 1, (S,), generator=g).tolist()
    lens[-1] = keys
    c = ref.Cache(lens, Hkv, d, page, 18)
    q = torch.randn(S, Hq, d, generator=g).to(BF16)
    pp = ab.PagedParams(S, Hq, Hkv, d, page, c.num_pages, c.max_pages)
    args = [t.to(dev) for t in (q, c.K, c.V, c.table)] + [ints(lens, dev)]
    _check_attention(ab.ab_attention_paged(pp, *args).cpu(), q, c)
    lists = [[sorted(torch.randperm(ref.cdiv(n, page), generator=g)[:(s + h) % 9].tolist()) for h in range(Hkv)] for s, n in enumerate(lens)]
    idx = torch.full((S, Hkv, c.max_pages), -1, dtype=I32)
    for s in range(S):
        for h in range(Hkv):
            idx[s, h, :len(lists[s][h])] = torch.tensor(lists[s][h], dtype=I32)
    count = ints([[len(x) for x in y] for y in lists], dev)
    _check_attention(ab.ab_attention_paged(pp, *args, idx=idx.to(dev), count=count).cpu(), q, c, lists=lists)


def test_attention_rows_of_new_tokens(dev):
    # cu_new: the newest token's row of Q; sequences without one are left alone
    lens = [100, 50, 0, 33]
    c = ref.Cache(lens, 2, 128, 16, 52)
    g = torch.Generator().manual_seed(51)
    q = torch.randn(9, 4, 128, generator=g).to(BF16)
    pp = ab.PagedParams(4, 4, 2, 128, 16, c.num_pages, c.max_pages)
    cu = [0, 3, 3, 4, 8]
    O = torch.full((4, 4, 128), 9.0, dtype=BF16, device=dev)
    args = [t.to(dev) for t in (q, c.K, c.V, c.table)]
    ab.ab_attention_paged(pp, *args, ints(lens, dev), cu_new=ints(cu, dev), out=O)
    assert (O[1] == 9).all() and (O[2] == 0).all()
    _check_attention(O.cpu(), q, c, rows=[2, None, 3, 7])
    P = torch.full((4, 2, c.max_pages), -1.0, device=dev)
    ab.ab_paged_select(pp, args[0], c.ksum.to(dev), args[3], ints(lens, dev), cu_new=ints(cu, dev), out=P)
    assert (P[1] == -1).all() and (P[0, :, :7] > 0).all() and abs(P[3].clamp(min=0).sum().item() - 2) < 1e-5


def test_attention_extreme_scores(dev):
    # scores of +-hundreds, equal scores, a key that takes everything
    n, d = 500, 128
    c = ref.Cache([n, n, n], 1, d, 16, 62, kscale=30.0)
    c.keys[1][:] = 2.0
    q = torch.randn(3, 1, d, generator=torch.Generator().manual_seed(61)).to(BF16) * 8
    for s in (1,):
        for j in range(ref.cdiv(n, 16)):
            m = min(16, n - j * 16)
            c.K[c.table[s, j], :, :m] = 2.0
    pp = ab.PagedParams(3, 1, 1, d, 16, c.num_pages, c.max_pages)
    O = ab.ab_attention_paged(pp, *(t.to(dev) for t in (q, c.K, c.V, c.table)), ints([n] * 3, dev))
    assert torch.isfinite(O).all()
    _check_attention(O.cpu(), q, c)


@pytest.mark.parametrize("lists", [False, True])
def test_not_a_number_shows(dev, lists):
    # NaN in a valid key or a query reaches the heads that read it, in rows of one CTA and of many
    lens = [40000, 20, 300]
    Hq, Hkv, d, page = 6, 2, 128, 16
    c = ref.Cache(lens, Hkv, d, page, 75)
    q = torch.randn(3, Hq, d, generator=torch.Generator().manual_seed(76)).to(BF16)
    pp = ab.PagedParams(3, Hq, Hkv, d, page, c.num_pages, c.max_pages)
    more = {}
    if lists:
        idx = torch.arange(c.max_pages, dtype=I32).expand(3, Hkv, -1).contiguous()
        count = torch.tensor([[ref.cdiv(n, page)] * Hkv for n in lens], dtype=I32)
        more = dict(idx=idx.to(dev), count=count.to(dev))
    run = lambda q, K: ab.ab_attention_paged(pp, q.to(dev), K.to(dev), c.V.to(dev), c.table.to(dev), ints(lens, dev), **more).cpu()
    good = run(q, c.K)
    for s in range(3):
        K = c.K.clone()
        K[c.table[s, lens[s] // page // 2], 1, 3, 5] = float("nan")
        bad = run(q, K)
        assert torch.isnan(bad[s, 3:]).all()
        bad[s, 3:] = good[s, 3:]
        assert torch.equal(bad, good)
        q2 = q.clone()
        q2[s, 4, 9] = float("nan")
        bad = run(q2, c.K)
        assert torch.isnan(bad[s, 4]).all()
        bad[s, 4] = good[s, 4]
        assert torch.equal(bad, good)


@pytest.mark.parametrize("max_pages", [300, 1500])
def test_select_not_a_number_shows(dev, max_pages):
    lens = [4700, 40, 4000]
    Hq, Hkv, d, page = 6, 2, 64, 16
    c = ref.Cache(lens, Hkv, d, page, 77, max_pages=max_pages)
    q = torch.randn(3, Hq, d, generator=torch.Generator().manual_seed(78)).to(BF16)
    pp = ab.PagedParams(3, Hq, Hkv, d, page, c.num_pages, c.max_pages)
    run = lambda q, k: ab.ab_paged_select(pp, q.to(dev), k.to(dev), c.table.to(dev), ints(lens, dev),
                                          out=torch.full((3, Hkv, max_pages), -1.0, device=dev)).cpu()
    good = run(q, c.ksum)
    for s, n in enumerate(lens):
        k = ref.cdiv(n, page)
        q2, ksum = q.clone(), c.ksum.clone()
        q2[s, 4, 9] = float("nan")
        ksum[c.table[s, k // 2], 1, 60] = float("nan")
        for bad in (run(q2, c.ksum), run(q, ksum)):
            assert torch.isnan(bad[s, 1, :k]).all()
            bad[s, 1, :k] = good[s, 1, :k]
            assert torch.equal(bad, good)


def test_bad_entries_are_skipped(dev):
    # table and list entries, counts and lengths out of range: reported, left out
    lens = [100, 40]
    c = ref.Cache(lens, 1, 64, 16, 72)
    q = torch.randn(2, 1, 64, generator=torch.Generator().manual_seed(71)).to(BF16)
    pp = ab.PagedParams(2, 1, 1, 64, 16, c.num_pages, c.max_pages)
    args = [t.to(dev) for t in (q, c.K, c.V)]
    good = ab.ab_attention_paged(pp, *args, c.table.to(dev), ints(lens, dev))
    for wrong in (-1, c.num_pages, 2 ** 31 - 1):
        table = c.table.clone()
        table[0, 2] = wrong
        O = ab.ab_attention_paged(pp, *args, table.to(dev), ints(lens, dev))
        assert ab.device_error(dev) == CAPACITY
        _check_attention(O.cpu(), q, c, lists=[[[0, 1, 3, 4, 5, 6]], [[0, 1, 2]]])
        assert torch.equal(O[1], good[1])
        P = ab.ab_paged_select(pp, args[0], c.ksum.to(dev), table.to(dev), ints(lens, dev))
        assert ab.device_error(dev) == CAPACITY and torch.isfinite(P[1]).all()
    O = ab.ab_attention_paged(pp, *args, c.table.to(dev), ints([16 * c.max_pages + 1, 40], dev))
    assert ab.device_error(dev) == CAPACITY and (O[0] == 0).all() and torch.equal(O[1], good[1])
    idx = torch.zeros(2, 1, c.max_pages, dtype=I32)
    idx[0, 0, :3] = torch.tensor([1, 7, -2], dtype=I32)
    O = ab.ab_attention_paged(pp, *args, c.table.to(dev), ints(lens, dev), idx=idx.to(dev), count=ints([[3], [1]], dev))
    assert ab.device_error(dev) == CAPACITY
    _check_attention(O.cpu(), q, c, lists=[[[1]], [[0]]])
    O = ab.ab_attention_paged(pp, *args, c.table.to(dev), ints(lens, dev), idx=idx.to(dev), count=ints([[-1], [1]], dev))
    assert ab.device_error(dev) == CAPACITY and (O[0] == 0).all()
    _check_attention(O.cpu(), q, c, lists=[[[]], [[0]]])


@pytest.mark.parametrize("max_pages", [300, 1500])
def test_select_bad_entries(dev, max_pages):
    # an entry out of range has the score of a zero summary; other rows are as they were
    lens = [4700, 40, 0, 4000]
    Hq, Hkv, d, page = 6, 2, 64, 16
    c = ref.Cache(lens, Hkv, d, page, 73, max_pages=max_pages)
    q = torch.randn(4, Hq, d, generator=torch.Generator().manual_seed(74)).to(BF16)
    pp = ab.PagedParams(4, Hq, Hkv, d, page, c.num_pages, c.max_pages)
    ksum = torch.cat([c.ksum, torch.zeros(1, Hkv, d, dtype=BF16)])
    run = lambda pp, k, t: ab.ab_paged_select(pp, q.to(dev), k.to(dev), t.to(dev), ints(lens, dev),
                                              out=torch.full((4, Hkv, max_pages), -1.0, device=dev)).cpu()
    for wrong in (-1, c.num_pages, 2 ** 31 - 1):
        table, zero = c.table.clone(), c.table.clone()
        table[0, 5], zero[0, 5] = wrong, c.num_pages
        got = run(pp, c.ksum, table)
        assert ab.device_error(dev) == CAPACITY
        want = run(ab.PagedParams(4, Hq, Hkv, d, page, c.num_pages + 1, c.max_pages), ksum, zero)
        assert ab.device_error(dev) == 0 and torch.equal(got, want)


# -------------------------------------------------------------- together
@pytest.mark.parametrize("graph", [False, True])
def test_steps_together(dev, graph):
    """Prompts, then single tokens, a request that ends and one that joins: plan
    and the sparse step, eager or as one captured graph that is replayed."""
    S, Hq, Hkv, d, page = 5, 8, 2, 64, 16
    pp = ab.PagedParams(S, Hq, Hkv, d, page, 60, 20, keep_ratio=0.3, recent=1)
    cache = ab.PagedCache(pp, dev)
    cache.K.fill_(float("nan")), cache.V.fill_(float("nan")), cache.ksum.fill_(float("nan"))
    (wq, wk, cos, sin), nr = _rope("head", Hq, Hkv, d, 320, False, 81, dev)
    g = torch.Generator().manual_seed(82)
    steps = [[100, 40, 0, 7, 200], [1, 1, 64, 0, 1], [1, -1, 1, 1, 1], [0, 30, 1, 1, 1], [1, 1, 1, 1, 1]]
    T = 360
    n_new = torch.zeros(S, dtype=I32, device=dev)
    x = torch.zeros(T, Hq + 2 * Hkv, d, dtype=BF16, device=dev)
    lists = (torch.zeros(S + 1, dtype=I32, device=dev), torch.zeros(T, dtype=I32, device=dev), torch.zeros(T, dtype=I32, device=dev))
    bufs = ab.PagedBuffers(pp, T, dev)

    def step():
        ab.ab_paged_plan(pp, n_new, cache.lens, cache.table, cache.free_pages, cache.free_count, out=lists)
        ab.ab_paged_forward(pp, nr, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cache, *lists, bufs=bufs)

    run = step
    if graph:
        step()  # with no new tokens: nothing changes
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step()
        run = gr.replay
    keys, values = [torch.zeros(0, Hkv, d, dtype=BF16) for _ in range(S)], [torch.zeros(0, Hkv, d, dtype=BF16) for _ in range(S)]
    for new in steps:
        xc = torch.randn(T, Hq + 2 * Hkv, d, generator=g).to(BF16)
        n_new.copy_(ints(new, dev))
        x.copy_(xc)
        before = bufs.O.clone()
        run()
        torch.cuda.synchronize()
        assert ab.device_error(dev) == 0
        # the reference takes the rounded keys from the cache, checked on the way
        at = 0
        lens, table, count, idx, O = (t.cpu() for t in (cache.lens, cache.table, bufs.count, bufs.idx, bufs.O))
        Kc, Vc, P, Q = (t.cpu() for t in (cache.K, cache.V, bufs.P, bufs.Q))
        for s, m in enumerate(new):
            if m == -1:
                keys[s], values[s] = keys[s][:0], values[s][:0]
            m = max(m, 0)
            n0 = len(keys[s])
            assert lens[s] == n0 + m
            if m == 0:
                assert torch.equal(O[s], before[s].cpu())
                continue
            pos = torch.arange(n0, n0 + m)
            sl = table[s, pos // page].long()
            got = Kc[sl, :, pos % page]
            k, size = ref.norm_rotate(xc[at:at + m, Hq:Hq + Hkv], "head", wk, cos, sin, pos, False, 1e-6)
            ref.assert_norm_rotate(got, k, size, "head", d)
            assert torch.equal(Vc[sl, :, pos % page], xc[at:at + m, Hq + Hkv:])
            keys[s], values[s] = torch.cat((keys[s], got)), torch.cat((values[s], xc[at:at + m, Hq + Hkv:]))
            at += m
            q = Q[at - 1]
            n = len(keys[s])
            pages = ref.cdiv(n, page)
            for h in range(Hkv):
                ks = keys[s][:, h]
                sums = torch.stack([ks[j * page:(j + 1) * page].float().mean(0) for j in range(pages)])
                p, _ = ref.select(q[4 * h:4 * h + 4], sums, n, page, d)
                # means in bf16: scores off by up to 2^-8 sum |q kbar| / sqrt(d)
                a = (q[4 * h:4 * h + 4].abs().double() @ sums.abs().double().T / d ** 0.5).max().item()
                assert ((P[s, h, :pages].double() - p).abs() <= 1.01 * 2 * (2.0 ** -7.9) * a * p + 1e-6).all()
                want = ref.topk(P[s, h], pages, 0.3, 1)
                assert idx[s, h, :count[s, h]].tolist() == want
                rows = [i for j in want for i in range(j * page, min((j + 1) * page, n))]
                o, size, eps = ref.attention(q[4 * h:4 * h + 4], ks[rows], values[s][rows, h], d)
                ref.assert_attention(O[s, 4 * h:4 * h + 4], o, size, eps, len(rows))


def test_other_stream_and_shared_workspace(dev):
    lens = [900, 20]
    c = ref.Cache(lens, 2, 128, 32, 92)
    q = torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(91)).to(BF16)
    pp = ab.PagedParams(2, 8, 2, 128, 32, c.num_pages, c.max_pages)
    args = [t.to(dev) for t in (q, c.K, c.V, c.table)] + [ints(lens, dev)]
    want = ab.ab_attention_paged(pp, *args)
    ws = ab.alloc_paged_workspace(pp, dev)
    st = torch.cuda.Stream(dev)
    st.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(st):
        O = ab.ab_attention_paged(pp, *args, workspace=ws)
        ab.ab_paged_select(pp, args[0], c.ksum.to(dev), *args[3:], workspace=ws)  # the same workspace, other contents
        O2 = ab.ab_attention_paged(pp, *args, workspace=ws)
    torch.cuda.current_stream(dev).wait_stream(st)
    assert torch.equal(O, want) and torch.equal(O2, want)


def test_offsets_beyond_32_bits(dev):
    # K and V of 2.3e9 elements each, the sequence in the last pages
    num_pages, Hkv, page, d = 70000, 4, 64, 128
    K, V = (torch.zeros(num_pages, Hkv, page, d, dtype=BF16, device=dev) for _ in range(2))
    ksum = torch.zeros(num_pages, Hkv, d, dtype=BF16, device=dev)
    lens = [300, 7]
    c = ref.Cache(lens, Hkv, d, page, 95)
    c.table = torch.where(c.table >= 0, c.table + (num_pages - c.num_pages), c.table)
    for t, small in ((K, c.K), (V, c.V), (ksum, c.ksum)):
        t[num_pages - c.num_pages:] = small.to(dev)
    pp = ab.PagedParams(2, 8, Hkv, d, page, num_pages, c.max_pages)
    q = torch.randn(2, 8, d, generator=torch.Generator().manual_seed(96)).to(BF16)
    O = ab.ab_attention_paged(pp, q.to(dev), K, V, c.table.to(dev), ints(lens, dev))
    _check_attention(O.cpu(), q, c)
    small_pp = ab.PagedParams(2, 8, Hkv, d, page, c.num_pages, c.max_pages)
    small_table = torch.where(c.table >= 0, c.table - (num_pages - c.num_pages), c.table).to(dev)
    assert torch.equal(ab.ab_paged_select(pp, q.to(dev), ksum, c.table.to(dev), ints(lens, dev)),
                       ab.ab_paged_select(small_pp, q.to(dev), c.ksum.to(dev), small_table, ints(lens, dev)))
    # one more token, in the last slot of the cache
    x = torch.randn(1, 16, d, generator=torch.Generator().manual_seed(97)).to(BF16).to(dev)
    slot = num_pages * page - 1
    Q = ab.ab_paged_append(pp, ab.NormRope("none"), x[:, :8], x[:, 8:12], x[:, 12:], ints([slot], dev), ints([0], dev), K, V, ksum=ksum)
    assert torch.equal(Q, x[:, :8]) and torch.equal(K[-1, :, -1], x[0, 8:12]) and torch.equal(V[-1, :, -1], x[0, 12:])
    mean = K[-1].double().mean(1)
    assert torch.isnan(mean).any() or ((ksum[-1].double() - mean).abs() <= 2 * ref.HALF * mean.abs() + 1e-5).all()


def test_two_streams_at_once(dev):
    # calls that overlap, each with its own workspace
    g = torch.Generator().manual_seed(98)
    work = []
    for k in range(2):
        lens = [3000 + 999 * k, 50, 2000]
        c = ref.Cache(lens, 2, 64, 16, 99 + k)
        q = torch.randn(3, 6, 64, generator=g).to(BF16)
        pp = ab.PagedParams(3, 6, 2, 64, 16, c.num_pages, c.max_pages, keep_ratio=0.4)
        args = [t.to(dev) for t in (q, c.K, c.V, c.table, c.ksum)] + [ints(lens, dev)]
        work.append((pp, c, q, args, ab.alloc_paged_workspace(pp, dev), torch.cuda.Stream(dev)))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for k, (pp, c, q, (Q, K, V, table, ksum, lens), ws, st) in enumerate(work):
            with torch.cuda.stream(st):
                P = ab.ab_paged_select(pp, Q, ksum, table, lens, workspace=ws)
                idx, count = ab.ab_paged_topk(pp, P, lens)
                got[k].append((ab.ab_attention_paged(pp, Q, K, V, table, lens, workspace=ws),
                               ab.ab_attention_paged(pp, Q, K, V, table, lens, idx=idx, count=count, workspace=ws)))
    torch.cuda.synchronize()
    for k, (pp, c, q, *_) in enumerate(work):
        _check_attention(got[k][0][0].cpu(), q, c)
        for O, S in got[k][1:]:
            assert torch.equal(O, got[k][0][0]) and torch.equal(S, got[k][0][1])


def test_two_graphs_share_a_workspace(dev):
    cases = []
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=dev)
    for k, (Hq, d, page, lens) in enumerate(((4, 128, 16, [700, 3]), (12, 64, 32, [64, 1500, 0]))):
        c = ref.Cache(lens, 2 if k == 0 else 1, d, page, 110 + k)
        q = torch.randn(len(lens), Hq, d, generator=torch.Generator().manual_seed(k)).to(BF16)
        pp = ab.PagedParams(len(lens), Hq, c.Hkv, d, page, c.num_pages, c.max_pages)
        w = ab.alloc_paged_workspace(pp, dev) if ws.numel() < ab.paged_workspace_size(pp) else ws
        ws = w
        cases.append((pp, c, q, [t.to(dev) for t in (q, c.K, c.V, c.table)] + [ints(lens, dev)]))
    graphs = []
    for pp, c, q, args in cases:
        O = torch.zeros(len(c.lens), pp.Hq, pp.d, dtype=BF16, device=dev)
        ab.ab_attention_paged(pp, *args, workspace=ws, out=O)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            ab.ab_attention_paged(pp, *args, workspace=ws, out=O)
        graphs.append((gr, O))
    for _ in range(5):
        for gr, O in graphs:
            O.zero_()
            gr.replay()
    for (gr, O), (pp, c, q, args) in zip(graphs, cases):
        _check_attention(O.cpu(), q, c)
        # other lengths in the same graph
        args[4].clamp_(max=1)
        gr.replay()
        torch.cuda.synchronize()
        short = ref.Cache.__new__(ref.Cache)
        short.__dict__.update(c.__dict__)
        short.lens = [min(n, 1) for n in c.lens]
        short.keys = [k[:1] for k in c.keys]
        short.values = [v[:1] for v in c.values]
        _check_attention(O.cpu(), q, short)


def test_captured_between_copies_and_streams(dev):
    # a graph with fills and copies before the calls, and two branches that meet again
    lens = [3000, 50, 0, 700]
    c = ref.Cache(lens, 2, 64, 16, 120)
    q = torch.randn(4, 6, 64, generator=torch.Generator().manual_seed(121)).to(BF16)
    pp = ab.PagedParams(4, 6, 2, 64, 16, c.num_pages, c.max_pages, keep_ratio=0.3, recent=1)
    K, V, ksum, table = (t.to(dev) for t in (c.K, c.V, c.ksum, c.table))
    source = q.to(dev)
    Q, n = torch.zeros_like(source), torch.zeros(4, dtype=I32, device=dev)
    lens_in = ints(lens, dev)
    P = torch.zeros(4, 2, c.max_pages, device=dev)
    lists = torch.zeros(4, 2, c.max_pages, dtype=I32, device=dev), torch.zeros(4, 2, dtype=I32, device=dev)
    all_O, some_O = torch.zeros_like(source), torch.zeros_like(source)
    ws = [ab.alloc_paged_workspace(pp, dev) for _ in range(2)]
    side = torch.cuda.Stream(dev)

    def step():
        here = torch.cuda.current_stream(dev)
        Q.copy_(source)
        n.copy_(lens_in)
        P.zero_()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            ab.ab_attention_paged(pp, Q, K, V, table, n, workspace=ws[1], out=all_O)
        ab.ab_paged_select(pp, Q, ksum, table, n, out=P, workspace=ws[0])
        ab.ab_paged_topk(pp, P, n, out=lists)
        ab.ab_attention_paged(pp, Q, K, V, table, n, idx=lists[0], count=lists[1], workspace=ws[0], out=some_O)
        here.wait_stream(side)
        all_O.add_(some_O)
        n.zero_()

    step()
    torch.cuda.synchronize()
    want = all_O.clone(), some_O.clone()
    assert all(torch.isfinite(w).all() and (w[0] != 0).any() for w in want)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step()
    for _ in range(3):
        for t in (all_O, some_O, Q, P):
            t.fill_(-3)
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(all_O, want[0]) and torch.equal(some_O, want[1])
