"""Tokens that the append into the paged cache skips, and long lists of slots, on
the GPU against a plain reference in 64 bits."""
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


def _norm_rope(norm, Hq, Hk, d, n_pos, interleaved, seed, dev):
    g = torch.Generator().manual_seed(seed)
    shape = {"none": None, "head": lambda H: (d,), "token": lambda H: (H, d)}[norm]
    wq, wk = (None, None) if shape is None else (1 + 0.3 * torch.randn(shape(H), generator=g) for H in (Hq, Hk))
    a = torch.rand(n_pos, d // 2, generator=g) * 20
    up = lambda t: None if t is None else t.to(dev)  # noqa: E731
    return (wq, wk, a.cos(), a.sin()), ab.NormRope(norm, interleaved, 1e-6, up(wq), up(wk), up(a.cos()), up(a.sin()))


def _same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def _append_and_check(dev, pp, norm, interleaved, n_pos, slots, pos, seed, error=0, fill=()):
    """The call's outputs against the reference; the cache holds NaN before it, and keys in the slots `fill`."""
    T, Hq, Hkv, d, page = len(slots), pp.Hq, pp.Hkv, pp.d, pp.page
    (wq, wk, cos, sin), nr = _norm_rope(norm, Hq, Hkv, d, n_pos, interleaved, seed, dev)
    x = torch.randn(T, Hq + 2 * Hkv, d, generator=torch.Generator().manual_seed(seed + 1)).to(BF16)
    xd = x.to(dev)
    nan = float("nan")
    K, V = (torch.full((pp.num_pages, Hkv, page, d), nan, dtype=BF16, device=dev) for _ in range(2))
    ksum = torch.full((pp.num_pages, Hkv, d), nan, dtype=BF16, device=dev)
    fill = torch.tensor(fill, dtype=torch.long)
    K[(fill // page).to(dev), :, (fill % page).to(dev)] = torch.randn(len(fill), Hkv, d, generator=torch.Generator().manual_seed(seed + 2)).to(BF16).to(dev)
    old = K.cpu(), V.cpu(), ksum.cpu()
    Q = torch.full((T, Hq, d), 7.0, dtype=BF16, device=dev)
    ab.ab_paged_append(pp, nr, xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], torch.tensor(slots, dtype=I32).to(dev),
                       torch.tensor(pos, dtype=I32).to(dev), K, V, ksum=ksum, out=Q)
    assert ab.device_error(dev) == error
    Q, K, V, ksum = (t.cpu() for t in (Q, K, V, ksum))
    sl, at = torch.tensor(slots), torch.tensor(pos)
    ok = (sl >= 0) & (sl < pp.num_pages * page) & (at >= 0) & (at < n_pos)
    assert (Q[~ok] == 7.0).all()
    sl, at, x = sl[ok], at[ok], x[ok]
    q, size = ref.norm_rotate(x[:, :Hq], norm, wq, cos, sin, at, interleaved, 1e-6)
    ref.assert_norm_rotate(Q[ok], q, size, norm, Hq * d)
    k, size = ref.norm_rotate(x[:, Hq:Hq + Hkv], norm, wk, cos, sin, at, interleaved, 1e-6)
    ref.assert_norm_rotate(K[sl // page, :, sl % page], k, size, norm, Hkv * d)
    assert torch.equal(V[sl // page, :, sl % page], x[:, Hq + Hkv:])
    written = torch.zeros(pp.num_pages, page, dtype=torch.bool)
    written[sl // page, sl % page] = True
    for t, t0 in ((K, old[0]), (V, old[1])):
        assert _same_bits(t.transpose(1, 2)[~written], t0.transpose(1, 2)[~written])
    touched = written.any(1)
    assert _same_bits(ksum[~touched], old[2][~touched])
    written[fill // page, fill % page] = True
    w = written[:, None, :, None]
    n = written.sum(1).double()[:, None, None].clamp(min=1)
    keys = torch.where(w, K.double(), 0.0)
    mean, size = keys.sum(2) / n, keys.abs().sum(2) / n
    # a sum of up to 64 terms in fp32, a division, one rounding to bf16
    off = (ksum.double() - mean).abs() - (ref.HALF * mean.abs() + (page + 2) * ref.U * 1.01 * size)
    assert off[touched].max().item() <= 0


@pytest.mark.parametrize("norm,interleaved", [("none", True), ("head", False), ("token", True)])
@pytest.mark.parametrize("Hq,Hkv,d,page", [(4, 2, 64, 16), (9, 9, 128, 64), (8, 1, 128, 32)])
@pytest.mark.parametrize("pages", [3, 90])
def test_skipped_tokens_leave_no_trace(dev, norm, interleaved, Hq, Hkv, d, page, pages):
    # positions out of range at a page's first, middle and last tokens, at all of them, beside slots out of range; the means
    # are those of what was written (the cache is new: the other places hold NaN)
    n_pos, T = 50, pages * page
    slots = [page + t for t in range(T)]
    pos = [t % n_pos for t in range(T)]
    for p in range(0, pages, 3):
        pos[p * page] = -1
        pos[p * page + page // 2] = n_pos
        pos[p * page + page - 1] = 2 ** 31 - 1
    for t in range(page, 2 * page):
        pos[t] = n_pos + t
    if pages > 3:
        for t in range(6 * page, 7 * page):
            pos[t] = 3 if t == 6 * page + 5 else -5               # one is left
        for t in range(8 * page + page // 2, 9 * page):
            slots[t] = -1                                          # behind a sequence's last token
        slots[11 * page - 1] = 2 ** 31 - 1
    pp = ab.PagedParams(1, Hq, Hkv, d, page, pages + 2, pages + 2)
    _append_and_check(dev, pp, norm, interleaved, n_pos, slots, pos, 40, CAPACITY)


def test_steps_without_a_new_token(dev):
    # requests that end and none that goes on: the step gives pages back and leaves everything else alone
    pp = ab.PagedParams(3, 4, 2, 64, 16, 20, 10, keep_ratio=0.5)
    _, nr = _norm_rope("head", 4, 2, 64, 160, True, 60, dev)
    cache = ab.PagedCache(pp, dev)
    cache.K.zero_(), cache.V.zero_(), cache.ksum.zero_()
    x = torch.randn(40, 8, 64, generator=torch.Generator().manual_seed(61)).to(BF16).to(dev)

    def step(n_new, T, bufs):
        lists = ab.ab_paged_plan(pp, torch.tensor(n_new, dtype=I32).to(dev), cache.lens, cache.table, cache.free_pages,
                                 cache.free_count, T=T)
        y = x[:T]
        return lists, ab.ab_paged_forward(pp, nr, y[:, :4], y[:, 4:6], y[:, 6:], cache, *lists, bufs=bufs)

    step([20, 17, 3], 40, None)
    bufs = ab.PagedBuffers(pp, 0, dev)
    for t in (bufs.P, bufs.O):
        t.fill_(5)
    for t in (bufs.idx, bufs.count):
        t.fill_(5)
    before = [t.clone() for t in (cache.K, cache.V, cache.ksum)]
    (cu, slots, pos), got = step([-1, 0, -1], 0, bufs)
    assert got is bufs and all((t == 5).all() for t in (bufs.P, bufs.O, bufs.idx, bufs.count))
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.K, cache.V, cache.ksum)))
    assert cache.lens.tolist() == [0, 17, 0] and cache.free_count.item() == 18 and cu.tolist() == [0] * 4
    new = step([0, 0, -1], 0, None)[1]
    assert new.Q.shape == (0, 4, 64) and not new.O.any() and not new.count.any()
    Q = torch.zeros(0, 4, 64, dtype=BF16, device=dev)
    assert not ab.ab_paged_select(pp, Q, cache.ksum, cache.table, cache.lens, cu_new=cu).any()
    assert not ab.ab_attention_paged(pp, Q, cache.K, cache.V, cache.table, cache.lens, cu_new=cu).any()
    with pytest.raises(ValueError):
        ab.ab_paged_select(pp, Q, cache.ksum, cache.table, cache.lens)


@pytest.mark.parametrize("Hq,Hkv,d,page", [(4, 2, 64, 16), (16, 1, 128, 64)])
def test_reading_calls_share_pages(dev, Hq, Hkv, d, page):
    # two sequences on one beginning, each with pages of its own behind it: as if the shared pages were copied, and a token
    # of one of them, appended to its own page, changes nothing for the other
    shared, own = 5, (3, 7)
    lens = [(shared + k) * page - 5 for k in own]
    c = ref.Cache(lens, Hkv, d, page, 70)
    table = c.table.clone()
    table[1, :shared] = table[0, :shared]
    K, V, ksum = c.K.clone(), c.V.clone(), c.ksum.clone()
    K[c.table[1, :shared].long()] = K[c.table[0, :shared].long()]
    V[c.table[1, :shared].long()] = V[c.table[0, :shared].long()]
    ksum[c.table[1, :shared].long()] = ksum[c.table[0, :shared].long()]
    pp = ab.PagedParams(2, Hq, Hkv, d, page, c.num_pages, c.max_pages, keep_ratio=0.4)
    g = torch.Generator().manual_seed(71)
    q = torch.randn(2, Hq, d, generator=g).to(BF16).to(dev)
    up = lambda *t: [x.to(dev) for x in t]  # noqa: E731
    K, V, ksum, copied, table, n = up(K, V, ksum, c.table, table, torch.tensor(lens, dtype=I32))

    def read(table, n):
        P = ab.ab_paged_select(pp, q, ksum, table, n)
        idx, count = ab.ab_paged_topk(pp, P, n)
        return P, idx, ab.ab_attention_paged(pp, q, K, V, table, n), ab.ab_attention_paged(pp, q, K, V, table, n, idx=idx, count=count)

    want = read(copied, n)
    assert all(torch.equal(a, b) for a, b in zip(read(table, n), want))
    x = torch.randn(1, Hq + 2 * Hkv, d, generator=g).to(BF16).to(dev)
    slot = int(c.table[0, (lens[0]) // page]) * page + lens[0] % page
    ab.ab_paged_append(pp, ab.NormRope("none"), x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], torch.tensor([slot], dtype=I32).to(dev),
                       torch.tensor([lens[0]], dtype=I32).to(dev), K, V, ksum=ksum)
    n[0] += 1
    for a, b in zip(read(table, n), want):
        assert torch.equal(a[1], b[1]) and not torch.equal(a[0].float(), b[0].float()) or a.dtype == I32


@pytest.mark.parametrize("wrong", [-1, 8, 2 ** 31 - 1])
def test_plan_reports_bad_pages_that_come_back(dev, wrong):
    # an ended sequence whose table names a page that the cache does not have; handed out again, its tokens have no slot
    pp = ab.PagedParams(2, 1, 1, 64, 16, 8, 4)
    up = lambda v: torch.tensor(v, dtype=I32).to(dev)  # noqa: E731
    table, free, count, lens = up([[3, wrong, -9, -9], [-9] * 4]), up([0, 1, -5, -5, -5, -5, -5, -5]), up([2]), up([20, 0])
    cu, slots, pos = ab.ab_paged_plan(pp, up([-1, 0]), lens, table, free, count, T=4)
    assert ab.device_error(dev) == CAPACITY
    assert free.tolist()[:4] == [0, 1, 3, wrong] and count.item() == 4 and lens.tolist() == [0, 0] and slots.tolist() == [-1] * 4
    cu, slots, pos = ab.ab_paged_plan(pp, up([20, 0]), lens, table, free, count, T=24)
    assert ab.device_error(dev) == CAPACITY
    assert slots.tolist() == [-1] * 16 + [48, 49, 50, 51] + [-1] * 4 and table.tolist()[0][:2] == [wrong, 3]


@pytest.mark.parametrize("norm", ["none", "head", "token"])
@pytest.mark.parametrize("Hq,Hkv,d,page,T", [(3, 1, 64, 64, 1500), (9, 9, 128, 16, 2500), (2, 1, 64, 32, 40000), (2, 1, 64, 64, 40000)])
def test_long_lists_of_slots(dev, norm, Hq, Hkv, d, page, T):
    # several pages a CTA of the means, and pages whose slots lie in two CTAs' parts of the list; sequences of all lengths in
    # pages in random order, that begin inside a page, and slots without a token behind them
    g = torch.Generator().manual_seed(80)
    pages = torch.randperm(T // page * 3, generator=g).tolist()
    num_pages = len(pages)
    slots, pos = [], []
    for n in [1, page - 1, page, page + 1, 5, 3 * page + 7] * (T // (9 * page) + 1) + [T]:
        at = int(torch.randint(0, page, (1,), generator=g))       # keys that the sequence has
        for i in range(at, at + n):
            if i == at or i % page == 0:
                first = pages.pop() * page
            slots.append(first + i % page)
            pos.append(i % 200)
        if len(slots) > T - 20:
            break
    slots, pos = slots[:T - 20] + [-1] * 20, pos[:T - 20] + [0] * 20
    # the keys before a sequence's first are in its first page's mean: written, in a call before
    before = [(s, i) for s in range(T - 20) if s == 0 or slots[s] != slots[s - 1] + 1 and slots[s] % page for i in range(slots[s] % page)]
    pp = ab.PagedParams(1, Hq, Hkv, d, page, num_pages, num_pages)
    fill = [slots[s] - slots[s] % page + i for s, i in before]
    _append_and_check(dev, pp, norm, True, 200, slots, pos, 81, fill=fill)


def test_page_means_beyond_32_bits(dev):
    # K of 2.3e9 elements: the mean of the last page's keys
    num_pages, Hkv, page, d = 70000, 4, 64, 128
    K, V = (torch.zeros(num_pages, Hkv, page, d, dtype=BF16, device=dev) for _ in range(2))
    ksum = torch.zeros(num_pages, Hkv, d, dtype=BF16, device=dev)
    K[-1] = torch.randn(Hkv, page, d, generator=torch.Generator().manual_seed(90)).to(BF16).to(dev)
    pp = ab.PagedParams(1, 8, Hkv, d, page, num_pages, 10)
    x = torch.randn(1, 16, d, generator=torch.Generator().manual_seed(91)).to(BF16).to(dev)
    ab.ab_paged_append(pp, ab.NormRope("none"), x[:, :8], x[:, 8:12], x[:, 12:], torch.tensor([num_pages * page - 1], dtype=I32).to(dev),
                       torch.zeros(1, dtype=I32, device=dev), K, V, ksum=ksum)
    assert torch.equal(K[-1, :, -1], x[0, 8:12])
    keys = K[-1].double()
    off = (ksum[-1].double() - keys.mean(1)).abs() - (ref.HALF * keys.mean(1).abs() + (page + 2) * ref.U * 1.01 * keys.abs().mean(1))
    assert off.max().item() <= 0 and not ksum[:-1].any()
