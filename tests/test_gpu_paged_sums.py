"""Sums of the attention over the paged cache on the GPU that a rounding to one
side, or a value that is no finite number, would show in."""
import math

import pytest

import paged_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_sparse_attention_queries_b200 as ab  # noqa: E402

BF16, I32 = torch.bfloat16, torch.int32


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


@pytest.mark.parametrize("Hq,d", [(1, 128), (16, 128), (5, 64)])
@pytest.mark.parametrize("lists", [False, True])
def test_long_sums_round_both_ways(dev, Hq, d, lists):
    """Equal weights, values that rise to a large sum and fall back to 1: what
    remains of n keys is the roundings' own sum.  148 rows over the same pages, so
    that a GPU of 148 SMs has a row in each; with other numbers rows are divided,
    and sums are shorter."""
    S, page, tile = 148, 64, 128
    half = 1000 * tile                                            # keys that rise, as many that fall, one more
    n = 2 * half + 1
    g = torch.Generator().manual_seed(5)
    up = torch.randn(half, d, generator=g).abs().to(BF16)
    values = torch.cat([up, -up, torch.ones(1, d, dtype=BF16)])
    pages = ref.cdiv(n, page)
    V = torch.zeros(pages, 1, page, d, dtype=BF16)
    V.view(-1, d)[:n] = values
    pp = ab.PagedParams(S, Hq, 1, d, page, pages, pages)
    table = torch.arange(pages, dtype=I32).expand(S, -1).contiguous()
    more = {}
    if lists:
        more = dict(idx=table[:, None].contiguous().to(dev), count=torch.full((S, 1), pages, dtype=I32, device=dev))
    O = ab.ab_attention_paged(pp, torch.randn(S, Hq, d, generator=g).to(BF16).to(dev), torch.zeros_like(V).to(dev), V.to(dev),
                              table.to(dev), torch.full((S,), n, dtype=I32, device=dev), **more).double().cpu()
    # A warp's partial sums reach at most the sum of its share of `up`; an fp32
    # addition to nearest errs by at most half a step of that, 2^-24 of the power of
    # two below it, to either side.  With m additions the errors' sum exceeds
    # h sqrt(2 m ln(2/delta)) with probability delta (Hoeffding), delta = 1e-9.
    # Products of a tile are exact to 2^-23 of its values.
    most = up.double().view(-1, 64, d)
    most = torch.stack([most[:, 16 * w:16 * w + 16].sum((0, 1)) for w in range(4)]).amax()
    m = 4 * (ref.cdiv(n, 64) + 8)
    rounded = 2.0 ** -24 * 2.0 ** math.floor(math.log2(most)) * math.sqrt(2 * m * math.log(2e9))
    rounded += 2.0 ** -23 * math.sqrt(m) * 128 * up.max().item()
    assert rounded < 1                                           # of the 1 that remains
    want = 1.0 / n
    off = (O - want).abs().max().item()
    assert off <= (ref.HALF * (1 + rounded) + rounded) * want, (off / want, rounded)


@pytest.mark.parametrize("Hq,Hkv,d,page", [(1, 1, 64, 16), (8, 2, 128, 16), (16, 1, 128, 64), (12, 1, 64, 32)])
@pytest.mark.parametrize("lists", [False, True])
def test_infinite_values_show(dev, Hq, Hkv, d, page, lists):
    # +inf, -inf and NaN values at the first key, in the middle, at the last; rows of one key, of one CTA and of many
    lens = [1, 1, 40, 700, 30000, 90000]
    c = ref.Cache(lens, Hkv, d, page, 31)
    inf = float("inf")
    for s, n in enumerate(lens):
        for h in range(Hkv):
            for at, dim, x in ((0, 0, inf), (n // 2, 1, -inf), (n - 1, 2, inf), (n - 1, 3, -inf), (0, 4, inf), (n - 1, 4, -inf),
                               (n // 3, 5, float("nan")), (n // 4, 6, inf), (n // 5, 6, float("nan")), (n // 6, 7, inf)):
                c.values[s][at, h, dim] = x
        for j in range(ref.cdiv(n, page)):
            m = min(page, n - j * page)
            c.V[c.table[s, j], :, :m] = c.values[s][j * page:j * page + m].transpose(0, 1)
    q = torch.randn(len(lens), Hq, d, generator=torch.Generator().manual_seed(32)).to(BF16)
    pp = ab.PagedParams(len(lens), Hq, Hkv, d, page, c.num_pages, c.max_pages)
    more = {}
    if lists:
        more = dict(idx=torch.arange(c.max_pages, dtype=I32).expand(len(lens), Hkv, -1).contiguous().to(dev),
                    count=torch.tensor([[ref.cdiv(n, page)] * Hkv for n in lens], dtype=I32).to(dev))
    O = ab.ab_attention_paged(pp, *(t.to(dev) for t in (q, c.K, c.V, c.table)), torch.tensor(lens, dtype=I32).to(dev), **more).cpu()
    G = Hq // Hkv
    for s, n in enumerate(lens):
        for h in range(Hkv):
            got = O[s, h * G:(h + 1) * G].double()
            o, size, eps = ref.attention(q[s, h * G:(h + 1) * G], c.keys[s][:, h], c.values[s][:, h], d)
            fine = torch.isfinite(o)
            assert not fine[:, :8].any() or n == 1 and not fine[:, :7].all()
            assert torch.equal(torch.isnan(got), torch.isnan(o))
            assert torch.equal(torch.isinf(got), torch.isinf(o)) and torch.equal(got[torch.isinf(o)], o[torch.isinf(o)])
            ref.assert_attention(torch.where(fine, got, 0.0), torch.where(fine, o, 0.0), torch.where(fine, size, 0.0), eps, n)
