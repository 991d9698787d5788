"""Tensors that the binding of the norm, the rotation and the paged cache refuses,
on the GPU: one that does not fit in each place of each call, which raises before
anything is enqueued."""
import pytest

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


S, T, HQ, HKV, D, PAGE, PAGES, COLS = 3, 5, 4, 2, 64, 16, 11, 6
PP = ab.PagedParams(S, HQ, HKV, D, PAGE, PAGES, COLS)


def _wrong(t):
    """Tensors that differ from t in one thing each."""
    yield "another dtype", t.to(torch.float16 if t.dtype != torch.float16 else torch.float32)
    yield "a longer first dimension", torch.cat([t, t[:1]])
    yield "a shorter last dimension", t[..., :-1].contiguous()
    yield "one dimension more", t[None]
    wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype, device=t.device)
    yield "a stride in the last dimension", wide[..., ::2]
    yield "on the CPU", t.cpu()
    yield "no tensor", t.tolist()


def _calls(dev):
    z = lambda *shape, dtype=I32: torch.zeros(*shape, dtype=dtype, device=dev)  # noqa: E731
    b = lambda *shape: z(*shape, dtype=BF16)  # noqa: E731
    f = lambda *shape: z(*shape, dtype=torch.float32)  # noqa: E731
    nr = ab.NormRope("none")
    kv, rows = (PAGES, HKV, PAGE, D), (S, HKV, COLS)
    n = ab.paged_workspace_size(PP)
    ws = z(n, dtype=torch.uint8)
    p = ab.Params(B=2, H=HQ, L=7, d=D, L_kv=9, q_block=64, kv_block=16, C=4)
    yield "plan", lambda **a: ab.ab_paged_plan(PP, T=T, out=(a.pop("cu_new"), a.pop("slots"), a.pop("positions")), **a), dict(
        n_new=z(S), lens=z(S), table=z(S, COLS), free_pages=z(PAGES), free_count=z(1), lens_out=z(S), free_count_out=z(1),
        cu_new=z(S + 1), slots=z(T), positions=z(T))
    yield "append", lambda **a: ab.ab_paged_append(PP, nr, **a), dict(
        q=b(T, HQ, D), k=b(T, HKV, D), v=b(T, HKV, D), slots=z(T) - 1, positions=z(T), K=b(*kv), V=b(*kv), ksum=b(PAGES, HKV, D),
        out=b(T, HQ, D))
    yield "select", lambda **a: ab.ab_paged_select(PP, **a), dict(
        Q=b(T, HQ, D), ksum=b(PAGES, HKV, D), table=z(S, COLS), lens=z(S), cu_new=z(S + 1), workspace=ws, out=f(*rows))
    yield "topk", lambda **a: ab.ab_paged_topk(PP, a["P"], a["lens"], out=(a["idx"], a["count"])), dict(
        P=f(*rows), lens=z(S), idx=z(*rows), count=z(S, HKV))
    yield "attention", lambda **a: ab.ab_attention_paged(PP, **a), dict(
        Q=b(T, HQ, D), K=b(*kv), V=b(*kv), table=z(S, COLS), lens=z(S), idx=z(*rows), count=z(S, HKV), cu_new=z(S + 1), workspace=ws,
        out=b(S, HQ, D))

    def forward(**a):
        cache, bufs = ab.PagedCache.__new__(ab.PagedCache), ab.PagedBuffers.__new__(ab.PagedBuffers)
        for name in ("K", "V", "ksum", "table", "lens"):
            setattr(cache, name, a[name])
        cache.ws = ws
        for name in ("Q", "P", "idx", "count", "O"):
            setattr(bufs, name, a[name])
        return ab.ab_paged_forward(PP, nr, a["q"], a["k"], a["v"], cache, a["cu_new"], a["slots"], a["positions"], bufs=bufs)
    yield "forward", forward, dict(
        q=b(T, HQ, D), k=b(T, HKV, D), v=b(T, HKV, D), slots=z(T) - 1, positions=z(T), K=b(*kv), V=b(*kv), ksum=b(PAGES, HKV, D),
        table=z(S, COLS), lens=z(S), cu_new=z(S + 1), Q=b(T, HQ, D), P=f(*rows), idx=z(*rows), count=z(S, HKV), O=b(S, HQ, D))
    yield "norm", lambda **a: ab.ab_qk_norm_rope(p, nr, a["q"], a["k"], a["v"], a["pos_q"], a["pos_k"], out=(a["Q"], a["K"], a["V"])), dict(
        q=b(2, 7, HQ, D), k=b(2, 9, HQ, D), v=b(2, 9, HQ, D), pos_q=z(2, 7), pos_k=z(2, 9), Q=b(2, HQ, 7, D), K=b(2, HQ, 9, D), V=b(2, HQ, 9, D))


@pytest.mark.parametrize("call", ["plan", "append", "select", "topk", "attention", "forward", "norm"])
def test_each_tensor_is_checked(dev, call):
    run, good = next((r, a) for name, r, a in _calls(dev) if name == call)
    run(**good)                                                   # the call itself is right
    torch.cuda.synchronize()
    for name, t in good.items():
        for what, wrong in _wrong(t):
            if name == "workspace" and what in ("a longer first dimension", "a shorter last dimension"):
                continue                                          # its length is its own
            if call in ("select", "attention") and (name, what) == ("Q", "a longer first dimension"):
                continue                                          # so is T, with cu_new
            if t.shape[-1] == 1 and what == "a stride in the last dimension":
                continue                                          # which is not used
            with pytest.raises((ValueError, AttributeError, TypeError)) as e:
                run(**{**good, name: wrong})
            assert e.type is ValueError or what == "no tensor", (name, what, e.value)
            if what in ("another dtype", "a stride in the last dimension") and e.type is ValueError:
                assert "expected" in str(e.value), (name, what)
    run(**good)
    torch.cuda.synchronize()


def test_strides_of_tokens(dev):
    # outer strides that are no multiple of 8, bases off 16 bytes: refused by the library; of dimensions of size 1: not looked at
    p = ab.Params(B=1, H=2, L=4, d=64)
    nr = ab.NormRope("none")
    flat = torch.randn(4096, device=dev).to(BF16)
    for strides, at in (((0, 132, 64, 1), 0), ((0, 128, 68, 1), 0), ((0, 128, 64, 1), 4)):
        with pytest.raises(ab.AbError) as e:
            ab.ab_qk_norm_rope(p, nr, flat.as_strided((1, 4, 2, 64), strides, at))
        assert e.value.status == 1
    x = flat.as_strided((1, 4, 2, 64), (3, 128, 64, 1), 8)
    assert torch.equal(ab.ab_qk_norm_rope(p, nr, x)[0], x.transpose(1, 2))


def test_workspace_too_small(dev):
    z = lambda *shape, dtype=I32: torch.zeros(*shape, dtype=dtype, device=dev)  # noqa: E731
    small = z(16, dtype=torch.uint8)
    with pytest.raises(ab.AbError) as e:
        ab.ab_paged_select(PP, z(S, HQ, D, dtype=BF16), z(PAGES, HKV, D, dtype=BF16), z(S, COLS), z(S), workspace=small)
    assert e.value.status == 6
    kv = z(PAGES, HKV, PAGE, D, dtype=BF16)
    with pytest.raises(ab.AbError) as e:
        ab.ab_attention_paged(PP, z(S, HQ, D, dtype=BF16), kv, kv, z(S, COLS), z(S), workspace=small)
    assert e.value.status == 6


def test_an_output_over_its_inputs_is_refused(dev):
    z = lambda *shape, dtype=I32: torch.zeros(*shape, dtype=dtype, device=dev)  # noqa: E731
    Q, K, V = z(S, HQ, D, dtype=BF16), z(PAGES, HKV, PAGE, D, dtype=BF16), z(PAGES, HKV, PAGE, D, dtype=BF16)
    more = dict(idx=z(S, HKV, COLS), count=z(S, HKV))
    for out in (Q, K.view(-1)[-S * HQ * D:].view(S, HQ, D), V.view(-1)[:S * HQ * D].view(S, HQ, D)):
        for kw in ({}, more):
            with pytest.raises(ab.AbError) as e:
                ab.ab_attention_paged(PP, Q, K, V, z(S, COLS), z(S), out=out, **kw)
            assert e.value.status == 1
    cache, bufs = ab.PagedCache(PP, dev), ab.PagedBuffers(PP, S, dev)
    bufs.O = bufs.Q
    with pytest.raises(ab.AbError) as e:
        ab.ab_paged_forward(PP, ab.NormRope("none"), Q.clone(), z(S, HKV, D, dtype=BF16), z(S, HKV, D, dtype=BF16), cache, z(S + 1),
                            z(S) - 1, z(S), bufs=bufs)
    assert e.value.status == 1
