"""Norm and rotation into the attention's layout on the GPU, against a plain
reference in 64 bits, and the path from the projections."""
import pytest

import paged_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_sparse_attention_queries_b200 as ab  # noqa: E402

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.fail("no CUDA device")
    from block_sparse_attention_queries_b200 import build as abbuild
    abbuild.build()
    ab.lib()
    return torch.device("cuda:0")


def _setup(norm, H, d, n_pos, seed, weights=True, rotate=True):
    g = torch.Generator().manual_seed(seed)
    shape = (H, d) if norm == "token" else (d,)
    w = [1 + 0.3 * torch.randn(shape, generator=g) if weights and norm != "none" else None for _ in range(2)]
    a = torch.rand(n_pos, d // 2, generator=g) * 50
    cos, sin = (a.cos(), a.sin()) if rotate else (None, None)
    return w, cos, sin


def _nr(norm, interleaved, eps, w, cos, sin, dev):
    up = [None if t is None else t.to(dev) for t in (*w, cos, sin)]
    return ab.NormRope(norm, interleaved, eps, *up)


def _check(got, x, norm, w, cos, sin, pos, interleaved, eps):
    B, L, H, d = x.shape
    for b in range(B):
        y, size = ref.norm_rotate(x[b], norm, w, cos, sin, pos[b], interleaved, eps)
        ref.assert_norm_rotate(got[b].transpose(0, 1).cpu(), y, size, norm, H * d)


@pytest.mark.parametrize("norm", ["none", "head", "token"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,L,Lk,d", [(1, 1, 1, 1, 64), (2, 3, 37, 37, 128), (1, 40, 9, 21, 128), (3, 5, 11, 4, 64), (1, 17, 300, 2, 128)])
def test_norm_rope(dev, norm, interleaved, B, H, L, Lk, d):
    g = torch.Generator().manual_seed(1)
    n_pos = max(L, Lk) + 3
    w, cos, sin = _setup(norm, H, d, n_pos, 2)
    nr = _nr(norm, interleaved, 1e-6, w, cos, sin, dev)
    p = ab.Params(B=B, H=H, L=L, d=d, L_kv=Lk)
    q = torch.randn(B, L, H, d, generator=g).to(BF16)
    kv = (3 * torch.randn(B, Lk, 2, H, d, generator=g)).to(BF16)
    k, v = kv[:, :, 0], kv[:, :, 1]
    kvd = kv.to(dev)
    Q, K, V = ab.ab_qk_norm_rope(p, nr, q.to(dev), kvd[:, :, 0], kvd[:, :, 1])
    pos = [torch.arange(n)[None].expand(B, -1) for n in (L, Lk)]
    _check(Q, q, norm, w[0], cos, sin, pos[0], interleaved, 1e-6)
    _check(K, k, norm, w[1], cos, sin, pos[1], interleaved, 1e-6)
    assert torch.equal(V.cpu(), v.transpose(1, 2))
    # explicit positions, and each tensor alone
    pos = [torch.randint(0, n_pos, (B, n), generator=g, dtype=torch.int32) for n in (L, Lk)]
    Q2, K2, V2 = ab.ab_qk_norm_rope(p, nr, q.to(dev), kvd[:, :, 0], None, pos[0].to(dev), pos[1].to(dev))
    assert V2 is None
    _check(Q2, q, norm, w[0], cos, sin, pos[0], interleaved, 1e-6)
    _check(K2, k, norm, w[1], cos, sin, pos[1], interleaved, 1e-6)
    _, K3, V3 = ab.ab_qk_norm_rope(p, nr, None, kvd[:, :, 0], kvd[:, :, 1], pos_k=pos[1].to(dev))
    assert torch.equal(K3, K2) and torch.equal(V3, V)
    assert torch.equal(ab.ab_qk_norm_rope(p, nr, q.to(dev), pos_q=pos[0].to(dev))[0], Q2)
    assert ab.device_error(dev) == 0


@pytest.mark.parametrize("norm,H,d", [("head", 256, 128), ("token", 256, 128), ("token", 512, 64), ("token", 129, 128), ("none", 70, 64)])
def test_many_heads(dev, norm, H, d):
    w, cos, sin = _setup(norm, H, d, 3, 3)
    nr = _nr(norm, True, 1e-5, w, cos, sin, dev)
    x = torch.randn(1, 3, H, d, generator=torch.Generator().manual_seed(4)).to(BF16)
    Q, _, _ = ab.ab_qk_norm_rope(ab.Params(B=1, H=H, L=3, d=d), nr, x.to(dev))
    _check(Q, x, norm, w[0], cos, sin, [torch.arange(3)], True, 1e-5)
    with pytest.raises(ab.AbError) as e:
        big = torch.zeros(1, 3, 256 * 128 // d + 1, d, dtype=BF16, device=dev)
        ab.ab_qk_norm_rope(ab.Params(B=1, H=big.shape[2], L=3, d=d), ab.NormRope("none"), big)
    assert e.value.status == 2


def test_without_weights_or_rotation_and_zeros(dev):
    x = torch.randn(1, 5, 4, 64, generator=torch.Generator().manual_seed(5)).to(BF16)
    x[0, 2] = 0  # a token of zeros stays zero
    p = ab.Params(B=1, H=4, L=5, d=64)
    pos = [torch.arange(5)]
    for norm in ("head", "token"):
        Q, _, _ = ab.ab_qk_norm_rope(p, ab.NormRope(norm, eps=1e-6), x.to(dev))
        _check(Q, x, norm, None, None, None, pos, True, 1e-6)
        assert not Q[0, :, 2].any()
    Q, _, _ = ab.ab_qk_norm_rope(p, ab.NormRope("none"), x.to(dev))
    assert torch.equal(Q.cpu(), x.transpose(1, 2))


def test_strides(dev):
    # heads outermost, tokens expanded, a slice that begins 16 bytes into a row
    g = torch.Generator().manual_seed(6)
    w, cos, sin = _setup("head", 3, 64, 20, 7)
    nr = _nr("head", False, 1e-6, w, cos, sin, dev)
    p = ab.Params(B=2, H=3, L=20, d=64)
    base = torch.randn(2, 3, 20, 64, generator=g).to(BF16)
    wide = torch.randn(2, 20, 3, 80, generator=g).to(BF16)
    for x, xd in ((base.transpose(1, 2), base.to(dev).transpose(1, 2)), (wide[..., 8:72], wide.to(dev)[..., 8:72]),
                  (wide[:, :1, :, 16:].expand(2, 20, 3, 64), wide.to(dev)[:, :1, :, 16:].expand(2, 20, 3, 64))):
        Q, _, _ = ab.ab_qk_norm_rope(p, nr, xd)
        _check(Q, x, "head", w[0], cos, sin, [torch.arange(20)] * 2, False, 1e-6)


def test_bad_positions_leave_their_rows(dev):
    _, cos, sin = _setup("none", 2, 64, 6, 8)
    nr = _nr("none", True, 0.0, (None, None), cos, sin, dev)
    p = ab.Params(B=1, H=2, L=3, d=64)
    x = torch.randn(1, 3, 2, 64, device=dev).to(BF16)
    Q = torch.zeros(1, 2, 3, 64, dtype=BF16, device=dev)
    pos = torch.tensor([[6, 2, -1]], dtype=torch.int32, device=dev)
    ab.ab_qk_norm_rope(p, nr, x, pos_q=pos, out=(Q, None, None))
    assert ab.device_error(dev) == 4
    assert not Q[0, :, 0].any() and Q[0, :, 1].any() and not Q[0, :, 2].any()


@pytest.mark.parametrize("Lk", [0, 700])
def test_forward_qkv(dev, Lk):
    p = ab.Params(B=1, H=4, L=900, d=64, q_block=64, kv_block=16, C=4, keep_ratio=0.3, L_kv=Lk)
    g = torch.Generator().manual_seed(9)
    w, cos, sin = _setup("token", 4, 64, 900, 10)
    nr = _nr("token", True, 1e-6, w, cos, sin, dev)
    q, k, v = (torch.randn(1, n, 4, 64, generator=g).to(BF16).to(dev) for n in (p.L, p.Lk, p.Lk))
    bufs = ab.ab_forward_qkv(p, nr, q, k, v)
    Q, K, V = ab.ab_qk_norm_rope(p, nr, q, k, v)
    want = ab.ab_forward(p, Q, K, V)
    assert torch.equal(bufs.Q, Q) and torch.equal(bufs.K, K) and torch.equal(bufs.V, V)
    assert torch.equal(bufs.O, want.O) and torch.equal(bufs.count, want.count) and torch.equal(bufs.P, want.P)
    again = ab.ab_forward_qkv(p, nr, q, k, v, bufs=bufs)
    assert again is bufs and torch.equal(bufs.O, want.O)
    assert ab.device_error(dev) == 0


@pytest.mark.parametrize("norm", ["none", "head"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,L,Lk,d", [(1, 17, 3900, 3900, 64), (2, 9, 1500, 2050, 128),             # units of one step, many a warp
                                        (1, 5, 5000, 5000, 64), (2, 9, 6200, 6200, 128), (1, 40, 12500, 12500, 64),
                                        (3, 17, 3000, 800, 64), (1, 19, 2600, 11000, 128)])           # units of a whole token
def test_many_units_a_warp(dev, norm, interleaved, B, H, L, Lk, d):
    # more units than warps: rows, tables and weights of one unit behind another's, with tokens of q, k and v in turn
    # (as many of each) or one list after the other, and head counts that leave a step's rows idle
    g = torch.Generator(device=dev).manual_seed(20)
    n_pos = 300
    w, cos, sin = _setup(norm, H, d, n_pos, 21)
    nr = _nr(norm, interleaved, 1e-6, w, cos, sin, dev)
    w, cos, sin = [None if t is None else t.to(dev) for t in w], cos.to(dev), sin.to(dev)
    p = ab.Params(B=B, H=H, L=L, d=d, L_kv=Lk)
    q = torch.randn(B, L, H, d, generator=g, device=dev).to(BF16)
    kv = torch.randn(B, Lk, 2, H, d, generator=g, device=dev).to(BF16)
    k, v = kv[:, :, 0], kv[:, :, 1]
    pos = [torch.randint(0, n_pos, (B, n), generator=g, dtype=torch.int32, device=dev) for n in (L, Lk)]
    Q, K, V = ab.ab_qk_norm_rope(p, nr, q, k, v, *pos)
    assert torch.equal(V, v.transpose(1, 2))
    for got, x, side in ((Q, q, 0), (K, k, 1)):
        for b in range(B):
            y, size = ref.norm_rotate(x[b], norm, w[side], cos, sin, pos[side][b], interleaved, 1e-6)
            ref.assert_norm_rotate(got[b].transpose(0, 1), y, size, norm, H * d)
    assert ab.device_error(dev) == 0
