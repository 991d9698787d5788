"""Refusals and arguments of the norm and rotation that the library and the
binding decide on the host (pointers here are never read)."""
import pytest

import block_sparse_attention_queries_b200 as ab
from block_sparse_attention_queries_b200 import build as abbuild

GOOD, IN = 0x1000, 0x40000000
OUT = (0x1000, 0x1000000, 0x2000000)


@pytest.fixture(scope="module")
def lib():
    abbuild.build()
    return ab.lib()


def _nr(**kw):
    a = dict(norm=1, interleaved=0, eps=1e-6, n_pos=100, wq=GOOD, wk=None, cos_table=GOOD, sin_table=GOOD)
    a.update(kw)
    return ab.ab_norm_rope(*a.values())


def test_tables_without_rows_are_refused(lib):
    p = ab.Params(B=1, H=4, L=5, d=64, q_block=64, kv_block=16, C=4)
    t = ab.ab_tokens(IN, 0, 256, 64)
    empty = _nr(n_pos=0)
    assert lib.ab_qk_norm_rope(p.c(), empty, t, None, None, GOOD, None, *OUT, None) == 1
    assert lib.ab_forward_qkv(p.c(), empty, t, t, t, GOOD, GOOD, *OUT, *[GOOD] * 6, 1 << 45, None) == 1
    pp = ab.PagedParams(S=4, Hq=4, Hkv=4, d=64, page=16, num_pages=100, max_pages=20)
    assert lib.ab_paged_append(pp.c(), empty, 5, t, t, t, *[GOOD] * 6, None) == 1
    assert lib.ab_paged_append(pp.c(), empty, 0, None, None, None, *[None] * 6, None) == 1
    assert lib.ab_paged_forward(pp.c(), empty, 5, t, t, t, *[GOOD] * 14, 1 << 45, None) == 1


@pytest.mark.parametrize("rest", [dict(q_block=0), dict(q_block=96), dict(q_block=-5),
                                  dict(kv_block=7, C=3, kmeans_iters=-1, keep_ratio=9.0),
                                  dict(q_block=0, kv_block=0, C=0, kmeans_iters=0, keep_ratio=0.0)])
def test_only_the_documented_sizes_count(lib, rest):
    # B, H, L, L_kv and d: what is refused here is refused for what stands behind them (too few rows: 1, too many heads: 2)
    t = ab.ab_tokens(IN, 50 * 256, 256, 64)
    p = ab.Params(B=2, H=4, L=50, d=64, **rest).c()
    assert lib.ab_qk_norm_rope(p, _nr(n_pos=49), t, None, None, None, None, *OUT, None) == 1
    p = ab.Params(B=2, H=257, L=50, d=128, **rest).c()
    assert lib.ab_qk_norm_rope(p, _nr(), t, None, None, None, None, *OUT, None) == 2


class _OnDevice:
    """What NormRope looks at in a tensor, without a GPU."""

    def __init__(self, *shape):
        import torch
        self.shape, self.dtype, self.device, self.is_cuda = torch.Size(shape), torch.float32, "cuda:0", True

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0

    at = GOOD

    def data_ptr(self):
        return self.at if self.shape.numel() else 0


def test_binding_refuses_tables_without_rows():
    pytest.importorskip("torch")
    assert ab.NormRope("none", cos=_OnDevice(1, 32), sin=_OnDevice(1, 32)).n_pos == 1
    with pytest.raises(ValueError, match="row"):  # their address is null, as if there were no rotation
        ab.NormRope("none", cos=_OnDevice(0, 32), sin=_OnDevice(0, 32))


def test_a_norm_rope_does_not_change():
    # the library's copy holds the tensors' addresses: another table would be ignored, and the first one freed
    pytest.importorskip("torch")
    nr = ab.NormRope("none", cos=_OnDevice(3, 32), sin=_OnDevice(3, 32))
    for name, value in (("cos", _OnDevice(9, 32)), ("sin", None), ("wq", _OnDevice(64)), ("eps", 1e-5), ("norm", "head"), ("n_pos", 9)):
        with pytest.raises(AttributeError):
            setattr(nr, name, value)
    with pytest.raises(AttributeError):
        del nr.cos
    nr.check(4, 2, 64, 0)
    assert nr.n_pos == 3 and nr._c.n_pos == 3


def test_a_tensor_with_other_storage():
    # as after `.data = ...`: the address and the checks are those of the storage that the call meets
    pytest.importorskip("torch")
    w, cos, sin = _OnDevice(64), _OnDevice(3, 32), _OnDevice(3, 32)
    nr = ab.NormRope("head", wq=w, cos=cos, sin=sin)
    nr.check(4, 2, 64, 0)
    w.at = 0x5000
    cos.at, cos.shape, sin.at, sin.shape = 0x6000, type(cos.shape)((9, 32)), 0x7000, type(cos.shape)((9, 32))
    nr.check(4, 2, 64, 0)
    assert (nr._c.wq, nr._c.cos_table, nr._c.sin_table, nr._c.n_pos, nr.n_pos) == (0x5000, 0x6000, 0x7000, 9, 9)
    w.at, w.shape = 0x8000, type(w.shape)((32,))
    with pytest.raises(ValueError, match="fit"):
        nr.check(4, 2, 64, 0)
    w.at, w.is_cuda = 0x9000, False
    with pytest.raises(ValueError, match="CUDA"):
        nr.check(4, 2, 64, 0)


def test_attention_output_over_its_inputs(lib):
    # addresses alone: refused on the host, whatever part overlaps
    pp = ab.PagedParams(S=4, Hq=8, Hkv=2, d=128, page=16, num_pages=100, max_pages=20)
    n, cache, big = 4 * 8 * 128 * 2, 100 * 2 * 16 * 128 * 2, 1 << 45
    Q, K, V = 0x10000000, 0x20000000, 0x30000000
    for at, size in ((Q, n), (K, cache), (V, cache)):
        for O in (at, at - n + 16, at + size - 16):
            assert lib.ab_attention_paged(pp.c(), 4, Q, K, V, GOOD, GOOD, None, None, None, O, GOOD, big, None) == 1
            assert lib.ab_attention_paged(pp.c(), 4, Q, K, V, GOOD, GOOD, None, GOOD, GOOD, O, GOOD, big, None) == 1
            t = ab.ab_tokens(0x50000000, 0, 8 * 128, 128)
            assert lib.ab_paged_forward(pp.c(), _nr(), 4, t, t, t, GOOD, GOOD, GOOD, GOOD, GOOD, Q, K, V, 0x60000000, GOOD, GOOD, GOOD,
                                        O, GOOD, big, None) == 1
