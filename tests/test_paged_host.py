"""Refusals of the norm and rotation and of the paged cache: the library finds a
bad argument on the host before anything is enqueued (pointers here are never
read), the binding finds tensors that do not fit."""
import ctypes
import os
import shutil
import subprocess
from dataclasses import replace

import pytest

import block_sparse_attention_queries_b200 as ab
from block_sparse_attention_queries_b200 import build as abbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GOOD, BAD = 0x1000, 0x1008
IN = 0x40000000                       # inputs, apart from the outputs
OUT = (0x1000, 0x1000000, 0x2000000)
BIG = 1 << 45


@pytest.fixture(scope="module")
def lib():
    abbuild.build()
    return ab.lib()


PP = ab.PagedParams(S=4, Hq=8, Hkv=2, d=128, page=16, num_pages=100, max_pages=20)


def _size(lib, pp, select=1):
    n = ctypes.c_size_t(0)
    return lib.ab_paged_workspace_size(pp.c(), select, ctypes.byref(n)), n.value


@pytest.mark.parametrize("field,value,status", [
    ("S", 0, 1), ("S", 8193, 2), ("Hq", 0, 1), ("Hq", 9, 1), ("Hkv", 0, 1), ("Hq", 34, 2), ("d", 96, 2), ("d", 0, 1),
    ("page", 8, 2), ("page", 0, 1), ("page", 128, 2), ("num_pages", 0, 1), ("num_pages", 2 ** 27, 1), ("max_pages", 0, 1),
    ("max_pages", 2 ** 20 + 1, 1), ("recent", -1, 1), ("keep_ratio", 0.0, 1), ("keep_ratio", 1.5, 1), ("keep_ratio", float("nan"), 1),
])
def test_parameters(lib, field, value, status):
    pp = replace(PP, **{field: value})
    assert _size(lib, pp)[0] == status
    assert lib.ab_paged_topk(pp.c(), GOOD, GOOD, GOOD, GOOD, None) == status
    assert lib.ab_paged_plan(pp.c(), 4, *[GOOD] * 10, None) == status


def test_too_many_rows(lib):
    assert _size(lib, replace(PP, S=8192, Hq=9, Hkv=9))[0] == 2
    assert _size(lib, replace(PP, S=1, Hq=65536, Hkv=65536, max_pages=1))[0] == 2
    assert _size(lib, replace(PP, S=8192, Hq=8, Hkv=8, max_pages=4))[0] == 0
    assert _size(lib, replace(PP, S=8192, Hq=8, Hkv=8, max_pages=2 ** 15))[0] == 2   # 2^35 keys of all heads


def test_workspace(lib):
    s, small = _size(lib, PP, 0)
    assert s == 0 and small == ab.paged_workspace_size(PP, select=False)
    wide = replace(PP, S=64, max_pages=10000)
    assert _size(lib, wide, 0)[1] == small                     # the attention's does not grow with the table
    assert _size(lib, wide, 1)[1] >= 64 * 8 * 10000 * 4
    assert lib.ab_paged_workspace_size(PP.c(), 1, None) == 1
    q = [GOOD] * 5
    assert lib.ab_attention_paged(PP.c(), 4, *q, None, None, None, GOOD, GOOD, small - 1, None) == 6
    assert lib.ab_paged_select(wide.c(), 64, *[GOOD] * 4, None, GOOD, GOOD, small, None) == 6


def _each(args):
    """The arguments with one pointer null or misaligned, one after the other."""
    for k in range(len(args)):
        for wrong in (None, BAD):
            yield [*args[:k], wrong, *args[k + 1:]]


def test_pointers(lib):
    for a in _each([GOOD] * 10):
        assert lib.ab_paged_plan(PP.c(), 4, *a, None) == 1
    assert lib.ab_paged_plan(PP.c(), -1, *[GOOD] * 10, None) == 1
    for a in _each([GOOD] * 4):
        assert lib.ab_paged_topk(PP.c(), *a, None) == 1
    for a in _each([GOOD] * 6):                                  # Q, ksum, table, lens, P, workspace
        assert lib.ab_paged_select(PP.c(), 4, *a[:4], None, *a[4:], BIG, None) == 1
    for a in _each([GOOD] * 7):                                  # Q, K, V, table, lens, O, workspace
        assert lib.ab_attention_paged(PP.c(), 4, *a[:5], None, None, None, *a[5:], BIG, None) == 1
    ok = [GOOD] * 5
    for cu, idx, count in ((BAD, None, None), (None, GOOD, None), (None, None, GOOD), (None, BAD, GOOD), (None, GOOD, BAD)):
        assert lib.ab_attention_paged(PP.c(), 4, *ok, cu, idx, count, GOOD, GOOD, BIG, None) == 1
    for cu, T in ((None, 3), (None, 5), (GOOD, 0), (GOOD, -1)):  # rows of Q
        assert lib.ab_attention_paged(PP.c(), T, *ok, cu, None, None, GOOD, GOOD, BIG, None) == 1
        assert lib.ab_paged_select(PP.c(), T, *[GOOD] * 4, cu, GOOD, GOOD, BIG, None) == 1


def _nr(**kw):
    a = dict(norm=1, interleaved=0, eps=1e-6, n_pos=100, wq=GOOD, wk=None, cos_table=GOOD, sin_table=GOOD)
    a.update(kw)
    return ab.ab_norm_rope(*a.values())


BAD_NR = [dict(norm=3), dict(norm=-1), dict(interleaved=2), dict(eps=-1.0), dict(eps=float("nan")), dict(n_pos=-1),
          dict(wq=BAD), dict(wk=BAD), dict(cos_table=BAD), dict(cos_table=None), dict(sin_table=None)]


def test_norm_rope(lib):
    p = ab.Params(B=2, H=4, L=50, d=64).c()
    t = ab.ab_tokens(IN, 50 * 256, 256, 64)

    def call(nr=None, tok=(t, t, t), pos=(None, None), out=OUT, p=p):
        return lib.ab_qk_norm_rope(p, nr or _nr(), *tok, *pos, *out, None)

    for kw in BAD_NR:
        assert call(_nr(**kw)) == 1, kw
    assert lib.ab_qk_norm_rope(p, None, t, t, t, None, None, GOOD, GOOD, GOOD, None) == 1
    assert call(tok=(None, None, None)) == 1
    for wrong in (ab.ab_tokens(None, 8, 8, 8), ab.ab_tokens(BAD, 8, 8, 8), ab.ab_tokens(GOOD, 12, 8, 8), ab.ab_tokens(GOOD, 8, 4, 8),
                  ab.ab_tokens(GOOD, 8, 8, 1)):
        for k in range(3):
            assert call(tok=tuple(wrong if j == k else t for j in range(3))) == 1
    for out in _each(list(OUT)):
        assert call(out=out) == 1
    assert call(pos=(BAD, None)) == 1 and call(pos=(None, BAD)) == 1
    assert call(_nr(n_pos=49)) == 1                              # no positions: every token needs its row
    assert call(p=ab.Params(B=1, H=257, L=50, d=128).c()) == 2
    assert call(p=ab.Params(B=1, H=4, L=50, d=96).c()) == 2
    assert call(p=ab.Params(B=1 << 13, H=1, L=1 << 18, d=64).c(), nr=_nr(n_pos=1 << 18)) == 2  # more CTAs than a grid has


def test_overlapping_outputs(lib):
    # inputs of 50 tokens in a fused projection of 3 x 4 x 64; outputs of 50 x 256 values
    p = ab.Params(B=1, H=4, L=50, d=64).c()
    fused, n = 50 * 768 * 2, 50 * 256 * 2
    t = [ab.ab_tokens(0x100000 + 512 * k, 0, 768, 64) for k in range(3)]
    out = [0x200000 + n * k for k in range(3)]

    for k in range(3):
        for wrong in (0x100000 + 16, 0x100000 + fused - 16, 0x100000 - n + 16, out[k - 1] + 16):
            a = [wrong if j == k else out[j] for j in range(3)]
            assert lib.ab_qk_norm_rope(p, _nr(), *t, None, None, *a, None) == 1, (k, hex(wrong))
    paged = [ab.ab_tokens(0x100000 + 2048 * k, 0, 1536, 128) for k in range(3)]
    for wrong in (0x100000, 0x100000 + 16):
        assert lib.ab_paged_append(PP.c(), _nr(), 5, *paged, GOOD, GOOD, wrong, GOOD, GOOD, None, None) == 1


def test_append_and_forward(lib):
    t = ab.ab_tokens(IN, 0, 8 * 128, 128)
    nr = _nr()

    def append(T=5, tok=(t, t, t), ptr=(GOOD,) * 6, nr=nr, pp=PP):
        return lib.ab_paged_append(pp.c(), nr, T, *tok, *ptr, None)

    for kw in BAD_NR:
        assert append(nr=_nr(**kw)) == 1
        assert append(T=0, nr=_nr(**kw)) == 1
    assert append(T=0, tok=(None,) * 3, ptr=(None,) * 6) == 0    # no tokens: nothing to do
    assert append(T=-1) == 1
    for ptr in _each([GOOD] * 5):                                # slots, positions, Q, K, V
        assert append(ptr=(*ptr, GOOD)) == 1
    assert append(ptr=(*[GOOD] * 5, BAD)) == 1
    for k in range(3):
        for wrong in (None, ab.ab_tokens(BAD, 0, 8, 8), ab.ab_tokens(GOOD, 0, 4, 8), ab.ab_tokens(GOOD, 0, 8, 4)):
            assert append(tok=tuple(wrong if j == k else t for j in range(3))) == 1
    assert append(pp=replace(PP, Hq=272, Hkv=17)) == 2

    def forward(T=5, ptr=(GOOD,) * 14, ws=BIG):
        return lib.ab_paged_forward(PP.c(), nr, T, t, t, t, *ptr, ws, None)

    for ptr in _each([GOOD] * 14):
        assert forward(ptr=ptr) == 1
    assert forward(T=0) == 1 and forward(ws=16) == 6


def test_append_refuses_tokens_inside_the_cache(lib):
    # the cache has 100 * 2 * 16 * 128 values of 2 bytes, a step of 5 tokens 5 * 8 * 128 of queries
    size = 100 * 2 * 16 * 128 * 2
    at = [0x100000000 + k * 0x1000000 for k in range(6)]          # slots, positions, Q, K, V, ksum
    apart = ab.ab_tokens(IN, 0, 8 * 128, 128)
    for out, n in ((2, 5 * 8 * 128 * 2), (3, size), (4, size)):
        for where in (at[out], at[out] + n - 16):
            for k in range(3):
                inside = ab.ab_tokens(where, 0, 8 * 128, 128)
                tok = [inside if j == k else apart for j in range(3)]
                assert lib.ab_paged_append(PP.c(), _nr(), 5, *tok, *at, None) == 1


def test_forward_qkv(lib):
    p = ab.Params(B=1, H=2, L=256, d=64, q_block=64, kv_block=16, C=4).c()
    t = ab.ab_tokens(IN, 0, 128, 64)
    nr = _nr(n_pos=256)
    ok = [*OUT] + [GOOD] * 6                                     # Q, K, V, P, idx, pi_q32, count, O, workspace
    for ptr in _each(ok):
        assert lib.ab_forward_qkv(p, nr, t, t, t, None, None, *ptr, BIG, None) == 1
    for k in range(3):
        tok = [None if j == k else t for j in range(3)]
        assert lib.ab_forward_qkv(p, nr, *tok, None, None, *ok, BIG, None) == 1
    assert lib.ab_forward_qkv(p, _nr(n_pos=255), t, t, t, None, None, *ok, BIG, None) == 1
    assert lib.ab_forward_qkv(p, nr, t, t, t, None, None, *ok, 16, None) == 6


def test_structs_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = (ab.ab_norm_rope, ab.ab_tokens, ab.ab_paged_params)
    src = tmp_path / "layout.c"
    lines = "".join(f'  printf("%zu\\n", offsetof({s.__name__}, {n}));\n' for s in structs for n, _ in s._fields_)
    lines += "".join(f'  printf("%zu\\n", sizeof({s.__name__}));\n' for s in structs)
    src.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "ab.h"\nint main(void) {{\n{lines}  return 0;\n}}\n')
    exe = tmp_path / "layout"
    subprocess.check_call([cc, "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)])
    got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    assert got == [getattr(s, n).offset for s in structs for n, _ in s._fields_] + [ctypes.sizeof(s) for s in structs]


def test_binding_checks():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):                              # no CPU path
        ab.ab_attention_paged(PP, x, x, x, i, i)
    with pytest.raises(ValueError):
        ab.ab_paged_plan(PP, i, i, i, i, i, T=4)
    with pytest.raises(ValueError):
        ab.ab_paged_topk(PP, x, i)
    with pytest.raises(ValueError):
        ab.ab_paged_append(PP, ab.NormRope("none"), x, x, x, i, i, x, x)
    with pytest.raises(ValueError):
        ab.ab_qk_norm_rope(ab.Params(B=1, H=8, L=4, d=128), ab.NormRope("none"), x[None])
    with pytest.raises(ValueError):
        ab.ab_qk_norm_rope(ab.Params(B=1, H=8, L=4, d=128), ab.NormRope("none"), None)
    for kw in (dict(norm="rms"), dict(cos=torch.zeros(3, 64)), dict(wq=torch.zeros(128)),
               dict(cos=torch.zeros(3, 64), sin=torch.zeros(3, 64))):
        with pytest.raises(ValueError):
            ab.NormRope(**kw)
