"""The binding's checks of tensors (csrc/marshal.cpp), on the CPU: what they refuse
and say.  Tensors that pass need a GPU: test_gpu_binding.py."""
import pytest

torch = pytest.importorskip("torch")

import block_sparse_attention_queries_b200 as ab  # noqa: E402
from block_sparse_attention_queries_b200 import build as abbuild  # noqa: E402

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def m():
    abbuild.build()
    return ab._m()


def test_none_and_nothing(m):
    assert m.tensors(0) == ()
    assert m.tensors(0, None, BF16, (1, 2), "Q", None, I32, (), "n") == (None, None)


def test_tensors_says_what_it_wants_and_gets(m):
    x = torch.zeros(3, 4, dtype=F32)
    with pytest.raises(ValueError, match=r"P: expected contiguous Int \(3, 5\) on cuda:2, got Float \[3, 4\], strides \[4, 1\], on cpu"):
        m.tensors(2, x, I32, (3, 5), "P")
    with pytest.raises(ValueError, match="lens.*got list"):
        m.tensors(0, None, F32, (1,), "P", [1, 2], I32, (2,), "lens")  # the second of two
    with pytest.raises(ValueError, match="on cpu"):                     # right in all else
        m.tensors(0, x, F32, (3, 4), "P")
    with pytest.raises(ValueError, match="expected strided .*got int"):
        m.tokens(0, 7, (1, 2, 8), "q")
    with pytest.raises(ValueError, match="q: .*on cpu"):
        m.tokens(0, torch.zeros(1, 2, 8, dtype=BF16), (1, 2, 8), "q")


@pytest.mark.parametrize("args", [(), (0, None), (0, None, BF16, (1,)), (0, None, BF16, (1,), "a", None), (0, None, "bf16", (1,), "a"),
                                  (0, None, BF16, [1], "a"), (0, None, BF16, (1,), 5), ("0", None, BF16, (1,), "a"),
                                  (0, torch.zeros(1, dtype=BF16), BF16, ("1",), "a"), (0, torch.zeros(1, dtype=BF16), BF16, (1.0,), "a")])
def test_tensors_argument_errors(m, args):
    with pytest.raises(TypeError):
        m.tensors(*args)


@pytest.mark.parametrize("args", [(), (0, None, (1, 2, 8)), (0, None, [1, 2, 8], "q"), (0, None, (1, 2, 8), 5),
                                  ("0", torch.zeros(1, 2, 8, dtype=BF16), (1, 2, 8), "q"),
                                  (0, torch.zeros(1, 2, 8, dtype=BF16), (1, 2, "8"), "q")])
def test_tokens_argument_errors(m, args):
    with pytest.raises(TypeError):
        m.tokens(*args)
