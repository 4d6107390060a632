"""CPU tests of arguments that the binding, or the C entry, refuses: a prefix
without pages, packed rows with a bound of none, key positions whose tiles would
end past 2^31."""
import ctypes

import pytest
import torch

from exact_attention_forward_tiled_gb300 import api
from exact_attention_forward_tiled_gb300 import build as fa_build

INVALID = -1


@pytest.fixture(scope="module")
def L():
    fa_build.build()
    return api.lib()


def test_prefix_without_pages():
    """A length but no pages: refused, not run without the prefix."""
    with pytest.raises(ValueError, match="prefix_pages"):
        api.attention_forward_prefix(None, None, None, 5, None, None)
    with pytest.raises(ValueError, match="negative"):
        api.attention_forward_prefix(None, None, None, -1, None, None)


def _append(L, B, S, cu, total):
    return L.fa_kv_append(0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, 0x7000, 0x8000, B, 2, S, 128, 8, 16, 4, None, cu,
                          total, api.FA_BF16, api.FA_FP8_E4M3, None)


def _attn(L, B, S, cu, total, max_pages=4, P=0):
    return L.fa_fwd_prefix(0x1000, 0x3000, 0x4000, 0x5000, 0x6000, 0xc000, P, 0x7000, 0x8000, 0xa000, 0xb000, B, 4, 2, S, 128,
                           8, 16, max_pages, ctypes.c_float(0.1), 1, cu, total, 0x10000, 1 << 40, api.FA_FP16, api.FA_INT8,
                           None)


@pytest.mark.parametrize("f", [_append, _attn])
def test_rows_but_a_bound_of_none(L, f):
    """Packed rows whose sequences may have none: not taken for nothing to do."""
    assert f(L, 2, 0, 0x9000, 5) == INVALID
    assert f(L, 2, 0, 0x9000, 0) == 0 and f(L, 0, 0, 0x9000, 5) == 0 and f(L, 2, 0, None, 0) == 0


def test_rows_but_a_bound_of_none_from_python():
    cu = torch.tensor([0, 2, 5], dtype=torch.int32)
    for bound in (0, -1):
        with pytest.raises(ValueError, match="max_seqlen_q"):
            api._rows_per_seq(5, 2, cu, bound, "q", -1)
    assert api._rows_per_seq(5, 0, cu[:1], 0, "q", -1) == 0      # rows, but no sequences: nothing to do
    assert api._rows_per_seq(0, 2, cu, 0, "q", -1) == 0 and api._rows_per_seq(5, 2, cu, 3, "q", -1) == 3


def test_keys_up_to_the_last_of_32_bits(L):
    """The last tile's end is counted in 32 bits too: 256 positions are left."""
    top = 2 ** 31 - 1 - 256 - 1                       # less one query row
    for pages, P in ((2 ** 27 - 1, 0), (4, top - 64 + 1), (2 ** 26, 2 ** 30 - 17), (top // 16 + 1, 0)):
        assert _attn(L, 1, 1, None, 0, pages, P) == INVALID, (pages, P)
    if not torch.cuda.is_available():
        for pages, P in ((top // 16, 0), (4, top - 64)):
            assert _attn(L, 1, 1, None, 0, pages, P) == -7, (pages, P)
