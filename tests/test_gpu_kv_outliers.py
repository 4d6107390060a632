"""Queries with one channel far above the rest, over 8-bit caches whose keys are
small there: the other channels decide the scores and must not be lost beside
it. Against the plain form in 64 bits.

Bounds: those of tests/kv_reference.py for a query held exactly, and what the
header states on top, as an error of a score: a bf16 query element may be off by
2^-38 of its row's largest (f16 has 2^-25 as its half smallest step, the largest
is brought into [2^14, 2^15)), or, as the power of two that does it is 2^114 at
most, by 2^-139; fp16 queries are exact. A score that is off by x moves LSE by at
most x, and O by at most 2 x max |v| (to first order; 2.1 covers x up to 0.02).
"""
import pytest
import torch

from exact_attention_forward_tiled_gb300 import api
from exact_attention_forward_tiled_gb300 import build as fa_build
from tests import kv_reference as ref

pytestmark = pytest.mark.gpu
E4M3, I8, F16, BF16 = torch.float8_e4m3fn, torch.int8, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    fa_build.build()
    api.lib()


def _lost(q, k, scale, dtype):
    """Bound [n, Hq] of what the query's representation moves a score by."""
    kk = k.abs().repeat_interleave(q.shape[1] // k.shape[1], 1)
    top = q.abs().amax(-1)
    return (2.0 ** -38 * top).clamp(min=2.0 ** -139) * kk.sum(-1).amax(0) * scale if dtype == BF16 else torch.zeros_like(top)


def _run(seed, lens, nq, G, Hk, D, kind, dtype, power, P=0, rows=None):
    """power: the channel's size above the rest, 2^power; rows: the query rows
    that have it (default: all)."""
    rng = torch.Generator().manual_seed(seed)
    cache, table, seqlens, _, _ = ref.fill_cache(rng, lens + [P], 16, Hk, D, kind, dtype)
    B, Hq = len(lens), G * Hk
    hot = D // 2 + 5
    cache[0].view(torch.uint8)[..., hot] = 1             # the smallest code there is: 2^-9, or 1
    where = [[int(table[b, j // 16]) * 16 + j % 16 for j in range(n)] for b, n in enumerate(lens + [P])]
    k, v = ([ref.values(cache, i)[w] for w in where] for i in range(2))
    q = torch.randn((B * nq, Hq, D), generator=rng)
    pick = torch.ones(B * nq, dtype=torch.bool) if rows is None else torch.zeros(B * nq, dtype=torch.bool)
    if rows is not None:
        pick[rows] = True
    q[pick, :, hot] = 2.0 ** power * (1 + torch.rand((int(pick.sum()), Hq), generator=rng))
    q = q.to(dtype)
    args = (q.cuda(), api.KVCache(*cache)) + ((table[B, :-(-P // 16)].contiguous(), P) if P else ())
    f = api.attention_forward_prefix if P else api.attention_forward_kvcache
    out, lse = f(*args, table[:B].contiguous(), seqlens[:B].contiguous(), causal=False)
    api.fa_get_device_status()
    for b in range(B):
        x = q[b * nq:(b + 1) * nq].double()
        kk, vv = torch.cat([k[B], k[b]]), torch.cat([v[B], v[b]])
        o, l, bo, bl = ref.attention(x, kk, vv, D ** -0.5, False, dtype, F16, False)
        lost = _lost(x, kk, D ** -0.5, dtype)
        ref.check(out[b * nq:(b + 1) * nq], o, bo + (2.1 * lost * vv.abs().amax())[..., None], f"O of sequence {b}")
        ref.check(lse[b], l, bl + lost.t(), f"LSE of sequence {b}")


@pytest.mark.parametrize("power", [0, 2, 4, 6, 8, 10, 12])
@pytest.mark.parametrize("kind,dtype", [(E4M3, BF16), (E4M3, F16), (I8, BF16), (I8, F16)])
@pytest.mark.parametrize("D,G,nq", [(64, 4, 1), (128, 4, 1), (128, 16, 1), (256, 8, 1), (256, 3, 5), (128, 4, 20)])
def test_one_channel_above_the_rest(power, kind, dtype, D, G, nq):
    """Few rows (tiles of 8 and 16) and many; sequences of one key, whose LSE is
    the score, and of several."""
    _run(power, [1, 2, 33, 300], nq, G, 2, D, kind, dtype, power)


@pytest.mark.parametrize("kind,dtype", [(E4M3, BF16), (E4M3, F16), (I8, BF16)])
@pytest.mark.parametrize("P", [50, 700])
def test_behind_a_prefix(kind, dtype, P):
    _run(P, [1, 0, 20], 1, 4, 2, 128, kind, dtype, 11, P=P)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("G,nq", [(4, 2), (2, 7)])
def test_one_row_among_ordinary_ones(dtype, G, nq):
    """Rows of one tile of which only some have the channel."""
    _run(3, [1, 60, 200], nq, G, 2, 128, E4M3, dtype, 12, rows=[0, nq + 1])


@pytest.mark.parametrize("size", [-120, -100, 100, 126])
def test_rows_far_from_one(size):
    """bf16 queries whose largest element is about 2^size."""
    rng = torch.Generator().manual_seed(4)
    cache, table, seqlens, ks, vs = ref.fill_cache(rng, [1, 200], 16, 2, 128, E4M3, BF16)
    q = torch.randn((2, 8, 128), generator=rng).double() * 2.0 ** size
    q = (q / q.abs().amax() * 2.0 ** size).bfloat16()
    scale = 2.0 ** -size if size > -110 else 2.0 ** 110
    out, lse = api.attention_forward_kvcache(q.cuda(), api.KVCache(*cache), table, seqlens, scale=scale)
    api.fa_get_device_status()
    for b in range(2):
        x = q[b:b + 1].double()
        o, l, bo, bl = ref.attention(x, ks[b], vs[b], scale, False, BF16, F16, False)
        lost = _lost(x, ks[b], scale, BF16)
        ref.check(out[b:b + 1], o, bo + (2.1 * lost * vs[b].abs().amax())[..., None], "O")
        ref.check(lse[b], l, bl + lost.t(), "LSE")
