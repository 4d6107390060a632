"""Scales past the end of a sequence, or of the shared prefix, may hold
anything: finite ones of any size and sign, not only NaN. Odd lengths, several
key blocks, and a score that comes late and far above the ones before, which has
to move the running max however those scales look. Against the plain form in 64
bits; bounds: tests/kv_reference.py."""
import math

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


SMALL = 2.0 ** -9
STALE = [(-1.0, SMALL), (-0.0, SMALL), (-math.inf, SMALL), (3e38, 3e38), (-3e38, -3e38), (math.inf, -0.0), (math.nan, math.nan)]


@pytest.mark.parametrize("stale", STALE)
@pytest.mark.parametrize("kind,dtype,D", [(E4M3, BF16, 64), (I8, F16, 128), (I8, BF16, 256)])
@pytest.mark.parametrize("P", [0, 385])
@pytest.mark.parametrize("nq", [3, 70])
def test_scales_past_the_end(stale, kind, dtype, D, P, nq):
    """nq rows per sequence: the few-row and the many-row kernel; the last
    key of the prefix, or of the sequence, scores about 60 for every query.
    stale: K's and V's scales past the end."""
    rng = torch.Generator().manual_seed(int(P + nq))
    lens, Hq, Hk, page = [257, 129], 77, 77, 16      # more heads than half the SMs: a worker has all blocks of an item
    cache, table, seqlens, _, _ = ref.fill_cache(rng, lens + [P], page, Hk, D, kind, dtype)
    k, v, ks, vs = cache
    q = (torch.randn((2 * nq, Hq, D), generator=rng) * 0.25).to(dtype)
    q[..., 0] = 8.0
    for b, n in enumerate(lens + [P]):
        for i in range(n, -(-n // page) * page):       # the rest of the last page
            at = int(table[b, i // page]), slice(None), i % page
            ks[at], vs[at] = stale
        if n and (P == 0 or b == 2):                   # the late key: all of it in the first element
            at = int(table[b, (n - 1) // page]), (n - 1) % page
            row = torch.zeros(Hk, D)
            row[:, 0] = 7.5 * D ** 0.5
            codes, scale = ref.quantise(row.to(dtype), kind)
            k.view(torch.uint8)[at] = codes.view(torch.uint8).cuda()
            ks[at[0], :, at[1]] = scale.cuda()
    keys = [[ref.values(cache, i)[[int(table[b, j // page]) * page + j % page for j in range(n)]]
             for b, n in enumerate(lens + [P])] for i in range(2)]
    args = (q.cuda(), api.KVCache(*cache)) + ((table[2, :-(-P // page)].contiguous(), P) if P else ())
    f = api.attention_forward_prefix if P else api.attention_forward_kvcache
    out, lse = f(*args, table[:2].contiguous(), seqlens[:2].contiguous(), causal=False)
    api.fa_get_device_status()
    for b in range(2):
        kk, vv = (torch.cat([keys[i][2], keys[i][b]]) for i in range(2))
        o, l, bo, bl = ref.attention(q[b * nq:(b + 1) * nq].double(), kk, vv, D ** -0.5, False, dtype, F16, True)
        ref.check(out[b * nq:(b + 1) * nq], o, bo, f"O of sequence {b}")
        ref.check(lse[b], l, bl, f"LSE of sequence {b}")


@pytest.mark.parametrize("nq", [3, 70])
def test_scale_of_minus_zero(nq):
    """A visible key whose scale is -0.0 (its value is a zero, its score 0)."""
    rng = torch.Generator().manual_seed(nq)
    n, H, D, page = 300, 77, 64, 16
    cache, table, seqlens, _, _ = ref.fill_cache(rng, [n], page, H, D, E4M3, BF16)
    q = torch.randn((nq, H, D), generator=rng).bfloat16()
    q[..., 0] = 8.0
    row = torch.zeros(H, D)
    row[:, 0] = 7.5 * D ** 0.5
    codes, scale = ref.quantise(row.bfloat16(), E4M3)
    at = int(table[0, 299 // page]), 299 % page
    cache[0].view(torch.uint8)[at] = codes.view(torch.uint8).cuda()
    cache[2][at[0], :, at[1]] = scale.cuda()
    cache[2][int(table[0, 290 // page]), :, 290 % page] = -0.0
    rows = [int(table[0, j // page]) * page + j % page for j in range(n)]
    out, lse = api.attention_forward_kvcache(q.cuda(), api.KVCache(*cache), table, seqlens)
    api.fa_get_device_status()
    o, l, bo, bl = ref.attention(q.double(), ref.values(cache, 0)[rows], ref.values(cache, 1)[rows], D ** -0.5, False, BF16,
                                 F16, True)
    ref.check(out, o, bo, "O")
    ref.check(lse[0], l, bl, "LSE")
