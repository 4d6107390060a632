"""Calls whose bounds say little about their rows: a max_seqlen_q far above the
rows that there are, wide block tables, prefix sums that go down in between.
Against the plain form in 64 bits; bounds: tests/kv_reference.py."""
import pytest
import torch

from exact_attention_forward_tiled_gb300 import api
from exact_attention_forward_tiled_gb300 import build as fa_build
from tests import kv_reference as ref
from tests.test_gpu_kv_edges import Case

pytestmark = pytest.mark.gpu
E4M3, I8, F16, BF16 = torch.float8_e4m3fn, torch.int8, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    fa_build.build()
    api.lib()


@pytest.mark.parametrize("kind,dtype,G", [(E4M3, BF16, 8), (BF16, BF16, 8), (I8, F16, 64)])
@pytest.mark.parametrize("P", [0, 200])
def test_loose_bound_and_wide_table(kind, dtype, G, P):
    """256 sequences of one or two rows, max_seqlen_q = 8192, a table for
    131072 keys: 256 * 8192 rows of all of these would be more units than 32
    bits count, the rows that there are make a few hundred thousand at most."""
    lens, nq = [(3 * i) % 25 for i in range(256)], [1 + i % 2 for i in range(256)]
    c = Case(21, lens, nq, G, 1, 64, 16, kind, dtype, True, P)
    cache, table, seqlens = c.args[0], c.args[-2], c.args[-1]
    wide = torch.full((256, 8192), 10 ** 7, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    c.args = c.args[:-2] + (wide, seqlens)
    c.kw["max_seqlen_q"] = 8192
    out, lse = c.call()
    api.fa_get_device_status()
    c.check(out, lse, only=set(range(0, 256, 5)) | {255})


@pytest.mark.parametrize("kind,dtype", [(E4M3, BF16), (BF16, BF16)])
@pytest.mark.parametrize("B,T,keys", [(4096, 2000, 40000), (1000, 20000, 500000)])
@pytest.mark.parametrize("P", [0, 33])
def test_sequences_that_overlap(kind, dtype, B, T, keys, P):
    """Prefix sums 0, T, 0, T, ...: every other sequence has all rows, many times
    the work that T rows can be. Nothing is done but reported, and the library
    goes on working. (Few-row kernel, many-row kernel.)"""
    Hq, Hk, D, page = 8, 1, 64, 16
    cache = api.kv_cache(3, page, Hk, D, dtype=kind)
    table = torch.zeros((B, keys // page), dtype=torch.int32, device="cuda")
    lens = torch.full((B,), keys, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, T] * (B // 2) + [0], dtype=torch.int32, device="cuda")
    q = torch.ones((T, Hq, D), dtype=dtype, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((Hq, T), 7.0, device="cuda")
    kw = dict(cu_seqlens_q=cu, max_seqlen_q=T, out=out, lse=lse)
    if P:
        pages = torch.zeros(-(-P // page), dtype=torch.int32, device="cuda")
        api.attention_forward_prefix(q, cache, pages, P, table, lens, **kw)
    else:
        api.attention_forward_kvcache(q, cache, table, lens, **kw)
    assert api.fa_get_device_status(check=False)[0] == -6
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all())
    Case(22, [200, 37], [3, 1], 3, 3, 128, 16, kind, dtype).run()


@pytest.mark.parametrize("kind,dtype,B", [(E4M3, BF16, 2900), (BF16, BF16, 3700), (I8, F16, 4096)])
def test_batches_that_leave_one_cta_per_sm(kind, dtype, B):
    """The sums of many sequences take the shared memory of a second CTA: the
    line is cut for the CTAs that fit, so it has half as many ranges (of two
    slots each in the workspace) and the results are right."""
    c = Case(23, [(7 * i) % 37 for i in range(B)], [1] * B, 4, 2, 128, 16, kind, dtype)
    out, lse = c.call()
    api.fa_get_device_status()
    c.check(out, lse, only=set(range(0, B, 13)) | {B - 1})
    size = [api.fa_fwd_kvcache_workspace_size(b, 4, 2, 1, 128) for b in (2000, 4096)]
    assert size[1] < 0.6 * size[0]
