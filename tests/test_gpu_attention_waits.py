"""The attention kernels' bounded waits, and what a call may touch.

A stage whose barrier is armed for 16 bytes more than its copies deliver makes the waiting warp
give up after a short limit. The copies have landed, the kernel returns with
RSSM_DEVERR_TIMEOUT, what it could not finish keeps its outputs, and the next call (with a
cleared workspace) runs normally. No wait is unbounded. Besides: tables written right before a
call, and a workspace of just the size asked for."""
import time

import pytest
import torch

from tests import test_gpu_attention as A

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    import ssm_linear_attention_gb300 as ssm
    ssm.lib()


# Lists of one key head: with few queries 16 tokens a tile, with many 128 a chunk and one unit more
# before a row's chunks. Row 1 begins in the list at tile 63 (unit 9), row 0's tile 20 is its
# 320th token on, its unit 3 its third chunk. A long row is shared by many CTAs.
@pytest.mark.parametrize("hq,cache,act,lens,stall", [
    (4, torch.bfloat16, torch.bfloat16, [1000, 40], 20),
    (4, torch.bfloat16, torch.float32, [1000, 40], 20),
    (4, torch.bfloat16, torch.bfloat16, [60000, 40], 1777),
    (16, torch.bfloat16, torch.bfloat16, [1000, 40], 3),
    (32, FP8, torch.bfloat16, [1000, 40], 3),
    (64, torch.bfloat16, torch.bfloat16, [60000, 40], 222),
])
def test_a_wait_that_runs_out_leaves_the_output_unwritten(hq, cache, act, lens, stall):
    import ssm_linear_attention_gb300 as ssm
    dec, ci, table, slots, g = A.make(2, lens, hq=hq, hkv=1, page=64, cache=cache, act=act, seed=3)
    A.fill(dec, ci, table, slots, lens, g)
    q = torch.randn(2, 1, hq, 128, generator=g, device="cuda").to(act)
    o = torch.full((2, 1, hq, 128), 7.0, device="cuda", dtype=act)
    lse = torch.full((2, 1, hq), 7.0, device="cuda")

    def call(tile):
        ssm.rssm_debug_attn_decode(dec.dims(2), dec.cache, False, dec.scale, 0, q, hq * 128, ci,
                                   dec.workspace, dec.ws_bytes, o, lse, tile, 2000, dec.dev_err)
        torch.cuda.synchronize()
    t0 = time.perf_counter()
    call(stall)
    took = time.perf_counter() - t0
    assert int(dec.dev_err[0]) == ssm.RSSM_DEVERR_TIMEOUT
    assert took < 1.0, took   # the limit and the wind-down's, not the 2 s of a call
    assert bool((o[0] == 7).all()) and bool((lse[0] == 7).all())
    ref = A.reference(dec, q, table, slots, lens, False)
    A.check(dec, o[1:], lse[1:], [t[1:] for t in ref])     # the other row is another CTA's
    dec.workspace.zero_()
    dec.dev_err.zero_()
    call(-1)
    assert int(dec.dev_err[0]) == 0
    A.check(dec, o, lse, ref)
    o2, lse2 = dec.decode(q, ci, appended=False, with_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(o2, o) and torch.equal(lse2, lse)


@pytest.mark.parametrize("hq,cache", [(4, torch.bfloat16), (4, FP8), (16, torch.bfloat16), (32, FP8)])
def test_a_page_table_written_just_before_the_call(hq, cache):
    """The kernels start while the one before them ends: a table, a length and a page that this one
    writes are read as it leaves them."""
    dec, ci, table, slots, g = A.make(3, [500, 70, 900], hq=hq, hkv=1, page=64, cache=cache, seed=5)
    A.fill(dec, ci, table, slots, [500, 70, 900], g)
    q = torch.randn(3, 1, hq, 128, generator=g, device="cuda").bfloat16()
    tables = [dec.page_table.clone(), dec.page_table.clone()]
    s = torch.from_numpy(slots).cuda()
    tables[1][s[0], :7] = tables[0][s[2], :7]                  # (full pages)
    tables[1][s[2], :7] = tables[0][s[0], :7]
    lens = [dec.slot_len.clone(), dec.slot_len.clone() - dec.slot_len // 3]
    want = []
    for t, n in zip(tables, lens):
        dec.page_table.copy_(t)
        dec.slot_len.copy_(n)
        torch.cuda.synchronize()
        want.append(dec.decode(q, ci, appended=False).clone())
        torch.cuda.synchronize()
    assert not torch.equal(*want)
    got = []
    for i in range(100):
        dec.page_table.copy_(tables[i % 2])
        dec.slot_len.copy_(lens[i % 2])
        got.append(dec.decode(q, ci, appended=False).clone())
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i % 2]) for i, o in enumerate(got))


@pytest.mark.parametrize("hq,cache,act,d,T", [
    (4, torch.bfloat16, torch.bfloat16, 128, 1), (4, torch.bfloat16, torch.bfloat16, 64, 2),
    (4, FP8, torch.bfloat16, 128, 1), (8, FP8, torch.bfloat16, 64, 2), (16, FP8, torch.bfloat16, 128, 1),
    (4, torch.bfloat16, torch.float32, 128, 1), (3, FP8, torch.float32, 64, 5),
    (8, torch.bfloat16, torch.float32, 128, 8), (16, torch.bfloat16, torch.bfloat16, 128, 1),
    (8, FP8, torch.bfloat16, 128, 4), (16, torch.bfloat16, torch.bfloat16, 64, 4),
])
def test_a_call_stays_within_its_workspace(hq, cache, act, d, T):
    """Rows that many CTAs and groups share, in a workspace of just the size asked for: what
    lies behind it stays."""
    import ssm_linear_attention_gb300 as ssm
    lens = [21000, 40, 7777, 1, 900]
    dec, ci, table, slots, g = A.make(5, lens, hq=hq, hkv=1, d=d, T=T, page=64, cache=cache, act=act, seed=7)
    A.fill(dec, ci, table, slots, lens, g)
    q = torch.randn(5, T, hq, d, generator=g, device="cuda").to(act)
    ws = torch.zeros(dec.ws_bytes + (8 << 20), device="cuda", dtype=torch.uint8)
    ws[dec.ws_bytes:] = 0xa5
    o = torch.empty(5, T, hq, d, device="cuda", dtype=act)
    lse = torch.empty(5, T, hq, device="cuda")
    for _ in range(2):
        ssm.rssm_attn_decode(dec.dims(5), dec.cache, False, dec.scale, 0, q, hq * d, ci, ws, dec.ws_bytes,
                             o, lse, dec.dev_err)
    torch.cuda.synchronize()
    assert bool((ws[dec.ws_bytes:] == 0xa5).all()) and int(dec.dev_err.sum()) == 0
    assert bool((ws[:1024] == 0).all())                  # the counters are back at zero
    A.check(dec, o, lse, A.reference(dec, q, table, slots, lens, False))
