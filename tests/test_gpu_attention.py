"""The attention layer's entry points against float64: the paged cache (append, read back,
advance) and the decode attention over it.

Tolerances, from the rounding each path makes:
  * a bf16 value carries half a spacing, at most 2^-8 relative (8 significant bits); a float32 output of float32
    activations 2^-17 of the largest weighted value (the sums run in float32 over exact
    or split operands);
  * with bf16 activations the softmax weights enter the value product in at least 16
    bits, so only the output's own rounding shows: |o - ref| <= 2^-8 (|ref| + 2^-8 w),
    w = sum_p p |v_p| the size of the terms;
  * 8-bit caches are compared through the values they stand for: the append must give the
    nearest e4m3 value of x / scale, ties aside (1 + 2^-20 of half a spacing)."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    import ssm_linear_attention_gb300 as ssm
    ssm.lib()


def make(batch, lens, hq=8, hkv=2, d=128, page=16, cache=torch.bfloat16, act=torch.bfloat16,
         out=None, T=1, window=0, seed=0, max_pages=None, num_slots=None, poison=True, spare=5):
    """A decoder with slots in a random order, pages scattered, `lens` committed tokens per
    row and room for T more, and (poison) NaN wherever no token lives."""
    import ssm_linear_attention_gb300 as ssm
    r = np.random.default_rng(seed)
    num_slots = batch + 3 if num_slots is None else num_slots
    need = [max(1, -(-(n + T) // page)) for n in lens]
    max_pages = max(need) + 1 if max_pages is None else max_pages
    num_pages = sum(need) + spare
    dec = ssm.PagedAttentionDecoder(hq, hkv, d, page, num_pages, num_slots, max_pages, batch, T=T,
                                    act_dtype=act, cache_dtype=cache, out_dtype=out or act,
                                    window=window)
    slots = r.permutation(num_slots)[:batch]
    order = r.permutation(num_pages)
    table = np.full((num_slots, max_pages), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[slots[b], :n] = order[at:at + n]
        at += n
    dec.page_table.copy_(torch.from_numpy(table))
    sl = np.zeros(num_slots, np.int32)
    sl[slots] = lens
    dec.slot_len.copy_(torch.from_numpy(sl))
    if poison:
        for t in (dec.k_cache, dec.v_cache):
            if cache == FP8:
                t.view(torch.uint8).fill_(0x7f)
            else:
                t.fill_(float("nan"))
        if cache == FP8:
            dec.k_scale.fill_(float("nan"))
            dec.v_scale.fill_(float("inf"))
    ci = torch.from_numpy(slots.astype(np.int32)).cuda()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    return dec, ci, table, slots, g


def fill(dec, ci, table, slots, lens, g, mul=1.0):
    """Committed tokens through append: sets slot_len to 0, appends, restores."""
    n = sum(lens)
    if n == 0:
        return
    k = (mul * torch.randn(n, dec.HKV, dec.D, generator=g, device="cuda")).to(dec.act_dtype)
    v = torch.randn(n, dec.HKV, dec.D, generator=g, device="cuda").to(dec.act_dtype)
    keep = dec.slot_len.clone()
    dec.slot_len.zero_()
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32, device="cuda")
    cu[1:] = torch.tensor(lens, device="cuda").cumsum(0)
    dec.append(k, v, ci, cu_tokens=cu)
    dec.advance(ci, cu_tokens=cu)
    torch.cuda.synchronize()
    assert torch.equal(dec.slot_len, keep)


def cached(dec, table, slot, lo, hi):
    """float64 keys and values of positions lo..hi-1, [n, HKV, D]."""
    pos = np.arange(lo, hi)
    p = torch.from_numpy(table[slot][pos // dec.page_size].astype(np.int64)).cuda()
    o = torch.from_numpy(pos % dec.page_size).cuda()
    out = []
    for c, s in ((dec.k_cache, dec.k_scale), (dec.v_cache, dec.v_scale)):
        x = c.view(torch.uint8)[p, :, o].view(FP8).double() if c.dtype == FP8 else c[p, :, o].double()
        out.append(x if s is None else x * s[p, :, o].double()[..., None])
    return out


def reference(dec, q, table, slots, lens, appended, hidden=()):
    """(o, lse, w) in float64; hidden: positions whose tokens are left out."""
    B, T, HQ, D = q.shape
    o = torch.zeros(B, T, HQ, D, dtype=torch.float64, device="cuda")
    w = torch.zeros_like(o)
    lse = torch.full((B, T, HQ), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        for j in range(T):
            hi = lens[b] + (j + 1 if appended else 0)
            lo = max(0, hi - dec.window) if dec.window else 0
            keep = [p for p in range(lo, hi) if p not in hidden]
            if not keep:
                continue
            k, v = cached(dec, table, slots[b], lo, hi)
            if hidden:
                sel = torch.tensor(keep, device="cuda") - lo
                k, v = k[sel], v[sel]
            qq = q[b, j].double().view(dec.HKV, -1, D)
            s = torch.einsum("hgd,nhd->hgn", qq, k) * dec.scale
            m = s.amax(-1, keepdim=True)
            p = (s - torch.where(m == -math.inf, 0.0, m)).exp()
            l = p.sum(-1, keepdim=True)
            z = l[..., 0] == 0
            pv = torch.einsum("hgn,nhd->hgd", p, v) / l
            o[b, j] = torch.where(z[..., None], 0.0, pv).reshape(HQ, D)
            w[b, j] = (torch.einsum("hgn,nhd->hgd", p, v.abs()) / l).reshape(HQ, D)
            lse[b, j] = (m + l.log())[..., 0].reshape(HQ)
    return o, lse, w


def check(dec, got, glse, ref, appended=True):
    o, lse, w = ref
    got = got.double()
    fine = torch.isfinite(o)
    assert torch.equal(torch.isnan(got), torch.isnan(o))
    if dec.out_dtype == torch.bfloat16:
        bound = 2.0 ** -8 * (o.abs() + 2.0 ** -8 * w) + 1e-30
    else:
        bound = (2.0 ** -17 if dec.act_dtype == torch.float32 else 2.0 ** -13) * (o.abs() + w) + 1e-30
    worst = ((got - o).abs() / bound)[fine]
    assert worst.numel() == 0 or float(worst.max()) <= 1.0, float(worst.max())
    dead = lse == -math.inf
    assert torch.equal(glse.double() == -math.inf, dead)
    assert float((glse.double() - lse)[~dead & torch.isfinite(lse)].abs().max()
                 if (~dead & torch.isfinite(lse)).any() else 0.0) <= 2e-5


CASES = [
    # batch, lens, kw
    (1, [0], {}),
    (1, [1], dict(d=64)),
    (2, [15, 16], dict(cache=FP8)),
    (3, [17, 300, 31], dict(hq=4, hkv=4, page=32)),
    (4, [5, 1000, 64, 63], dict(hq=16, hkv=1, d=64, page=64, cache=FP8)),
    (2, [777, 40], dict(hq=14, hkv=2, page=16)),
    (3, [100, 8, 513], dict(hq=32, hkv=2, page=128, T=4, cache=FP8)),
    (2, [33, 257], dict(hq=6, hkv=2, d=64, page=16, T=5)),
    (2, [700, 90], dict(window=100, page=256)),
    (2, [700, 9], dict(window=17, T=3, cache=FP8, page=16)),
    (2, [250, 129], dict(act=torch.float32, d=64)),
    (2, [250, 31], dict(act=torch.float32, cache=FP8, T=2, hq=32, hkv=2)),
    (2, [64, 1], dict(act=torch.float32, window=1, T=8, hq=16, hkv=2, page=32)),
    (1, [9000], dict(hq=8, hkv=1, page=16)),
    (1, [9001], dict(hq=8, hkv=2, page=64, cache=FP8, T=8, d=64)),
    (40, [(37 * i) % 251 for i in range(40)], dict(hkv=8, hq=8)),
    (300, [(91 * i) % 40 for i in range(300)], dict(hkv=4, hq=32, cache=FP8, page=32)),
    (5, [3000, 1, 40, 2999, 16], dict(hq=64, hkv=4, T=4, page=16)),
    (2, [600, 47], dict(out=torch.float32)),
    (1100, [(53 * i) % 35 for i in range(1100)], dict(hkv=2, hq=2, d=64, cache=FP8)),
]


@pytest.mark.parametrize("batch,lens,kw", CASES)
@pytest.mark.parametrize("appended", [True, False])
def test_decode_matches_float64(batch, lens, kw, appended):
    dec, ci, table, slots, g = make(batch, lens, seed=batch + len(lens) + lens[0], **kw)
    fill(dec, ci, table, slots, lens, g)
    q = (2 * torch.randn(batch, dec.T, dec.HQ, dec.D, generator=g, device="cuda")).to(dec.act_dtype)
    if appended:
        k = torch.randn(batch, dec.T, dec.HKV, dec.D, generator=g, device="cuda").to(dec.act_dtype)
        v = torch.randn(batch, dec.T, dec.HKV, dec.D, generator=g, device="cuda").to(dec.act_dtype)
        dec.append(k, v, ci)
    o, lse = dec.decode(q, ci, appended=appended, with_lse=True)
    o2, lse2 = o.clone(), lse.clone()
    o3, lse3 = dec.decode(q, ci, appended=appended, with_lse=True)
    torch.cuda.synchronize()
    assert int(dec.dev_err.sum()) == 0
    assert torch.equal(o2, o3) and torch.equal(lse2, lse3)     # same bits every time
    check(dec, o, lse, reference(dec, q, table, slots, lens, appended))


@pytest.mark.parametrize("cache", [torch.bfloat16, FP8])
@pytest.mark.parametrize("d", [64, 128])
def test_padding_rows_bad_slots_bad_lengths_and_bad_pages(cache, d):
    import ssm_linear_attention_gb300 as ssm
    lens = [40, 41, 42, 43, 44, 300]
    dec, ci, table, slots, g = make(6, lens, d=d, cache=cache, seed=3)
    fill(dec, ci, table, slots, lens, g)
    q = torch.randn(6, 1, 8, d, generator=g, device="cuda").to(torch.bfloat16)
    bad = ci.clone()
    bad[1] = -1
    bad[2] = dec.num_slots
    o = torch.full((6, 1, 8, d), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((6, 1, 8), 7.0, device="cuda")
    dec.slot_len[slots[3]] = dec.max_pages * dec.page_size       # no room for the appended token
    dec.slot_len[slots[4]] = -1
    dec.page_table[slots[5], 2] = dec.num_pages                  # positions 32..47 are hidden
    dec.page_table[slots[5], 4] = -7                             # and 64..79
    dec.decode(q, bad, appended=True, o=o, lse=lse)
    torch.cuda.synchronize()
    assert int(dec.dev_err[0]) == ssm.RSSM_DEVERR_SLOT | ssm.RSSM_DEVERR_CURSOR | ssm.RSSM_DEVERR_PAGE
    assert bool((o[1:5] == 7).all()) and bool((lse[1:5] == 7).all())
    # row 0 sees its appended position, which the poison fills: everything is NaN there
    assert bool(torch.isnan(o[0]).all())
    dec.dev_err.zero_()
    dec.decode(q, bad, appended=False, o=o, lse=lse)
    torch.cuda.synchronize()
    hidden = set(range(32, 48)) | set(range(64, 80))
    for b, hid in ((0, ()), (5, hidden)):
        ref = reference(dec, q[b:b + 1], table, slots[b:b + 1], lens[b:b + 1], False, hid)
        check(dec, o[b:b + 1], lse[b:b + 1], ref)
    # a row whose every page is bad sees nothing
    dec.page_table[slots[5]] = -1
    dec.decode(q, bad, appended=False, o=o, lse=lse)
    torch.cuda.synchronize()
    assert bool((o[5] == 0).all()) and bool((lse[5] == -math.inf).all())


@pytest.mark.parametrize("cache", [torch.bfloat16, FP8])
def test_drafts_do_not_see_what_comes_after_them_nan_included(cache):
    lens = [30, 5]
    dec, ci, table, slots, g = make(2, lens, T=4, cache=cache, seed=8)
    fill(dec, ci, table, slots, lens, g)
    shape = (2, 4, 2, 128)
    k = torch.randn(shape, generator=g, device="cuda").bfloat16()
    v = torch.randn(shape, generator=g, device="cuda").bfloat16()
    k[:, 3, 0, 5] = float("nan")
    v[:, 2, :, 9] = float("inf")
    v[:, 3, 1] = float("nan")
    dec.append(k, v, ci)
    q = torch.randn(2, 4, 8, 128, generator=g, device="cuda").bfloat16()
    o, lse = dec.decode(q, ci, with_lse=True)
    torch.cuda.synchronize()
    ref = reference(dec, q, table, slots, lens, True)
    check(dec, o[:, :2], lse[:, :2], [t[:, :2] for t in ref])
    assert bool(torch.isnan(o[:, 3]).all())
    if cache == torch.bfloat16:
        assert bool(torch.isinf(o[:, 2, :, 9]).all())
        rest = [c for c in range(128) if c != 9]
        check(dec, o[:, 2:3, :, rest], lse[:, 2:3], [ref[0][:, 2:3, :, rest], ref[1][:, 2:3],
                                                     ref[2][:, 2:3, :, rest]])


def test_window_does_not_see_what_lies_before_it_nan_included():
    lens = [100]
    dec, ci, table, slots, g = make(1, lens, T=3, window=40, seed=4)
    fill(dec, ci, table, slots, lens, g)
    # position 61 is the last that draft 0 sees alone (its window starts there)
    page, off = int(table[slots[0]][61 // 16]), 61 % 16
    dec.v_cache[page, :, off, 3] = float("nan")
    dec.k_cache[int(table[slots[0]][2]), :, :] = float("nan")     # positions 32..47: no draft
    k = torch.randn(1, 3, 2, 128, generator=g, device="cuda").bfloat16()
    dec.append(k, k, ci)
    q = torch.randn(1, 3, 8, 128, generator=g, device="cuda").bfloat16()
    o, lse = dec.decode(q, ci, with_lse=True)
    torch.cuda.synchronize()
    assert bool(torch.isnan(o[:, 0, :, 3]).all())
    assert int(torch.isnan(o).sum()) == 8
    ref = reference(dec, q, table, slots, lens, True)
    check(dec, o[:, 1:], lse[:, 1:], [t[:, 1:] for t in ref])


def test_infinite_scores():
    lens = [40]
    dec, ci, table, slots, g = make(1, lens, hq=2, hkv=2, seed=5)
    fill(dec, ci, table, slots, lens, g)
    q = torch.zeros(1, 1, 2, 128, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = 1.0
    dec.k_cache[:, :, :, 0] = -math.inf                       # every score -infinity: no weight
    o, lse = dec.decode(q, ci, appended=False, with_lse=True)
    torch.cuda.synchronize()
    # 0 * inf never arises: q's other entries meet finite keys
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    dec.k_cache[int(table[slots[0]][1]), :, 3, 0] = 1.0       # position 19 alone has a weight
    o, lse = dec.decode(q, ci, appended=False, with_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(o[0, 0], dec.v_cache[int(table[slots[0]][1]), :, 3])
    dec.k_cache[int(table[slots[0]][0]), 0, 3, 0] = math.inf  # +infinity: NaN, as the formula says
    o, lse = dec.decode(q, ci, appended=False, with_lse=True)
    torch.cuda.synchronize()
    assert bool(torch.isnan(o[0, 0, 0]).all()) and bool(torch.isfinite(o[0, 0, 1].float()).all())


@pytest.mark.parametrize("cache", [torch.bfloat16, FP8])
def test_large_scores_and_values_of_every_size(cache):
    lens = [500, 20]
    dec, ci, table, slots, g = make(2, lens, cache=cache, seed=6)
    n = sum(lens)
    k = (30 * torch.randn(n, 2, 128, generator=g, device="cuda")).bfloat16()
    # token magnitudes over 24 binades
    v = (torch.randn(n, 2, 128, generator=g, device="cuda")
         * 2.0 ** torch.randint(-12, 12, (n, 1, 1), generator=g, device="cuda")).bfloat16()
    keep = dec.slot_len.clone()
    dec.slot_len.zero_()
    cu = torch.tensor([0, 500, 520], dtype=torch.int32, device="cuda")
    dec.append(k, v, ci, cu_tokens=cu)
    dec.slot_len.copy_(keep)
    q = torch.randn(2, 1, 8, 128, generator=g, device="cuda").bfloat16()
    o, lse = dec.decode(q, ci, appended=False, with_lse=True)
    torch.cuda.synchronize()
    ref = reference(dec, q, table, slots, lens, False)
    o64, lse64, w = ref
    # scores reach the hundreds: float32 leaves 2^-24 of them, which the weights see absolutely
    bound = 2.0 ** -8 * o64.abs() + (2.0 ** -15 + 2.0 ** -16) * 8 * w + 1e-30
    assert float(((o.double() - o64).abs() / bound).max()) <= 1.0
    assert float((lse.double() - lse64).abs().max()) <= 2.0 ** -22 * float(lse64.abs().max()) + 2e-5


def test_strided_queries_keys_and_values_and_another_stream():
    lens = [50, 3, 200]
    dec, ci, table, slots, g = make(3, lens, hq=8, hkv=2, d=64, seed=7)
    fill(dec, ci, table, slots, lens, g)
    qkv = torch.randn(3, 12, 64, generator=g, device="cuda").bfloat16()
    q, k, v = qkv[:, :8].unsqueeze(1), qkv[:, 8:10], qkv[:, 10:]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o = dec.step(q, k, v, ci)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    now = [n + 1 for n in lens]
    assert [int(dec.slot_len[s]) for s in slots] == now
    ref = reference(dec, q, table, slots, now, False)
    _, glse = dec.decode(q, ci, appended=False, with_lse=True)
    torch.cuda.synchronize()
    check(dec, o, glse, ref)
    kk, vv = cached(dec, table, slots[1], 3, 4)
    assert torch.equal(kk[0], k[1].double()) and torch.equal(vv[0], v[1].double())


def test_steps_in_a_graph_follow_the_lengths():
    lens = [14, 40]
    dec, ci, table, slots, g = make(2, lens, seed=9, max_pages=8, spare=16)
    for b, s in enumerate(slots):                       # pages for everything to come
        dec.page_table[s] = torch.arange(8 * b, 8 * b + 8)
    table = dec.page_table.cpu().numpy()
    fill(dec, ci, table, slots, lens, g)
    x = torch.zeros(2, 12, 128, device="cuda", dtype=torch.bfloat16)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dec.decode(x[:, :8].unsqueeze(1), ci, appended=False)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = dec.step(x[:, :8].unsqueeze(1), x[:, 8:10], x[:, 10:], ci)
    for t in range(5):
        x.copy_(torch.randn(2, 12, 128, generator=g, device="cuda").bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        now = [n + t + 1 for n in lens]
        assert [int(dec.slot_len[s]) for s in slots] == now
        ref = reference(dec, x[:, :8].unsqueeze(1), table, slots, now, False)
        assert float((out.double() - ref[0]).abs().max()) <= 2.0 ** -8 * float(ref[0].abs().max())


# ---------------------------------------------------------------- the cache itself

def e4m3_table():
    b = torch.arange(256, dtype=torch.uint8).view(FP8).double().numpy()
    return np.unique(b[np.isfinite(b)])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cache", [torch.bfloat16, FP8])
@pytest.mark.parametrize("counts", [[1, 1, 1], [0, 33, 1], [200, 0, 7], [5, 40, 300]])
def test_append_and_read(d, act, cache, counts):
    lens = [3, 16, 40]
    dec, ci, table, slots, g = make(3, [n + c for n, c in zip(lens, counts)], d=d, act=act,
                                    cache=cache, hkv=3, hq=3, seed=11)
    for s, n in zip(slots, lens):
        dec.slot_len[s] = n
    before = [t.clone() for t in (dec.k_cache, dec.v_cache)]
    n = sum(counts)
    k = torch.randn(n, 3, d, generator=g, device="cuda").to(act)
    v = (2.0 ** torch.randint(-30, 30, (n, 3, 1), generator=g, device="cuda")
         * torch.randn(n, 3, d, generator=g, device="cuda")).to(act)
    v[0] = 0
    cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    dec.append(k, v, ci, cu_tokens=cu)
    torch.cuda.synchronize()
    assert int(dec.dev_err.sum()) == 0
    written = torch.zeros(dec.k_cache.shape[:1] + dec.k_cache.shape[2:3], dtype=torch.bool)
    at, grid = 0, e4m3_table()
    for b, c in enumerate(counts):
        pos = np.arange(lens[b], lens[b] + c)
        p, o = table[slots[b]][pos // 16].astype(np.int64), pos % 16
        written[torch.from_numpy(p), torch.from_numpy(o)] = True
        for x, cc, ss in ((k, dec.k_cache, dec.k_scale), (v, dec.v_cache, dec.v_scale)):
            src = x[at:at + c]
            pi, oi = torch.from_numpy(p).cuda(), torch.from_numpy(o).cuda()
            if cache == torch.bfloat16:
                assert torch.equal(cc[pi, :, oi], src.bfloat16())
                continue
            got = cc.view(torch.uint8)[pi, :, oi].view(FP8).double().cpu().numpy()
            sc = ss[pi, :, oi].double().cpu().numpy()
            s64 = src.double().cpu().numpy()
            amax = np.maximum(np.abs(s64).max(-1), 2.0 ** -100)
            assert np.all(np.abs(sc - amax / 448) <= 2.0 ** -23 * amax / 448)
            want = s64 * (448 / amax)[..., None]
            i = np.clip(np.searchsorted(grid, want), 1, len(grid) - 1)
            half = np.minimum(np.abs(want - grid[i - 1]), np.abs(want - grid[i]))
            assert np.all(np.abs(got - want) <= half + 2.0 ** -20 * np.abs(want) + 1e-300)
        at += c
    keep = ~written.cuda()
    for now, old in zip((dec.k_cache, dec.v_cache), before):
        a, b = (t.view(torch.uint8) if t.dtype == FP8 else t.view(torch.int16) for t in (now, old))
        assert torch.equal(a.permute(0, 2, 1, 3)[keep], b.permute(0, 2, 1, 3)[keep])
    # read it back, from the first new token on
    dec.advance(ci, cu_tokens=cu)
    first = torch.tensor(lens, dtype=torch.int32, device="cuda")
    rk, rv = dec.read(ci, cu, n, first=first)
    torch.cuda.synchronize()
    assert int(dec.dev_err.sum()) == 0
    at = 0
    for b, c in enumerate(counts):
        ek, ev = cached(dec, table, slots[b], lens[b], lens[b] + c)
        for got, e in ((rk, ek), (rv, ev)):
            assert torch.equal(got[at:at + c], e.to(act) if act == torch.bfloat16 and
                               cache == torch.bfloat16 else e.float().to(act))
        at += c


def test_uniform_append_advance_and_rejection():
    import ssm_linear_attention_gb300 as ssm
    lens = [3, 30]
    dec, ci, table, slots, g = make(2, lens, T=4, seed=12, hkv=1, hq=1)
    k = torch.randn(2, 4, 1, 128, generator=g, device="cuda").bfloat16()
    dec.append(k, k, ci)
    dec.advance(ci, num_accepted=torch.tensor([0, 3], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert [int(dec.slot_len[s]) for s in slots] == [3, 33]
    dec.advance(ci, num_accepted=torch.tensor([5, -1], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert [int(dec.slot_len[s]) for s in slots] == [3, 33]
    assert int(dec.dev_err[0]) == ssm.RSSM_DEVERR_CURSOR
    dec.reset_slots(ci)
    torch.cuda.synchronize()
    assert [int(dec.slot_len[s]) for s in slots] == [0, 0]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_vector_that_is_not_finite_reads_back_as_nan(bad):
    dec, ci, table, slots, g = make(1, [0], cache=FP8, T=4, hkv=2, seed=13)
    k = torch.randn(1, 4, 2, 128, generator=g, device="cuda").bfloat16()
    k[0, 1, 1, 77] = bad
    dec.append(k, k, ci)
    dec.advance(ci)
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    rk, rv = dec.read(ci, cu, 4)
    torch.cuda.synchronize()
    for r in (rk, rv):
        assert bool(torch.isnan(r[1, 1]).all())
        assert int(torch.isnan(r).sum()) == 128


def test_append_and_read_flag_what_they_cannot_place():
    import ssm_linear_attention_gb300 as ssm
    lens = [30, 3, 3, 3]
    dec, ci, table, slots, g = make(4, lens, hkv=2, seed=14, max_pages=2)
    dec.page_table[slots[1], 0] = dec.num_pages
    bad = ci.clone()
    bad[2], bad[3] = -1, dec.num_slots
    kb, vb = dec.k_cache.clone(), dec.v_cache.clone()
    k = torch.ones(12, 2, 128, device="cuda", dtype=torch.bfloat16)
    cu = torch.tensor([0, 3, 6, 9, 12], dtype=torch.int32, device="cuda")
    dec.append(k, k, bad, cu_tokens=cu)             # row 0: 30, 31, then past the table
    torch.cuda.synchronize()
    assert int(dec.dev_err[0]) == ssm.RSSM_DEVERR_SLOT | ssm.RSSM_DEVERR_CURSOR | ssm.RSSM_DEVERR_PAGE
    page = int(table[slots[0]][1])
    kb[page, :, 14:] = 1
    vb[page, :, 14:] = 1
    assert torch.equal(dec.k_cache.view(torch.int16), kb.view(torch.int16))
    assert torch.equal(dec.v_cache.view(torch.int16), vb.view(torch.int16))
    dec.dev_err.zero_()
    rk = torch.full((12, 2, 128), 5.0, device="cuda", dtype=torch.bfloat16)
    rv = rk.clone()
    dec.read(bad, cu, 12, k=rk, v=rv, first=torch.tensor([29, 0, 0, 0], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()                        # row 0: 29 is committed, 30 and 31 are not
    assert int(dec.dev_err[0]) == ssm.RSSM_DEVERR_SLOT | ssm.RSSM_DEVERR_CURSOR | ssm.RSSM_DEVERR_PAGE
    assert bool((rk[1:] == 5).all()) and bool((rv[1:] == 5).all())
    assert bool(torch.isnan(rk[0]).all())


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes and 2^31 elements per tensor: the last pages are
    written, read and attended like the first."""
    import ssm_linear_attention_gb300 as ssm
    num_pages = (1 << 31) // (8 * 256 * 128) + 1000               # 2^31 elements and then some
    dec = ssm.PagedAttentionDecoder(8, 8, 128, 256, num_pages, 2, 4, 2, T=1)
    dec.page_table.copy_(torch.tensor([[num_pages - 1, num_pages - 2, 5, 6], [0, 1, 2, 3]]))
    ci = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    one = torch.randn(300, 8, 128, generator=g, device="cuda").bfloat16()
    two = torch.randn(300, 8, 128, generator=g, device="cuda").bfloat16()
    cu = torch.tensor([0, 300, 600], dtype=torch.int32, device="cuda")
    dec.append(torch.cat([one, one]), torch.cat([two, two]), ci, cu_tokens=cu)
    dec.advance(ci, cu_tokens=cu)
    rk, rv = dec.read(ci, cu, 600)
    q = torch.randn(1, 1, 8, 128, generator=g, device="cuda").bfloat16().expand(2, 1, 8, 128).contiguous()
    o = dec.decode(q, ci, appended=False)
    torch.cuda.synchronize()
    assert torch.equal(rk, torch.cat([one, one])) and torch.equal(rv, torch.cat([two, two]))
    assert torch.equal(dec.k_cache[num_pages - 1, :, 255], one[255])
    assert float((o[0] - o[1]).abs().max()) <= 2.0 ** -8 * float(o[0].abs().max())


def test_wrapper_refuses_layouts_it_cannot_read():
    dec, ci, table, slots, g = make(2, [3, 3], seed=15)
    good = torch.zeros(2, 1, 8, 128, device="cuda", dtype=torch.bfloat16)
    for q in (good.float(), good.transpose(2, 3).contiguous().transpose(2, 3),
              torch.zeros(2, 1, 8, 256, device="cuda", dtype=torch.bfloat16)[..., ::2],
              torch.zeros(3, 1, 8, 128, device="cuda", dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            dec.decode(q, ci)
    with pytest.raises(ValueError):
        dec.append(good[:, :, :2], good[:1, :, :2], ci)


@pytest.mark.parametrize("d", [64, 128])
def test_every_8_bit_code_counts(d):
    """Scores and values made of one code each, the subnormal ones included: a key whose
    first element is the vector's largest (and meets a query element of 0) and whose second
    is code c scores exactly c * scale; the values' columns run through the codes."""
    codes = [c for c in range(256) if c & 0x7f != 0x7f]
    n = len(codes)
    dec, ci, table, slots, g = make(1, [n], hq=1, hkv=1, d=d, cache=FP8, out=torch.float32, seed=21)
    val = torch.tensor(codes, dtype=torch.uint8, device="cuda").view(FP8).float()
    k = torch.zeros(n, 1, d, device="cuda")
    v = torch.zeros(n, 1, d, device="cuda")
    k[:, 0, 0] = 448.0
    k[:, 0, 1] = val
    v[:, 0, 0] = 448.0
    for c in range(1, d):
        v[:, 0, c] = val.roll(c)
    dec.slot_len.zero_()
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    dec.append(k.bfloat16(), v.bfloat16(), ci, cu_tokens=cu)
    dec.advance(ci, cu_tokens=cu)
    p = torch.from_numpy(table[slots[0]][np.arange(n) // 16].astype(np.int64)).cuda()
    o = torch.arange(n, device="cuda") % 16
    assert torch.equal(dec.k_cache.view(torch.uint8)[p, 0, o, 1].cpu(), torch.tensor(codes, dtype=torch.uint8))
    for t in range(n):                                  # one token at a time: its value, exactly
        if t % 7:
            continue
        one = torch.zeros(1, 1, 1, d, device="cuda", dtype=torch.bfloat16)
        dec.slot_len[slots[0]] = t + 1
        dec.window = 1
        out, lse = dec.decode(one, ci, appended=False, with_lse=True)
        torch.cuda.synchronize()
        assert float((out[0, 0, 0] - v[t, 0]).abs().max()) <= 2.0 ** -20 * 448
        assert torch.all(((out[0, 0, 0] - v[t, 0]).abs() <= 2.0 ** -20 * v[t, 0].abs()))
        one[..., 1] = 1.0                               # its score: c * scale / sqrt(d)
        out, lse = dec.decode(one, ci, appended=False, with_lse=True)
        torch.cuda.synchronize()
        want = float(val[t]) * dec.scale
        assert abs(float(lse[0, 0, 0]) - want) <= 2.0 ** -19 * abs(want) + 2e-6


# 9 queries a key head and more: chunks of 128 tokens, query blocks of 16, 32 and 64
WIDE = [
    (9, [0, 1, 15, 16, 17, 127, 128, 129, 2500], dict(hq=18, hkv=2, page=16)),
    (9, [0, 1, 15, 16, 17, 127, 128, 129, 2500], dict(hq=16, hkv=1, d=64, page=64, cache=FP8)),
    (4, [255, 256, 257, 3], dict(hq=34, hkv=2, page=32, cache=FP8)),
    (4, [1000, 111, 112, 113], dict(hq=16, hkv=2, T=3, d=64, page=16)),
    (3, [5, 4000, 300], dict(hq=8, hkv=2, T=8, page=256, out=torch.float32)),
    (3, [130, 700, 64], dict(hq=22, hkv=2, T=3, page=16, cache=FP8, out=torch.float32)),
    (2, [640, 1300], dict(hq=21, hkv=1, T=3, d=64, page=128)),
    (2, [641, 1301], dict(hq=16, hkv=2, T=8, page=64, cache=FP8, d=64)),
    (1, [70001], dict(hq=32, hkv=1, page=64)),
    (2, [30000, 77], dict(hq=64, hkv=1, page=32, cache=FP8)),
    (3, [900, 60, 1025], dict(hq=16, hkv=2, T=4, window=130, page=16)),
    (3, [900, 60, 1025], dict(hq=16, hkv=2, T=8, window=128, page=64, cache=FP8)),
    (2, [500, 2], dict(hq=16, hkv=1, T=2, window=1, page=32, d=64)),
    (1100, [(53 * i) % 35 for i in range(1100)], dict(hkv=1, hq=16, d=64)),
    (200, [(37 * i) % 301 for i in range(200)], dict(hkv=3, hq=48, T=2, page=32)),
]


@pytest.mark.parametrize("batch,lens,kw", WIDE)
@pytest.mark.parametrize("appended", [True, False])
def test_decode_of_many_queries_matches_float64(batch, lens, kw, appended):
    test_decode_matches_float64(batch, lens, kw, appended)


@pytest.mark.parametrize("T,hq", [(2, 16), (4, 16), (8, 16)])
@pytest.mark.parametrize("cache", [torch.bfloat16, FP8])
def test_many_queries_and_missing_pages(cache, T, hq):
    """Pages that are missing at the start (the first chunk is hidden as a whole), inside a
    chunk, and of a whole row."""
    import ssm_linear_attention_gb300 as ssm
    lens = [400, 290, 33]
    dec, ci, table, slots, g = make(3, lens, hq=hq, hkv=2, T=T, cache=cache, seed=31)
    fill(dec, ci, table, slots, lens, g)
    q = torch.randn(3, T, hq, 128, generator=g, device="cuda").to(torch.bfloat16)
    dec.page_table[slots[0], :9] = -1                      # positions 0..143
    dec.page_table[slots[1], 3] = dec.num_pages            # 48..63
    dec.page_table[slots[1], 16] = -5                      # 256..271
    dec.page_table[slots[2]] = -1
    o, lse = dec.decode(q, ci, appended=False, with_lse=True)
    torch.cuda.synchronize()
    assert int(dec.dev_err[0]) == ssm.RSSM_DEVERR_PAGE
    for b, hid in ((0, set(range(144))), (1, set(range(48, 64)) | set(range(256, 272)))):
        ref = reference(dec, q[b:b + 1], table, slots[b:b + 1], lens[b:b + 1], False, hid)
        check(dec, o[b:b + 1], lse[b:b + 1], ref)
    assert bool((o[2] == 0).all()) and bool((lse[2] == -math.inf).all())


@pytest.mark.parametrize("T,hq", [(4, 8), (8, 8), (16, 8)])
def test_many_queries_window_and_drafts_nan_included(T, hq):
    """Values that are not finite at positions that only some drafts see: the last tokens and
    those at the windows' beginnings."""
    lens = [300]
    W = 150
    dec, ci, table, slots, g = make(1, lens, hq=hq, hkv=2, T=T, window=W, seed=41)
    fill(dec, ci, table, slots, lens, g)
    k = torch.randn(1, T, 2, 128, generator=g, device="cuda").bfloat16()
    v = torch.randn(1, T, 2, 128, generator=g, device="cuda").bfloat16()
    v[0, T - 1, :, 7] = float("nan")
    v[0, T - 2, 1, 100] = float("inf")
    dec.append(k, v, ci)
    first = lens[0] + 1 - W                                  # draft 0 alone sees this one
    page, off = int(table[slots[0]][first // 16]), first % 16
    dec.v_cache[page, 0, off, 64] = float("-inf")
    q = torch.randn(1, T, hq, 128, generator=g, device="cuda").bfloat16()
    o, lse = dec.decode(q, ci, with_lse=True)
    torch.cuda.synchronize()
    G = hq // 2
    want = torch.zeros(1, T, hq, 128, dtype=torch.bool, device="cuda")
    want[0, T - 1, :, 7] = True
    assert torch.equal(torch.isnan(o), want)
    inf = torch.zeros_like(want)
    inf[0, T - 2:, G:, 100] = True
    inf[0, 0, :G, 64] = True
    assert torch.equal(torch.isinf(o), inf)
    assert bool((o[0, T - 2:, G:, 100] > 0).all()) and bool((o[0, 0, :G, 64] < 0).all())
    ref = reference(dec, q, table, slots, lens, True)
    clean = [t.clone() for t in ref]
    bad = want | inf
    got = o.clone()
    got[bad] = 0
    clean[0][bad] = 0
    clean[2][bad] = 0
    check(dec, got, lse, clean)


@pytest.mark.parametrize("cache", [torch.bfloat16, FP8])
@pytest.mark.parametrize("T", [4, 8])
def test_many_queries_whose_maxima_move(cache, T):
    """Scores that rise through the row (each chunk passes the maximum by far), fall, and rise for
    some queries alone."""
    lens = [1500, 700]
    dec, ci, table, slots, g = make(2, lens, hq=16, hkv=2, T=T, cache=cache, seed=51)
    n = sum(lens)
    k = 0.1 * torch.randn(n, 2, 128, generator=g, device="cuda")
    v = torch.randn(n, 2, 128, generator=g, device="cuda")
    rise = torch.cat([torch.arange(m, device="cuda") for m in lens])[:, None] / 16.0
    k[:, :, 0], k[:, :, 1] = rise, -rise
    keep = dec.slot_len.clone()
    dec.slot_len.zero_()
    dec.append(k.bfloat16(), v.bfloat16(), ci,
               cu_tokens=torch.tensor([0, lens[0], n], dtype=torch.int32, device="cuda"))
    dec.slot_len.copy_(keep)
    q = 0.3 * torch.randn(2, T, 16, 128, generator=g, device="cuda")
    q[:, :, 0::3, 0] = 20.0
    q[:, :, 1::3, 1] = 20.0
    o, lse = dec.decode(q.bfloat16(), ci, appended=False, with_lse=True)
    torch.cuda.synchronize()
    assert int(dec.dev_err.sum()) == 0
    o64, lse64, w = reference(dec, q.bfloat16(), table, slots, lens, False)
    # scores reach the hundreds: float32 leaves 2^-24 of them, which the weights see absolutely
    bound = 2.0 ** -8 * o64.abs() + (2.0 ** -15 + 2.0 ** -16) * 8 * w + 1e-30
    assert float(((o.double() - o64).abs() / bound).max()) <= 1.0
    assert float((lse.double() - lse64).abs().max()) <= 2.0 ** -22 * float(lse64.abs().max()) + 2e-5


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 30, 2 ** 30 - 1])
@pytest.mark.parametrize("hq", [2, 16])
def test_a_window_beyond_any_length(window, hq):
    lens = [130, 20]
    dec, ci, table, slots, g = make(2, lens, hq=hq, hkv=2, T=4, window=window, seed=61)
    fill(dec, ci, table, slots, lens, g)
    k = torch.randn(2, 4, 2, 128, generator=g, device="cuda").bfloat16()
    dec.append(k, k, ci)
    q = torch.randn(2, 4, hq, 128, generator=g, device="cuda").bfloat16()
    o, lse = dec.decode(q, ci, with_lse=True)
    torch.cuda.synchronize()
    dec.window = 0
    check(dec, o, lse, reference(dec, q, table, slots, lens, True))
