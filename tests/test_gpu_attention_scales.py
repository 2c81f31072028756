"""Attention over an 8-bit cache whose value scales differ by much, or are zero, and whose weights
do: one token far ahead of the rest, as in a long context.

The outputs are float32, and each is compared with float64 in units of the terms' size
w = sum_p p |v_p| (of the same output). What the arithmetic leaves, for scores of up to some 40
(log2 units, made by one element of the query) and at most a few thousand additions a sum:
  * a score: 8 steps of the matrix unit, each cutting at most 2^-23 of some 64: 2^-14 absolute in
    the worst case, 2^-17 where the steps are not all at the top; a weight sees it times ln 2;
  * a weight in two bf16 parts: 2^-17; a value scale as a float32 factor: 2^-24;
  * the matrix unit's sums over a group's or chunk's tokens: 2^-16.
The weight and the sum of weights both carry the score's part: 2^-13 of w bounds them all."""
import math

import numpy as np
import pytest
import torch

from tests import test_gpu_attention as A

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn
BOUND = 2.0 ** -13

# Queries a key head that take each of the kernels: one warp a tile, warps that share a tile,
# the tensor-memory kernel's two query blocks; float32 activations in the first two forms.
FORMS = [(4, torch.bfloat16), (16, torch.bfloat16), (32, torch.bfloat16), (64, torch.bfloat16),
         (4, torch.float32), (32, torch.float32)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    import ssm_linear_attention_gb300 as ssm
    ssm.lib()


def row(n, M, act, d, seed, cache=FP8, hkv=2):
    """One row of n committed tokens with random keys and values; the first element of a key
    scores for itself (q's first element is 16, its others are small)."""
    import ssm_linear_attention_gb300 as ssm
    hkv = hkv if M < 64 else 1
    dec, ci, table, slots, g = A.make(1, [n], hq=hkv * M, hkv=hkv, d=d, page=64, cache=cache,
                                      act=act, out=torch.float32, seed=seed)
    k = 0.05 * torch.randn(n, hkv, d, generator=g, device="cuda")
    k[:, :, 0] = 0
    v = torch.randn(n, hkv, d, generator=g, device="cuda")
    q = 0.05 * torch.randn(1, 1, hkv * M, d, generator=g, device="cuda")
    q[..., 0] = 16.0
    return dec, ci, table, slots, g, k, v, q.to(act)


def append(dec, ci, k, v):
    n = k.shape[0]
    dec.slot_len.zero_()
    dec.append(k.to(dec.act_dtype), v.to(dec.act_dtype), ci,
               cu_tokens=torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    dec.slot_len[ci.long()] = n


def nats(x, d):
    """The key element that puts a token x ahead (its query element is 16)."""
    return x * d ** 0.5 / 16


def places(dec, table, slots, pos):
    pos = np.asarray(pos)
    return (torch.from_numpy(table[slots[0]][pos // dec.page_size].astype(np.int64)).cuda(),
            torch.from_numpy(pos % dec.page_size).cuda())


def compare(dec, ci, q, table, slots, n):
    o, lse = dec.decode(q, ci, appended=False, with_lse=True)
    torch.cuda.synchronize()
    assert int(dec.dev_err.sum()) == 0
    ro, rl, w = A.reference(dec, q, table, slots, [n], False)
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(lse).all())
    worst = float(((o.double() - ro).abs() - BOUND * w).max())
    assert worst <= 1e-30, (worst, float((o.double() - ro).abs().max()), float(w.max()))
    # (scores in the tens: 2^-22 of them, and the logarithm's own few 2^-22)
    assert float((lse.double() - rl).abs().max()) <= 2e-5 + 2.0 ** -20 * float(rl.abs().max())


@pytest.mark.parametrize("M,act", FORMS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,ahead", [(131072, 14.0), (131072, 17.0), (131072, 20.0), (20000, 30.0)])
def test_one_token_far_ahead_of_many(M, act, d, n, ahead):
    """Half of the leader's value is zero: these columns are the others' alone, with weights of
    e^-ahead."""
    dec, ci, table, slots, g, k, v, q = row(n, M, act, d, int(ahead))
    lead = n // 3
    k[lead, :, 0] = nats(ahead, d)
    v = v.abs() + 0.5
    v[lead, :, ::2] = 0
    append(dec, ci, k, v)
    compare(dec, ci, q, table, slots, n)


@pytest.mark.parametrize("M,act", FORMS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("which", ["first", "all", "some", "last"])
def test_value_scales_of_zero(M, act, d, which):
    """A token whose value scale is zero has its weight and adds nothing."""
    n = 700
    dec, ci, table, slots, g, k, v, q = row(n, M, act, d, 1)
    append(dec, ci, k, v)
    pos = {"first": range(40), "all": range(n), "some": range(3, n, 5), "last": range(n - 300, n)}[which]
    p, o = places(dec, table, slots, list(pos))
    dec.v_scale[p, :, o] = 0.0
    compare(dec, ci, q, table, slots, n)


@pytest.mark.parametrize("M,act", FORMS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ahead", [5.5, 10.0, 15.0])
@pytest.mark.parametrize("zero", [0.0, 2.0 ** -149, 2.0 ** -100])
def test_scaled_token_ahead_of_many_of_scale_zero(M, act, d, ahead, zero):
    """Thousands of tokens whose values vanish, behind one whose values do not: their weights
    are in the sum all the same."""
    n = 4096
    dec, ci, table, slots, g, k, v, q = row(n, M, act, d, 2)
    k[100, :, 0] = nats(ahead, d)
    append(dec, ci, k, v)
    p, o = places(dec, table, slots, [i for i in range(n) if i != 100])
    dec.v_scale[p, :, o] = zero
    compare(dec, ci, q, table, slots, n)


@pytest.mark.parametrize("M,act", FORMS)
@pytest.mark.parametrize("d", [64, 128])
def test_values_over_eighty_binades(M, act, d):
    n = 900
    dec, ci, table, slots, g, k, v, q = row(n, M, act, d, 3)
    k[:, :, 0] = nats(1.0, d) * torch.randn(n, 2 if M < 64 else 1, generator=g, device="cuda")
    v *= 2.0 ** torch.randint(-40, 41, (n, 1, 1), generator=g, device="cuda")
    append(dec, ci, k, v)
    compare(dec, ci, q, table, slots, n)


@pytest.mark.parametrize("M,act", FORMS)
@pytest.mark.parametrize("d", [64, 128])
def test_a_value_that_is_not_finite_leaves_the_sum_of_weights(M, act, d):
    """The outputs that see it are NaN; lse, which is the scores', is not."""
    n = 300
    dec, ci, table, slots, g, k, v, q = row(n, M, act, d, 4)
    v[123, 0, 5] = float("nan")
    append(dec, ci, k, v)
    o, lse = dec.decode(q, ci, appended=False, with_lse=True)
    torch.cuda.synchronize()
    heads = dec.HQ // dec.HKV
    assert bool(torch.isnan(o[:, :, :heads]).all())
    assert bool(torch.isfinite(o[:, :, heads:]).all())
    rl = A.reference(dec, q, table, slots, [n], False)[1]
    assert float((lse.double() - rl).abs().max()) <= 2e-5


@pytest.mark.parametrize("M,act", FORMS)
def test_8_bit_nan_codes_of_a_caller_s_cache_show(M, act):
    """append never writes the NaN codes, but a cache may be the caller's."""
    n = 200
    dec, ci, table, slots, g, k, v, q = row(n, M, act, 128, 5)
    append(dec, ci, k, v)
    p, o = places(dec, table, slots, [77])
    dec.v_cache.view(torch.uint8)[p, 0, o, 9] = 0x7f
    dec.v_cache.view(torch.uint8)[p, 0, o, 64] = 0xff
    out = dec.decode(q, ci, appended=False)
    torch.cuda.synchronize()
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[:, :, :dec.HQ // dec.HKV, [9, 64]] = True
    assert torch.equal(torch.isnan(out), bad)


@pytest.mark.parametrize("T,hq", [(3, 8), (4, 16), (8, 16)])
def test_drafts_and_scales_that_only_some_see(T, hq):
    """Infinite and NaN value scales at the drafts' own positions: the drafts before them do not
    see them, those from them on do."""
    lens = [61]
    dec, ci, table, slots, g = A.make(1, lens, hq=hq, hkv=2, T=T, cache=FP8, page=64,
                                      out=torch.float32, seed=9)
    A.fill(dec, ci, table, slots, lens, g)
    k = torch.randn(1, T, 2, 128, generator=g, device="cuda").bfloat16()
    dec.append(k, k, ci)
    p, o = places(dec, table, slots, [lens[0] + T - 1])
    dec.v_scale[p, 0, o] = float("nan")
    dec.v_scale[p, 1, o] = float("inf")
    q = torch.randn(1, T, hq, 128, generator=g, device="cuda").bfloat16()
    out, lse = dec.decode(q, ci, with_lse=True)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out[:, :-1]).all()) and not bool(torch.isfinite(out[:, -1]).any())
    assert bool(torch.isfinite(lse).all())
    ro, rl, w = A.reference(dec, q, table, slots, lens, True)
    assert float(((out.double() - ro).abs() - BOUND * w)[:, :-1].max()) <= 1e-30
    assert float((lse.double() - rl).abs().max()) <= 2e-5


@pytest.mark.parametrize("T,hq", [(2, 32), (4, 32), (8, 16)])
def test_many_short_rows_whose_queries_differ_in_size(T, hq):
    """(row, head)s of one chunk each, dozens to a CTA, with queries of sizes 2^-8 to 2^7: each
    one's score factors are its own, call after call."""
    B = 700
    lens = [1 + (61 * i) % 120 for i in range(B)]
    dec, ci, table, slots, g = A.make(B, lens, hq=hq, hkv=2, d=64, T=T, cache=FP8, page=128,
                                      out=torch.float32, seed=13)
    A.fill(dec, ci, table, slots, lens, g)
    q = torch.randn(B, T, hq, 64, generator=g, device="cuda")
    q *= 2.0 ** torch.randint(-8, 8, (B, T, hq, 1), generator=g, device="cuda") / 16
    q = q.bfloat16()
    o, lse = dec.decode(q, ci, appended=False, with_lse=True)
    torch.cuda.synchronize()
    first, first_lse = o.clone(), lse.clone()
    rows = [0, 1, 2, 350, 351, 697, 698, 699]
    ro, rl, w = A.reference(dec, q[rows], table, [slots[b] for b in rows], [lens[b] for b in rows], False)
    assert float(((o[rows].double() - ro).abs() - BOUND * w).max()) <= 1e-30
    assert float((lse[rows].double() - rl).abs().max()) <= 2e-5 + 2.0 ** -20 * float(rl.abs().max())
    for _ in range(50):
        o, lse = dec.decode(q, ci, appended=False, with_lse=True)
        assert torch.equal(o, first) and torch.equal(lse, first_lse)


@pytest.mark.parametrize("cache", [torch.bfloat16, FP8])
@pytest.mark.parametrize("M,act", FORMS)
@pytest.mark.parametrize("d", [64, 128])
def test_values_near_the_largest_float(M, act, d, cache):
    """Scores that rise by 5 nats through the row, values of 2^122: the sum of softmax weights times
    values stays below float32's largest, and no weight is above 1."""
    n = 640
    dec, ci, table, slots, g, k, v, q = row(n, M, act, d, 6, cache=cache)
    k[:, :, 0] = nats(1.0, d) * torch.linspace(0, 5, n, device="cuda")[:, None]
    v = (1 + v.abs()) * 2.0 ** 114
    v[n // 2:] *= 2.0 ** 4
    append(dec, ci, k, v)
    compare(dec, ci, q, table, slots, n)


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hq,d", [(2, 128), (2, 64), (32, 128), (32, 64)])
def test_infinite_keys_under_queries_of_any_size(act, hq, d):
    """An infinite element of a key makes its score infinite with the sign of the product, a weight of
    zero or (+infinity) a NaN, also where the query enters the product in parts."""
    lens = [300]
    dec, ci, table, slots, g = A.make(1, lens, hq=hq, hkv=2, d=d, act=act, out=torch.float32, seed=17)
    A.fill(dec, ci, table, slots, lens, g)
    q = torch.randn(1, 1, hq, d, generator=g, device="cuda").to(act)
    q[..., 3] = q[..., 3].abs() + 0.1
    p, o = places(dec, table, slots, range(300))
    dec.k_cache[p, :, o, 3] = -math.inf                      # every score -infinity
    out, lse = dec.decode(q, ci, appended=False, with_lse=True)
    torch.cuda.synchronize()
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    dec.k_cache[p[40:44], :, o[40:44], 3] = 0.5              # four tokens left
    out, lse = dec.decode(q, ci, appended=False, with_lse=True)
    torch.cuda.synchronize()
    ro, rl, w = A.reference(dec, q, table, slots, lens, False, hidden=set(range(300)) - {40, 41, 42, 43})
    assert float(((out.double() - ro).abs() - BOUND * w).max()) <= 1e-30
    assert float((lse.double() - rl).abs().max()) <= 2e-5
    dec.k_cache[p[100], 0, o[100], 3] = math.inf
    out, lse = dec.decode(q, ci, appended=False, with_lse=True)
    torch.cuda.synchronize()
    G = hq // 2
    assert bool(torch.isnan(out[:, :, :G]).all()) and bool(torch.isnan(lse[:, :, :G]).all())
    assert float(((out.double() - ro).abs() - BOUND * w)[:, :, G:].max()) <= 1e-30
