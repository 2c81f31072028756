"""rssm_rope against exact angles.

The angle's fraction of a turn is exact up to 2^-32 of a turn and the rounding to float32
(2^-25 of half a turn): at most 2^-22.7 rad together; the cosine and sine are within 2 units of the
last place of the true ones at that angle (2^-23), and the product with mscale and the two products
and their sum round once each (2^-24 of a term). In sum |y - ref| <= 2^-21 (|x| + |y|) mscale, and for bf16
half a spacing of the output (2^-8 of the value covers it) beside it."""
import fractions
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

PI2 = fractions.Fraction("6.283185307179586476925286766559005768")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    import ssm_linear_attention_gb300 as ssm
    ssm.lib()


def angles(positions, freqs):
    """pos * f modulo a turn, in exact fractions, then float64."""
    turns = [fractions.Fraction(f) / PI2 for f in freqs]
    return torch.tensor([[float(p * t % 1) * 2 * math.pi for t in turns] for p in positions], dtype=torch.float64, device="cuda")


def reference(x, a, m, R, inter):
    y = x.double().clone()
    c, s = (m * a.cos())[:, None], (m * a.sin())[:, None]
    i = (slice(0, R, 2), slice(1, R, 2)) if inter else (slice(0, R // 2), slice(R // 2, R))
    u, v = x.double()[..., i[0]], x.double()[..., i[1]]
    y[..., i[0]], y[..., i[1]] = u * c - v * s, v * c + u * s
    size = x.double().abs()
    both = size[..., i[0]] + size[..., i[1]]
    bound = torch.zeros_like(size)
    bound[..., i[0]] = bound[..., i[1]] = both * abs(m) * 2.0 ** -21
    return y, bound


def compare(got, x, a, rot):
    ref, bound = reference(x, a, rot.mscale, rot.R, rot.interleaved)
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * ref.abs()
    assert bool(((got.double() - ref).abs() <= bound + 1e-37).all())


SHAPES = [(1, 1, 64, 64), (8, 2, 128, 128), (5, 3, 80, 32), (2, 1, 128, 30), (4, 0, 96, 24), (2, 2, 64, 16), (3, 1, 512, 2),
          (2, 2, 256, 256), (1, 8, 40, 40), (7, 1, 8, 4), (12, 4, 192, 48)]


@pytest.mark.parametrize("hq,hk,d,r", SHAPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
def test_rope_matches_exact_angles(hq, hk, d, r, inter, act):
    import ssm_linear_attention_gb300 as ssm
    g = torch.Generator(device="cuda")
    g.manual_seed(hq * 100 + d + r)
    positions = [0, 1, -1, 17, 4095, 131071, 1000003, 2 ** 31 - 1, -2 ** 31, 123456789]
    n = len(positions)
    rot = ssm.Rotary(hq, hk, d, rot_dim=r, interleaved=inter, base=500000.0, act_dtype=act,
                     scaling={"type": "yarn", "factor": 4.0, "original": 2048})
    pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
    a = angles(positions, rot.frequencies)
    # slices of a fused projection, into dense tensors and in place
    fused = torch.randn(n, hq + 2 * hk + 1, d, generator=g, device="cuda").to(act)
    q, k = fused[:, :hq], fused[:, hq:hq + hk]
    qd, kd = q.clone(), k.clone()
    if hk == 0:
        qo = torch.full_like(qd, 7)
        rot(q, positions=pos, q_out=qo)
        outs = [(qo, qd)]
    else:
        qo, ko = torch.full_like(qd, 7), torch.full_like(kd, 7)
        rot(q, k, positions=pos, q_out=qo, k_out=ko)
        outs = [(qo, qd), (ko, kd)]
    torch.cuda.synchronize()
    for got, x in outs:
        if x.numel():
            compare(got, x, a, rot)
            assert torch.equal(got[..., r:], x[..., r:])
    rest = fused[:, hq + hk:].clone()
    rot(q, k if hk else None, positions=pos)
    torch.cuda.synchronize()
    assert torch.equal(q, outs[0][0]) and torch.equal(fused[:, hq + hk:], rest)
    if hk:
        assert torch.equal(k, outs[1][0])


@pytest.mark.parametrize("n_rows,most", [(1, 1), (3, 70), (40, 9), (2, 1500)])
def test_positions_from_slots_are_those_of_an_append(n_rows, most):
    import ssm_linear_attention_gb300 as ssm
    g = torch.Generator().manual_seed(n_rows)
    counts = [int(torch.randint(0, most + 1, (1,), generator=g)) for _ in range(n_rows)]
    counts[0] = most
    n = sum(counts)
    slots = torch.randperm(n_rows + 3, generator=g)[:n_rows].to(torch.int32)
    lens = torch.randint(0, 3000, (n_rows + 3,), generator=g).to(torch.int32)
    cu = torch.zeros(n_rows + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(counts).cumsum(0)
    pos = torch.cat([lens[s] + torch.arange(c) for s, c in zip(slots.tolist(), counts)]).to(torch.int32).cuda()
    rot = ssm.Rotary(4, 2, 64)
    q, k = torch.randn(n, 4, 64, device="cuda").bfloat16(), torch.randn(n, 2, 64, device="cuda").bfloat16()
    want = rot(q, k, positions=pos, q_out=torch.empty_like(q), k_out=torch.empty_like(k))
    got = rot(q, k, cache_indices=slots.cuda(), slot_len=lens.cuda(), cu_tokens=cu.cuda(), q_out=torch.empty_like(q),
              k_out=torch.empty_like(k))
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and int(rot.dev_err.sum()) == 0


def test_padding_rows_and_tokens_outside_rows_are_left_alone():
    import ssm_linear_attention_gb300 as ssm
    rot = ssm.Rotary(2, 1, 64, act_dtype=torch.float32)
    q, k = torch.randn(12, 2, 64, device="cuda"), torch.randn(12, 1, 64, device="cuda")
    qo, ko = torch.full_like(q, 5), torch.full_like(k, 5)
    slots = torch.tensor([1, -1, 3, 99], dtype=torch.int32, device="cuda")
    lens = torch.tensor([0, 10, 0, 7], dtype=torch.int32, device="cuda")
    cu = torch.tensor([1, 4, 6, 8, 10], dtype=torch.int32, device="cuda")   # token 0 and 10, 11: nobody's
    rot(q, k, cache_indices=slots, slot_len=lens, cu_tokens=cu, q_out=qo, k_out=ko)
    torch.cuda.synchronize()
    assert int(rot.dev_err[0]) == ssm.RSSM_DEVERR_SLOT
    for o in (qo, ko):
        assert bool((o[[0, 4, 5, 8, 9, 10, 11]] == 5).all()) and not bool((o[[1, 2, 3, 6, 7]] == 5).any())
    a = angles([10, 11, 12, 7, 8], rot.frequencies)
    at = [1, 2, 3, 6, 7]
    compare(qo[at], q[at], a, rot)
    # rows of equal length
    want, _ = reference(q, angles([10, 11, 12, 0, 0, 0, 7, 8, 9, 0, 0, 0], rot.frequencies), 1.0, 64, False)
    qo.fill_(5)
    rot(q, k, cache_indices=slots, slot_len=lens, q_out=qo, k_out=ko)
    torch.cuda.synchronize()
    assert bool((qo[3:6] == 5).all()) and bool((qo[9:] == 5).all())
    assert float((qo[[0, 1, 2, 6, 7, 8]].double() - want[[0, 1, 2, 6, 7, 8]]).abs().max()) < 1e-4


def test_negative_positions_turn_back():
    import ssm_linear_attention_gb300 as ssm
    rot = ssm.Rotary(3, 3, 128, interleaved=True, act_dtype=torch.float32)
    x = torch.randn(50, 3, 128, device="cuda")
    pos = torch.randint(0, 10 ** 6, (50,), dtype=torch.int32, device="cuda")
    y, _ = rot(x, x.clone(), positions=pos, q_out=torch.empty_like(x))
    z, _ = rot(y, y.clone(), positions=-pos, q_out=torch.empty_like(x))
    torch.cuda.synchronize()
    # two rotations, each within 2^-21 (|x| + |y|) of exact, of values up to 6
    assert float((z - x).abs().max()) <= 2 * 2.0 ** -21 * 16


def test_captured_rotation_follows_the_lengths():
    import ssm_linear_attention_gb300 as ssm
    rot = ssm.Rotary(4, 1, 64, act_dtype=torch.float32)
    q, k = torch.randn(3, 4, 64, device="cuda"), torch.randn(3, 1, 64, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    slots = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    lens = torch.tensor([3, 5, 7], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rot(q, k, cache_indices=slots, slot_len=lens, q_out=qo, k_out=ko)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rot(q, k, cache_indices=slots, slot_len=lens, q_out=qo, k_out=ko)
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        compare(qo, q, angles([int(lens[s]) for s in (2, 0, 1)], rot.frequencies), rot)
        lens += 1000


def test_runner_refusals():
    import ssm_linear_attention_gb300 as ssm
    rot = ssm.Rotary(4, 2, 64)
    q, k = torch.randn(6, 4, 64, device="cuda").bfloat16(), torch.randn(6, 2, 64, device="cuda").bfloat16()
    pos = torch.zeros(6, dtype=torch.int32, device="cuda")
    slots, lens = pos[:2].clone(), pos[:3].clone()
    for args, kw in (((q, k), {}), ((q, None), dict(positions=pos)), ((q, k[:5]), dict(positions=pos)),
                     ((q, k), dict(positions=pos[:5])), ((q, k), dict(positions=pos.long())), ((q.float(), k), dict(positions=pos)),
                     ((q, k), dict(positions=pos, cache_indices=slots, slot_len=lens)), ((q, k), dict(cache_indices=slots)),
                     ((q, k), dict(positions=pos.cpu())), ((q.cpu(), k), dict(positions=pos)),
                     ((q[:5], k[:5]), dict(cache_indices=slots, slot_len=lens)), ((q, k), dict(positions=pos, q_out=q[:5])),
                     ((q.transpose(1, 2), k), dict(positions=pos)), ((q, k), dict(cache_indices=slots, slot_len=lens, cu_tokens=pos[:2]))):
        with pytest.raises(ValueError):
            rot(*args, **kw)
    with pytest.raises(ValueError):
        ssm.Rotary(4, 2, 64, frequencies=[1.0] * 31)
    with pytest.raises(ssm.RSSMError):
        ssm.Rotary(1, 1, 100)(torch.zeros(1, 1, 100, device="cuda").bfloat16(), torch.zeros(1, 1, 100, device="cuda").bfloat16(),
                              positions=pos[:1])
