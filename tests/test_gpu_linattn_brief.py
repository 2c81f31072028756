"""rssm_linattn_prompt over rows of few tokens, which have a kernel of their own for bf16 activations (rows of at most 32, where
that is no less than the average): the bounds of longer rows, whose sums have more terms and the same parts."""
import pytest
import torch

from .test_gpu_linattn import BF, F32, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    import ssm_linear_attention_gb300 as ssm
    ssm.lib()


@pytest.mark.parametrize("state", [BF, F32])
@pytest.mark.parametrize("out", [BF, F32])
def test_every_length(state, out):
    import ssm_linear_attention_gb300 as ssm
    c = Case(list(range(65)), H=3, G=3, state=state, out=out, resume=0x5a5a5a5a5a5a5a5a5)
    c.check(*c.run(ssm))


@pytest.mark.parametrize("N,P", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("H,G", [(1, 1), (6, 2), (5, 1)])
@pytest.mark.parametrize("decay,w", [("head", False), ("token", True)])
def test_head_layouts(N, P, H, G, decay, w):
    import ssm_linear_attention_gb300 as ssm
    c = Case([17, 0, 64, 1, 16, 31, 33], H=H, G=G, N=N, P=P, decay=decay, w=w, resume=0b0101110)
    c.check(*c.run(ssm))


def test_a_longer_row_among_them():
    import ssm_linear_attention_gb300 as ssm
    c = Case([5, 65, 2, 32, 130, 1, 64, 0, 24, 7, 31, 8], resume=0b1011101)
    assert sum(c.lens) <= 32 * len(c.lens)
    c.check(*c.run(ssm))


def test_resets_and_strong_decays():
    import ssm_linear_attention_gb300 as ssm
    c = Case([48, 20, 3], rate=60.0, resume=0b111)
    c.g[7, 1] = -float("inf")
    c.g[50, 0] = -1000.0
    c.check(*c.run(ssm))


@pytest.mark.parametrize("token", [0, 1, 8, 15, 16, 25, 31, 32, 47])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_value_that_is_not_finite_stays_behind_its_token(token, bad):
    import ssm_linear_attention_gb300 as ssm
    good = Case([50, 3, 11], resume=0b111)
    o, s = good.run(ssm)
    for p in (0, 9, 77):
        c = Case([50, 3, 11], resume=0b111)
        c.v[token, 2, p] = bad
        oo, ss = c.run(ssm)
        assert not bool(torch.isfinite(oo[token:50, 2, p].float()).any())
        assert not bool(torch.isfinite(ss[c.slots[0], 2, p].float()).any())
        oo, ss = oo.clone(), ss.clone()
        oo[token:50, 2, p] = o[token:50, 2, p]
        ss[c.slots[0], 2, p] = s[c.slots[0], 2, p]
        assert torch.equal(oo, o) and torch.equal(ss, s)


@pytest.mark.parametrize("each", [1, 24, 32, 33])
def test_equal_rows_without_a_list(each):
    import ssm_linear_attention_gb300 as ssm
    c = Case([each] * 5, resume=0b10110)
    want, state = (x.clone() for x in c.run(ssm))
    layer = c.layer(ssm)
    o = layer.prompt(c.q, c.k, c.v, c.g, c.slots, w=c.w, resume=c.resume)
    torch.cuda.synchronize()
    c.check(o, layer.state)
    assert torch.equal(o, want) and torch.equal(layer.state, state)


@pytest.mark.parametrize("lens", [[5, 7, 3], [5, 70, 3, 2, 4, 1, 8]])
def test_padding_and_bad_rows(lens):
    import ssm_linear_attention_gb300 as ssm
    c = Case(lens, resume=0)
    want, state = (x.clone() for x in c.run(ssm))
    layer = c.layer(ssm)
    slots = c.slots.clone()
    slots[0], slots[2] = -1, len(lens) + 2
    layer.o.fill_(7)
    o = layer.prompt(c.q, c.k, c.v, c.g, slots, cu_tokens=c.cu, w=c.w)
    torch.cuda.synchronize()
    assert int(layer.dev_err[0]) == ssm.RSSM_DEVERR_SLOT
    left = torch.zeros(sum(lens), dtype=torch.bool, device="cuda")
    for b in (0, 2):
        left[c.starts[b]:c.starts[b + 1]] = True
    assert bool((o[left] == 7).all()) and torch.equal(o[~left], want[~left])
    kept = c.slots[[0, 2]].long()
    assert torch.equal(layer.state[kept], c.state0[kept])
    others = [b for b in range(len(lens)) if b not in (0, 2)]
    assert torch.equal(layer.state[c.slots[others].long()], state[c.slots[others].long()])


def test_a_captured_call_follows_its_rows_lengths():
    import ssm_linear_attention_gb300 as ssm
    cases = [Case(x, resume=0b1010) for x in ([32, 32, 32, 32], [1, 120, 0, 7], [100, 2, 25, 1])]
    assert len({sum(c.lens) for c in cases}) == 1
    first = cases[0]
    q, k, v, g, w = (x.clone() for x in (first.q.contiguous(), first.k.contiguous(), first.v.contiguous(), first.g, first.w))
    layer, cu, slots = first.layer(ssm), first.cu.clone(), first.slots.clone()
    layer.prompt(q, k, v, g, slots, cu_tokens=cu, w=w, resume=first.resume)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = layer.prompt(q, k, v, g, slots, cu_tokens=cu, w=w, resume=first.resume)
    for _ in range(2):
        for c in cases:
            for to, new in ((q, c.q), (k, c.k), (v, c.v), (g, c.g), (w, c.w), (cu, c.cu), (slots, c.slots), (layer.state, c.state0)):
                to.copy_(new)
            graph.replay()
            torch.cuda.synchronize()
            c.check(o, layer.state)
    assert int(layer.dev_err.sum()) == 0
