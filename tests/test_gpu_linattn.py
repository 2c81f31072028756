"""rssm_linattn_prompt and rssm_linattn_step against the recurrence in float64.

Bounds. Let A be the same recurrence on absolute values (|q|, |k|, |v|, |w|, |S_0|): no sum of its terms
in any order exceeds it. Each way of computing is off by at most a fraction of A:
  bf16 activations, chunks of 64: products of bf16 values are exact in float32. A weight, a state value or
    a decayed value enters a product as two bf16 parts: off by at most 2^-17 of itself; a term passes two
    such places at most. The sum of a chunk's products takes 8 + 16 additions that the tensor core cuts: 24 *
    2^-23. A state takes two roundings a chunk, 2^-24 each, and 2^-18 in total over 64 chunks; a chunk's
    decay 2^-x is exp2 (2^-22) of an x that is rounded by 2^-24 of itself (2^-17.5 where x = 90; what is
    decayed further is below 2^-90). In total 2 * 2^-17 + 2^-18.4 + 2^-18 + 2^-22 + 2^-17.5 < 2^-15.3.
  float32 activations and steps, one token after another: a term that is d tokens old was multiplied by d
    decays (expf: 2^-23 each, and a rounding), added N times: (3 T + N) 2^-24 at most.
An output rounded to bf16 is off by 2^-8 of the value at most (half a spacing), a bf16 state alike."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    import ssm_linear_attention_gb300 as ssm
    ssm.lib()


def recurrence(q, k, v, g, w, s0, scale):
    """One row's tokens: q, k [n, G, N], v [n, H, P], g [n, H] -> o [n, H, P], S [H, P, N], float64."""
    n, H = v.shape[0], v.shape[1]
    many = H // q.shape[1]
    q, k, v = q.double().repeat_interleave(many, 1), k.double().repeat_interleave(many, 1), v.double()
    f = g.double().exp().expand(n, H)
    if w is not None:
        v = v * w.double()[..., None]
    s, o = s0.double().clone(), torch.empty_like(v)
    for t in range(n):
        s = s * f[t][:, None, None] + v[t][:, :, None] * k[t][:, None, :]
        o[t] = (s * q[t][:, None, :]).sum(-1) * scale
    return o, s


def fraction(act, T, N):
    return 2.0 ** -15.3 if act == BF else (3 * T + N) * 2.0 ** -24


class Case:
    def __init__(self, lens, H=4, G=2, N=128, P=128, act=BF, state=F32, decay="token", w=True, resume=None, seed=0, rate=1.0,
                 out=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + sum(lens) + H * N)
        self.lens, self.H, self.G, self.N, self.P, self.act, self.sd = lens, H, G, N, P, act, state
        self.out = out or act
        n, b = sum(lens), len(lens)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        # slices of fused projections
        self.qk = rnd(n, 2 * G + 1, N).to(act)
        self.q, self.k = self.qk[:, :G], self.qk[:, G:2 * G]
        self.v = rnd(n, H + 1, P).to(act)[:, :H]
        per = -rate * torch.rand(H, generator=g, device="cuda") ** 3
        self.g = per if decay == "head" else per * (0.3 + 1.4 * torch.rand(n, H, generator=g, device="cuda"))
        self.w = rnd(n, H) if w else None
        self.slots = torch.randperm(b + 2, generator=g, device="cuda")[:b].to(torch.int32)
        self.state0 = rnd(b + 2, H, P, N).to(state)
        self.resume = None if resume is None else torch.tensor([bool(resume >> i & 1) for i in range(b)], device="cuda")
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        self.starts, self.cu = cu, torch.tensor(cu, dtype=torch.int32, device="cuda")
        self.scale = N ** -0.5

    def layer(self, ssm):
        return ssm.LinearAttention(self.H, self.G, self.N, self.P, len(self.lens) + 2, len(self.lens), max_tokens=max(sum(self.lens), 1),
                                   state_dtype=self.sd, act_dtype=self.act, out_dtype=self.out, state=self.state0.clone())

    def run(self, ssm, layer=None):
        layer = layer or self.layer(ssm)
        o = layer.prompt(self.q, self.k, self.v, self.g, self.slots, cu_tokens=self.cu, w=self.w, resume=self.resume)
        torch.cuda.synchronize()
        assert int(layer.dev_err.sum()) == 0
        return o, layer.state

    def check(self, o, state):
        untouched = torch.ones(len(self.lens) + 2, dtype=torch.bool)
        for b, n in enumerate(self.lens):
            i, j, s = self.starts[b], self.starts[b + 1], int(self.slots[b])
            if n == 0:
                continue
            untouched[s] = False
            s0 = self.state0[s] if self.resume is not None and bool(self.resume[b]) else torch.zeros_like(self.state0[s])
            g = self.g if self.g.dim() == 1 else self.g[i:j]
            w = None if self.w is None else self.w[i:j]
            args = (self.q[i:j], self.k[i:j], self.v[i:j])
            ro, rs = recurrence(*args, g, w, s0, self.scale)
            ao, as_ = recurrence(*(x.abs() for x in args), g, None if w is None else w.abs(), s0.abs(), self.scale)
            f = fraction(self.act, n, self.N)
            for name, got, ref, size, dt in (("o", o[i:j], ro, ao, self.out), ("state", state[s], rs, as_, self.sd)):
                bound = f * size + (2.0 ** -8 * ref.abs() if dt == BF else 0) + 1e-37
                off = ((got.double() - ref).abs() / bound).max()
                assert bool(off <= 1), "row %d of %d tokens: %s off by %.2f of its bound" % (b, n, name, float(off))
        assert torch.equal(state[untouched.to(state.device)], self.state0[untouched.to(state.device)])


LENS = [[1], [64], [65], [63, 1, 0, 2], [128, 127, 129], [200], [0, 0, 5], [300, 17, 64, 1]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("act", [BF, F32])
def test_prompt_lengths(lens, act):
    import ssm_linear_attention_gb300 as ssm
    c = Case(lens, act=act, resume=0b0101)
    c.check(*c.run(ssm))


@pytest.mark.parametrize("N,P", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("H,G", [(1, 1), (3, 3), (6, 2), (8, 2), (10, 2), (16, 1)])
@pytest.mark.parametrize("act", [BF, F32])
def test_prompt_head_layouts(N, P, H, G, act):
    import ssm_linear_attention_gb300 as ssm
    c = Case([70, 33, 129], H=H, G=G, N=N, P=P, act=act, resume=0b010)
    c.check(*c.run(ssm))


@pytest.mark.parametrize("act", [BF, F32])
@pytest.mark.parametrize("state", [BF, F32])
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("w", [False, True])
def test_prompt_types_and_factors(act, state, decay, w):
    import ssm_linear_attention_gb300 as ssm
    c = Case([90, 130], act=act, state=state, decay=decay, w=w, resume=0b10, P=64, out=F32 if state == BF else None)
    c.check(*c.run(ssm))


@pytest.mark.parametrize("H,G,P,T", [(1, 1, 128, 5000), (2, 1, 64, 3001), (4, 4, 128, 2500), (16, 1, 64, 1100)])
def test_long_rows(H, G, P, T):
    """Rows that several parts of the GPU share, beside short ones (4096 tokens take 64 chunks)."""
    import ssm_linear_attention_gb300 as ssm
    c = Case([17, T, 0, T // 3, 64], H=H, G=G, P=P, resume=0b01010, rate=0.02)
    o, state = c.run(ssm)
    c.check(o, state)
    o2, state2 = c.run(ssm)   # the same bits again
    assert torch.equal(o, o2) and torch.equal(state, state2)


def test_many_rows():
    import ssm_linear_attention_gb300 as ssm
    lens = [(7 * i) % 5 for i in range(700)]
    c = Case(lens, H=2, G=1, N=64, P=64, resume=0xAAAAAAAAAAAA)
    c.check(*c.run(ssm))


@pytest.mark.parametrize("act", [BF, F32])
def test_resets_and_strong_decays(act):
    import ssm_linear_attention_gb300 as ssm
    c = Case([150, 70], act=act, resume=0b11)
    c.g[5] = -float("inf")
    c.g[64] = -float("inf")
    c.g[100, 1] = -float("inf")
    c.g[101:110] = -20.0
    c.g[160] = -300.0
    c.g[170] = -1e30
    c.check(*c.run(ssm))


@pytest.mark.parametrize("act", [BF, F32])
@pytest.mark.parametrize("what", ["v", "k", "w", "g", "q"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_behind_its_token(act, what, bad):
    import ssm_linear_attention_gb300 as ssm
    lens, at = [40, 130, 70], 40 + 69
    c = Case(lens, act=act, G=2, H=4, P=64)
    clean, clean_state = (x.clone() for x in c.run(ssm))
    if what == "g":
        c.g[at, 2] = float("nan")
    elif what == "w":
        c.w[at, 2] = bad
    elif what == "v":
        c.v[at, 2, 7] = bad
    elif what == "k":
        c.k[at, 1, 9] = bad
    else:
        c.q[at, 1, 9] = bad
    o, state = c.run(ssm)
    fine = torch.ones_like(o, dtype=torch.bool)
    heads = slice(2, 4) if what in "kq" else slice(2, 3)
    values = slice(7, 8) if what == "v" else slice(None)
    fine[at:at + 1 if what == "q" else 170, heads, values] = False
    assert torch.equal(o[fine], clean[fine])
    assert not bool(torch.isfinite(o[~fine].float()).any())
    same = torch.ones_like(state, dtype=torch.bool)
    if what != "q":
        s = int(c.slots[1])
        same[s, heads, values, 9 if what == "k" else slice(None)] = False
        assert not bool(torch.isfinite(state[~same].float()).any())
    assert torch.equal(state[same], clean_state[same])


@pytest.mark.parametrize("act", [BF, F32])
def test_fresh_rows_ignore_what_their_slot_holds_and_rows_around_them(act):
    import ssm_linear_attention_gb300 as ssm
    c = Case([10, 70, 3], act=act)
    layer = c.layer(ssm)
    layer.state.fill_(float("nan"))
    # tokens of the row behind are NaN: none of them reaches the row before
    c.q[80:], c.k[80:], c.v[80:] = float("nan"), float("nan"), float("nan")
    o, state = c.run(ssm, layer)
    for b in (0, 1):
        i, j = c.starts[b], c.starts[b + 1]
        assert bool(torch.isfinite(o[i:j].float()).all()) and bool(torch.isfinite(state[int(c.slots[b])].float()).all())
    c.lens = c.lens[:2]
    c.state0 = torch.cat([c.state0[:0]] + [state[i:i + 1] for i in range(5)])
    for b in (0, 1):
        i, j, s = c.starts[b], c.starts[b + 1], int(c.slots[b])
        ro, rs = recurrence(c.q[i:j], c.k[i:j], c.v[i:j], c.g[i:j], c.w[i:j], torch.zeros_like(state[s]), c.scale)
        assert float((o[i:j].double() - ro).norm() / ro.norm()) < 2.0 ** -8
        assert float((state[s].double() - rs).norm() / rs.norm()) < 2.0 ** -15


@pytest.mark.parametrize("act", [BF, F32])
def test_padding_tails_and_bad_lists(act):
    import ssm_linear_attention_gb300 as ssm
    n, H = 100, 4
    c = Case([n], H=H, act=act)
    layer = ssm.LinearAttention(H, 2, 128, 128, 6, 5, max_tokens=n, act_dtype=act, out_dtype=act)
    layer.state.fill_(3)
    layer.o.fill_(5)
    slots = torch.tensor([4, -1, 6, 0, 2], dtype=torch.int32, device="cuda")
    cu = torch.tensor([3, 20, 30, 40, 40, 90], dtype=torch.int32, device="cuda")
    o = layer.prompt(c.q, c.k, c.v, c.g, slots, cu_tokens=cu, w=c.w)
    torch.cuda.synchronize()
    assert int(layer.dev_err[0]) == ssm.RSSM_DEVERR_SLOT
    for i, j, s in ((3, 20, 4), (40, 90, 2)):
        ro, rs = recurrence(c.q[i:j], c.k[i:j], c.v[i:j], c.g[i:j], c.w[i:j], torch.zeros(H, 128, 128, device="cuda"), c.scale)
        assert float((o[i:j].double() - ro).norm() / ro.norm()) < 2.0 ** -8
        assert float((layer.state[s].double() - rs).norm() / rs.norm()) < 2.0 ** -15
    assert bool((o[:3] == 5).all()) and bool((o[20:40] == 5).all()) and bool((o[90:] == 5).all())
    assert bool((layer.state[[0, 1, 3, 5]] == 3).all())
    # lists that are not lists: flagged, and nothing outside of the buffers
    layer.o.fill_(5)
    for bad in ([0, 10, 1 << 30, -5, 40, 101], [50, 40, 30, 20, 10, 0], [-1, 200, 0, 7, 5, 100]):
        layer.dev_err.zero_()
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        layer.prompt(c.q, c.k, c.v, c.g, torch.arange(5, dtype=torch.int32, device="cuda"), cu_tokens=cu, w=c.w)
        torch.cuda.synchronize()
        assert int(layer.dev_err[0]) == ssm.RSSM_DEVERR_CURSOR
    assert bool((layer.state[5] == 3).all())


@pytest.mark.parametrize("act", [BF, F32])
@pytest.mark.parametrize("state", [BF, F32])
@pytest.mark.parametrize("N,P,H,G", [(64, 64, 3, 3), (64, 128, 4, 2), (128, 64, 8, 1), (128, 128, 6, 2)])
def test_steps(act, state, N, P, H, G):
    import ssm_linear_attention_gb300 as ssm
    b, T = 5, 6
    c = Case([T] * b, H=H, G=G, N=N, P=P, act=act, state=state)
    layer = c.layer(ssm)
    outs = []
    slots = torch.cat([c.slots[:3], torch.tensor([-1], dtype=torch.int32, device="cuda"), c.slots[4:]])
    layer.o.fill_(9)
    want_state = [c.state0[int(s)].double() for s in c.slots]
    bound_state = [s.abs() for s in want_state]
    for t in range(T):
        at = torch.arange(b, device="cuda") * T + t
        q, k, v = c.qk[at][:, :G], c.qk[at][:, G:2 * G], c.v[at]
        o = layer.step(q, k, v, c.g[at], slots, w=c.w[at])
        torch.cuda.synchronize()
        for r in (0, 1, 2, 4):
            # from the state that the step found, whatever its type
            ro, rs = recurrence(q[r:r + 1], k[r:r + 1], v[r:r + 1], c.g[at][r:r + 1], c.w[at][r:r + 1], want_state[r], c.scale)
            ao, as_ = recurrence(q[r:r + 1].abs(), k[r:r + 1].abs(), v[r:r + 1].abs(), c.g[at][r:r + 1], c.w[at][r:r + 1].abs(),
                                 want_state[r].abs(), c.scale)
            f = fraction(F32, 1, N)
            got = layer.state[int(c.slots[r])].double()
            assert bool(((o[r:r + 1].double() - ro).abs() <= f * ao + (2.0 ** -8 * ro.abs() if act == BF else 0) + 1e-37).all())
            assert bool(((got - rs).abs() <= f * as_ + (2.0 ** -8 * rs.abs() if state == BF else 0) + 1e-37).all())
            want_state[r] = got
        assert bool((o[3] == 9).all())
    assert torch.equal(layer.state[int(c.slots[3])], c.state0[int(c.slots[3])])
    assert int(layer.dev_err.sum()) == 0
    layer.step(q, k, v, c.g[at], torch.tensor([0, 1, 2, 3, b + 2], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert int(layer.dev_err[0]) == ssm.RSSM_DEVERR_SLOT


def test_prompt_in_parts_and_steps_agree_with_the_whole():
    import ssm_linear_attention_gb300 as ssm
    c = Case([200, 150], H=4, G=4, P=64)
    whole, state = (x.clone() for x in c.run(ssm))
    layer = c.layer(ssm)
    parts, cut = [], (90, 64)
    for lo, hi in ((0, 1), (1, 2)):
        at = torch.cat([torch.arange(c.starts[b] + (cut[b] if lo else 0), c.starts[b] + (c.lens[b] - 3 if lo else cut[b])) for b in (0, 1)]).cuda()
        n0 = c.lens[0] - 3 - cut[0] if lo else cut[0]
        cu = torch.tensor([0, n0, len(at)], dtype=torch.int32, device="cuda")
        o = layer.prompt(c.q[at], c.k[at], c.v[at], c.g[at], c.slots, cu_tokens=cu, w=c.w[at], resume=bool(lo))
        torch.cuda.synchronize()
        parts.append((at, o.clone()))
    for t in (3, 2, 1):
        at = torch.tensor([c.starts[b + 1] - t for b in (0, 1)]).cuda()
        o = layer.step(c.q[at], c.k[at], c.v[at], c.g[at], c.slots, w=c.w[at])
        torch.cuda.synchronize()
        parts.append((at, o.clone()))
    c.check(whole, state)
    o = torch.empty_like(whole)
    for at, x in parts:
        o[at] = x
    c.check(o, layer.state)


def test_mamba2_prompt_then_replay_decode():
    """A Mamba2 layer's prompt through the same pool that its decode steps go on from."""
    import numpy as np

    import ssm_linear_attention_gb300 as ssm
    H, P, N, G, L, b = 8, 64, 128, 2, 4, 3
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    A = -torch.rand(H, generator=g, device="cuda") - 0.2
    D = torch.randn(H, generator=g, device="cuda")
    dec = ssm.Mamba2ReplayDecoder(H, P, N, G, L, 6, b, A, D, None, dt_softplus=False, state_dtype=F32, act_dtype=F32, out_dtype=F32)
    layer = ssm.LinearAttention(H, G, N, P, 6, b, max_tokens=200, scale=1.0, act_dtype=F32, out_dtype=F32, state=dec.state)
    lens, steps = [70, 1, 40], 6
    slots = torch.tensor([5, 0, 3], dtype=torch.int32, device="cuda")
    n = sum(lens)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, B_, C, z = rnd(b, 200, H, P), rnd(b, 200, G, N), rnd(b, 200, G, N), rnd(b, 200, H, P)
    dt = 0.05 + 0.1 * torch.rand(b, 200, H, generator=g, device="cuda")
    pick = lambda t: torch.cat([t[r, :lens[r]] for r in range(b)])  # noqa: E731
    cu = torch.tensor([0, 70, 71, 111], dtype=torch.int32, device="cuda")
    y = layer.prompt(pick(C), pick(B_), pick(x), pick(dt) * A, slots, cu_tokens=cu, w=pick(dt))
    torch.cuda.synchronize()
    states = []
    for r in range(b):
        i, j = int(cu[r]), int(cu[r + 1])
        ro, rs = recurrence(C[r, :lens[r]], B_[r, :lens[r]], x[r, :lens[r]], dt[r, :lens[r]].double() * A.double(), dt[r, :lens[r]],
                            torch.zeros(H, P, N, device="cuda"), 1.0)
        assert float((y[i:j].double() - ro).abs().max()) < 1e-4 * max(1.0, float(ro.abs().max()))
        states.append(rs)
    rows = torch.arange(b, device="cuda")
    for t in range(steps):
        at = torch.tensor(lens, device="cuda") + t
        xs, bs, cs, zs, ds = (u[rows, at].contiguous() for u in (x, B_, C, z, dt))
        out = dec.step(xs, ds, bs, cs, zs, slots)
        torch.cuda.synchronize()
        for r in range(b):
            ro, states[r] = recurrence(cs[r:r + 1], bs[r:r + 1], xs[r:r + 1], ds[r:r + 1].double() * A.double(), ds[r:r + 1], states[r], 1.0)
            want = (ro[0] + D.double()[:, None] * xs[r].double()) * zs[r].double() * torch.sigmoid(zs[r].double())
            assert float((out[r].double() - want).abs().max()) < 1e-4 * max(1.0, float(want.abs().max()))
    assert int(dec.dev_err.sum()) == 0 and n == 111


@pytest.mark.parametrize("act", [BF, F32])
def test_captured_calls_follow_lengths_and_inputs(act):
    import ssm_linear_attention_gb300 as ssm
    c = Case([300, 100, 48], H=4, G=2, act=act, resume=0b010)
    layer = c.layer(ssm)
    q, k, v, g, w = c.q.contiguous(), c.k.contiguous(), c.v.contiguous(), c.g.clone(), c.w.clone()
    cu, resume = c.cu.clone(), c.resume.to(torch.uint8)
    call = lambda: layer.prompt(q, k, v, g, c.slots, cu_tokens=cu, w=w, resume=resume)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = call()
    for lens, mask in (([300, 100, 48], 0b010), ([0, 448, 0], 0b111), ([1, 1, 446], 0b100)):
        n = Case(lens, H=4, G=2, act=act, resume=mask, seed=mask)
        q.copy_(n.q), k.copy_(n.k), v.copy_(n.v), g.copy_(n.g), w.copy_(n.w), cu.copy_(n.cu), resume.copy_(n.resume)
        n.slots = c.slots
        layer.state.copy_(n.state0)
        graph.replay()
        torch.cuda.synchronize()
        n.check(o, layer.state)
    assert int(layer.dev_err.sum()) == 0


def test_calls_on_two_streams():
    import ssm_linear_attention_gb300 as ssm
    cases = [Case([500, 90], seed=s, H=8, G=4) for s in (1, 2)]
    layers = [c.layer(ssm) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        outs = []
        for c, l, s in zip(cases, layers, streams):
            with torch.cuda.stream(s):
                outs.append(l.prompt(c.q, c.k, c.v, c.g, c.slots, cu_tokens=c.cu, w=c.w))
    torch.cuda.synchronize()
    for c, l, o in zip(cases, layers, outs):
        c.check(o, l.state)


def test_rotated_layers_together():
    """A rotary linear-attention layer and its single tokens as a model runs them: rotate, prompt, then
    rotate and step, against the same in float64."""
    import ssm_linear_attention_gb300 as ssm
    H, D, b, steps = 4, 64, 3, 4
    lens = [33, 70, 1]
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    slots = torch.tensor([1, 4, 2], dtype=torch.int32, device="cuda")
    slot_len = torch.zeros(6, dtype=torch.int32, device="cuda")
    rot = ssm.Rotary(H, H, D, rot_dim=32, act_dtype=F32)
    layer = ssm.LinearAttention(H, H, D, D, 6, b, max_tokens=128, act_dtype=F32, out_dtype=F32)
    decay = -2.0 ** (-3.0 - torch.arange(H, device="cuda"))
    total = [n + steps for n in lens]
    x = [torch.randn(t, 3 * H, D, generator=g, device="cuda") for t in total]
    f = torch.tensor(rot.frequencies, dtype=torch.float64, device="cuda")

    def turned(y):
        y = y.double().clone()
        a = torch.arange(len(y), dtype=torch.float64, device="cuda")[:, None] * f
        c, s, u, w = a.cos()[:, None], a.sin()[:, None], y[..., :16].clone(), y[..., 16:32].clone()
        y[..., :16], y[..., 16:32] = u * c - w * s, w * c + u * s
        return y
    want = [recurrence(turned(y[:, :H]), turned(y[:, H:2 * H]), y[:, 2 * H:], decay, None, torch.zeros(H, D, D, device="cuda"),
                       D ** -0.5)[0] for y in x]
    fused = torch.cat([y[:n] for y, n in zip(x, lens)])
    cu = torch.tensor([0, 33, 103, 104], dtype=torch.int32, device="cuda")
    q, k = rot(fused[:, :H], fused[:, H:2 * H], cache_indices=slots, slot_len=slot_len, cu_tokens=cu)
    o = layer.prompt(q, k, fused[:, 2 * H:], decay, slots, cu_tokens=cu)
    slot_len[slots.long()] += (cu[1:] - cu[:-1])
    torch.cuda.synchronize()
    for r in range(b):
        assert float((o[int(cu[r]):int(cu[r + 1])].double() - want[r][:lens[r]]).abs().max()) < 2e-4
    for t in range(steps):
        token = torch.stack([y[n + t] for y, n in zip(x, lens)])
        q, k = rot(token[:, :H], token[:, H:2 * H], cache_indices=slots, slot_len=slot_len)
        o = layer.step(q, k, token[:, 2 * H:], decay, slots)
        slot_len[slots.long()] += 1
        torch.cuda.synchronize()
        for r in range(b):
            assert float((o[r].double() - want[r][lens[r] + t]).abs().max()) < 2e-4
    assert int(rot.dev_err.sum()) == 0 and int(layer.dev_err.sum()) == 0


def test_runner_refusals():
    import ssm_linear_attention_gb300 as ssm
    c = Case([10, 6], H=4, G=2, P=64)
    layer = c.layer(ssm)
    ok = dict(q=c.q, k=c.k, v=c.v, g=c.g, cache_indices=c.slots, cu_tokens=c.cu, w=c.w)
    for kw in (dict(q=c.q.float()), dict(q=c.q[:15]), dict(k=c.k[..., :64]), dict(v=c.v[:, :3]), dict(g=c.g.double()),
               dict(g=c.g[:15]), dict(g=c.g[0, :3]), dict(w=c.w[0]), dict(w=c.w.t()), dict(cache_indices=c.slots.long()),
               dict(cache_indices=c.slots.repeat(2)), dict(cu_tokens=c.cu[:2]), dict(cu_tokens=c.cu.long()),
               dict(q=c.q.cpu()), dict(resume=torch.ones(3, device="cuda", dtype=torch.bool)),
               dict(resume=torch.ones(2, device="cuda")), dict(o=torch.empty(15, 4, 64, device="cuda", dtype=BF)),
               dict(o=torch.empty(16, 4, 64, device="cuda")), dict(q=c.qk[:, ::2][:, :2])):
        with pytest.raises((ValueError, IndexError)):
            layer.prompt(**dict(ok, **kw))
    with pytest.raises(ValueError):
        layer.prompt(**dict(ok, cu_tokens=None, q=c.q[:15], k=c.k[:15], v=c.v[:15], g=c.g[:15], w=c.w[:15]))
    with pytest.raises(ValueError):   # more tokens than the runner is made for
        two = lambda t: torch.cat([t, t])  # noqa: E731
        layer.prompt(two(c.q), two(c.k), two(c.v), two(c.g), c.slots, cu_tokens=c.cu, w=two(c.w))
    with pytest.raises(ValueError):
        layer.step(c.q, c.k, c.v, c.g, c.slots)
    with pytest.raises(AttributeError):
        layer.state = None
    with pytest.raises(ValueError):
        ssm.LinearAttention(4, 2, 128, 64, 4, 2, state=torch.zeros(4, 4, 64, 64, device="cuda"))
    assert torch.equal(layer.state, c.state0)
