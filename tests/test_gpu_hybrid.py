"""The hybrid example: norms, Mamba2 layers and attention layers together, step by step in one
captured graph, against a float64 run of the same model.

With float32 activations, unquantised norms and a bf16 cache the only roundings beyond
float32 are the cached keys' and values', which the reference makes too. A layer's float32
sums of a few hundred terms carry some 1e-6 relative; a key that sits at a rounding midpoint
may fall to the other bf16 neighbour, 2^-8 of it, in one of many weights. The bar is 2e-3 of
the output's scale (the norm makes it 1)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    import ssm_linear_attention_gb300 as ssm
    ssm.lib()
    spec = importlib.util.spec_from_file_location("hybrid_decode", os.path.join(ROOT, "examples",
                                                                                "hybrid_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Reference:
    """The model in float64, one history per row."""

    def __init__(self, model, batch):
        self.m, self.state = model, [{} for _ in model.layers]
        self.batch = batch

    def norm(self, n, r):
        return r / (r.square().mean(-1, keepdim=True) + n.eps).sqrt() * n.weight.double()

    def step(self, x):
        residual = torch.zeros_like(x)
        for i, (n, l) in enumerate(zip(self.m.norms, self.m.layers)):
            residual = residual + x
            h = self.norm(n, residual)
            x = (self.mamba if hasattr(l, "w_in") else self.attention)(l, self.state[i], h)
        return self.norm(self.m.norms[-1], residual + x)

    def mamba(self, l, st, h):
        b, width = h.shape
        x, z, B, C, dt = (h @ l.w_in.double()).split([width, width, l.N, l.N, l.H], -1)
        x, z = x.view(b, l.H, l.P), z.view(b, l.H, l.P)
        dt = torch.nn.functional.softplus(dt + l.bias.double())
        s = st.setdefault("s", torch.zeros(b, l.H, l.P, l.N, dtype=torch.float64, device="cuda"))
        s.mul_((l.A.double() * dt).exp()[..., None, None])
        s.add_((dt[..., None] * x)[..., None] * B[:, None, None, :])
        y = (s * C[:, None, None, :]).sum(-1) + l.D.double()[:, None] * x
        return (y * z * torch.sigmoid(z)).reshape(b, width) @ l.w_out.double()

    def attention(self, l, st, h):
        b = h.shape[0]
        qkv = (h @ l.w_qkv.double()).view(b, -1, l.hd)
        q, k, v = qkv.split([l.HQ, l.HKV, l.HKV], 1)
        ks, vs = st.setdefault("k", []), st.setdefault("v", [])
        ks.append(k.bfloat16().double())
        vs.append(v.bfloat16().double())
        kk, vv = torch.stack(ks, 1), torch.stack(vs, 1)                  # [b, n, HKV, hd]
        s = torch.einsum("bhgd,bnhd->bhgn", q.view(b, l.HKV, -1, l.hd), kk) * l.hd ** -0.5
        return torch.einsum("bhgn,bnhd->bhgd", s.softmax(-1), vv).reshape(b, -1) @ l.w_out.double()


def test_hybrid_steps_match_float64(example):
    model = example.HybridModel(layers="mama", width=256, max_batch=5, max_tokens=64, act=torch.float32,
                                cache_dtype=torch.bfloat16, norm_dtype=torch.float32)
    slots = torch.tensor([7, 0, 3, 9, 4], dtype=torch.int32, device="cuda")
    model.capture(5)
    ref = Reference(model, 5)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    for t in range(40):
        x = torch.randn(5, 256, generator=g, device="cuda")
        out = model.replay(x, slots)
        want = ref.step(x.double())
        torch.cuda.synchronize()
        assert float((out.double() - want).abs().max()) <= 2e-3, t
    assert all(int(l.dec.dev_err.sum()) == 0 for l in model.layers)
    assert model.pages["slot_len"][slots.long()].tolist() == [40] * 5


def test_hybrid_with_eight_bit_cache_and_norms_runs_and_leaves_padding_alone(example):
    model = example.HybridModel(width=512, max_batch=4, max_tokens=32)
    slots = torch.tensor([5, -1, 2, -1], dtype=torch.int32, device="cuda")
    model.capture(4)
    for t in range(20):
        out = model.replay(torch.randn(4, 512, device="cuda").bfloat16(), slots)
    torch.cuda.synchronize()
    assert all(int(l.dec.dev_err.sum()) == 0 for l in model.layers)
    lens = model.pages["slot_len"].tolist()
    assert [n for i, n in enumerate(lens) if i in (5, 2)] == [20, 20] and sum(lens) == 40
    assert bool(torch.isfinite(out[[0, 2]].float()).all())


@pytest.mark.parametrize("device", [None, "cuda", 0, torch.device("cuda"), "cuda:0"])
def test_runners_take_the_device_however_it_is_named(example, device):
    import ssm_linear_attention_gb300 as ssm
    cache = torch.zeros(4, 2, 16, 64, device="cuda", dtype=torch.bfloat16)
    dec = ssm.PagedAttentionDecoder(8, 2, 64, 16, 4, 4, 2, 3, device=device, k_cache=cache,
                                    v_cache=cache.clone())
    assert dec.k_cache is cache and dec.device == cache.device
    dec.page_table.copy_(torch.arange(4)[:, None].expand(4, 2))
    ci = torch.tensor([2, 0, -1], dtype=torch.int32, device="cuda")
    x = torch.ones(3, 12, 64, device="cuda", dtype=torch.bfloat16)
    dec.step(x[:, :8].unsqueeze(1), x[:, 8:10], x[:, 10:], ci)
    norm = ssm.AddRMSNorm(torch.ones(64), 1e-5, 3, device=device)
    y, _ = norm(x[:, 0].contiguous())
    torch.cuda.synchronize()
    assert dec.slot_len.tolist() == [1, 0, 1, 0] and int(dec.dev_err.sum()) == 0
    assert bool((dec.o[:2] == 1).all()) and bool((y == 1).all())
