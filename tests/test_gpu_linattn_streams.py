"""LinearAttention's calls on a stream of the caller's, while the current stream is busy."""
import pytest
import torch

from .test_gpu_linattn import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    import ssm_linear_attention_gb300 as ssm
    ssm.lib()


@pytest.mark.parametrize("lens", [[7, 20, 3], [70, 200, 30], [3000]])
def test_every_row_resumes_on_a_stream_of_its_own(lens):
    import ssm_linear_attention_gb300 as ssm
    c = Case(lens, resume=(1 << len(lens)) - 1)
    want, state = (x.clone() for x in c.run(ssm))
    layer = c.layer(ssm)
    side = torch.cuda.Stream()
    old = torch.zeros(len(lens), device="cuda", dtype=torch.uint8)
    torch.cuda.synchronize()
    del old
    torch.cuda._sleep(20_000_000)  # (some 10 ms)
    o = layer.prompt(c.q, c.k, c.v, c.g, c.slots, cu_tokens=c.cu, w=c.w, resume=True, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(layer.state, state)


def test_a_new_layer_is_ready_on_any_stream():
    import ssm_linear_attention_gb300 as ssm
    c = Case([900, 1300])
    want, state = (x.clone() for x in c.run(ssm))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        held = torch.full((64 << 20,), 255, device="cuda", dtype=torch.uint8)
        del held  # (the layer's buffers come from memory that is not zero)
        state0 = c.state0.clone()
        torch.cuda._sleep(20_000_000)
        layer = ssm.LinearAttention(c.H, c.G, c.N, c.P, 4, 2, max_tokens=2200, state=state0)
        o = layer.prompt(c.q, c.k, c.v, c.g, c.slots, cu_tokens=c.cu, w=c.w, stream=side.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(layer.state, state)
