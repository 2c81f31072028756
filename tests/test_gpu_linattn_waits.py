"""The bounded waits of the chunked linear attention: a wait that runs out sets its bit, the kernel returns and the
context stays usable (a barrier is armed for 16 bytes more than its copies deliver; the copies themselves land)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    import ssm_linear_attention_gb300 as ssm
    ssm.lib()


@pytest.mark.parametrize("P,H", [(128, 2), (64, 4), (64, 3)])
@pytest.mark.parametrize("stall", [0, 1, 3])
def test_a_wait_that_runs_out_ends_the_kernel(P, H, stall):
    import ssm_linear_attention_gb300 as ssm
    from ssm_linear_attention_gb300 import _binding as B
    g = torch.Generator(device="cuda")
    g.manual_seed(P + H + stall)
    n, N, G = 600, 128, 1
    layer = ssm.LinearAttention(H, G, N, P, 4, 2, max_tokens=n)
    q, k = (torch.randn(n, G, N, generator=g, device="cuda").bfloat16() for _ in range(2))
    v = torch.randn(n, H, P, generator=g, device="cuda").bfloat16()
    decay = -torch.rand(n, H, generator=g, device="cuda")
    slots = torch.tensor([1, 3], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 300, n], dtype=torch.int32, device="cuda")
    want = layer.prompt(q, k, v, decay, slots, cu_tokens=cu).clone()
    want_state = layer.state.clone()
    layer.o.fill_(7)
    layer.state.fill_(7)
    inputs = B.linattn_inputs(q, k, v, decay, scale=layer.scale, q_stride=G * N, k_stride=G * N, v_stride=H * P, g_stride=H)

    def call(stall_chunk):
        B.rssm_debug_linattn_prompt(layer.dims(2), inputs, n, cu, None, layer.state, slots, layer.workspace, layer.ws_bytes,
                                    layer.o, stall_chunk, 20000, layer.dev_err)
        torch.cuda.synchronize()
    call(stall)
    assert int(layer.dev_err[0]) == ssm.RSSM_DEVERR_TIMEOUT
    # the first CTA's unit is not finished: its state is as it was
    assert bool((layer.state[1, 0] == 7).all())
    # without the stall, after the counters are zero again, everything is as before
    layer.dev_err.zero_()
    layer.workspace.zero_()
    call(-1)
    assert int(layer.dev_err[0]) == 0
    assert torch.equal(layer.o[:n], want) and torch.equal(layer.state[slots.long()], want_state[slots.long()])


def test_refusals():
    import ssm_linear_attention_gb300 as ssm
    from ssm_linear_attention_gb300 import _binding as B
    layer = ssm.LinearAttention(2, 1, 64, 64, 2, 1, max_tokens=64)
    x = torch.zeros(64, 1, 64, device="cuda").bfloat16()
    v = torch.zeros(64, 2, 64, device="cuda").bfloat16()
    inputs = B.linattn_inputs(x, x, v, torch.zeros(2, device="cuda"))
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")
    for wait in (0, 2000001):
        with pytest.raises(ssm.RSSMError):
            B.rssm_debug_linattn_prompt(layer.dims(1), inputs, 64, None, None, layer.state, slots, layer.workspace, layer.ws_bytes,
                                        layer.o, -1, wait)
    for ws, size in ((None, layer.ws_bytes), (layer.workspace, layer.ws_bytes - 1)):
        with pytest.raises(ssm.RSSMError):
            B.rssm_linattn_prompt(layer.dims(1), inputs, 64, None, None, layer.state, slots, ws, size, layer.o)
