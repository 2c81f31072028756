"""The attention and norm entry points reject bad arguments on the host before any launch
(no GPU needed)."""
import ctypes

import pytest
import torch

import ssm_linear_attention_gb300 as ssm
from ssm_linear_attention_gb300 import _binding as B
from ssm_linear_attention_gb300 import build as rbuild

INV, UNS, CFG = B.RSSM_ERR_INVALID_ARG, B.RSSM_ERR_UNSUPPORTED, B.RSSM_ERR_CONFIG
FAKE = 0x10000  # aligned non-null address; never dereferenced (validation fails first)


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return ssm.lib()


def _dims(**kw):
    d = dict(batch=4, q_tokens=1, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16,
             num_pages=64, max_pages=8, num_slots=8, act_dtype=B.RSSM_BF16,
             cache_dtype=B.RSSM_E4M3, out_dtype=B.RSSM_BF16)
    d.update(kw)
    return B.AttnDims(**d)


def _cache(**kw):
    c = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, page_table=FAKE, slot_len=FAKE)
    c.update(kw)
    return B.AttnCache(**c)


def _decode(d, c=None, window=0, q=FAKE, q_stride=1024, ci=FAKE, ws=FAKE, wsb=1 << 40, o=FAKE,
            lse=None):
    c = _cache() if c is None else c
    return ssm.lib().rssm_attn_decode(ctypes.byref(d), ctypes.byref(c), 1, 1.0, window, q, q_stride,
                                      ci, ws, wsb, o, lse, None, None)


def _append(d, c=None, n=4, cu=None, k=FAKE, ks=256, v=FAKE, vs=256, ci=FAKE):
    c = _cache() if c is None else c
    return ssm.lib().rssm_attn_append(ctypes.byref(d), ctypes.byref(c), n, cu, k, ks, v, vs, ci,
                                      None, None)


def _read(d, c=None, n=4, cu=None, first=None, ci=FAKE, k=FAKE, v=FAKE):
    c = _cache() if c is None else c
    return ssm.lib().rssm_attn_read(ctypes.byref(d), ctypes.byref(c), n, cu, first, ci, k, v, None,
                                    None)


def _advance(d, c=None, cu=None, acc=None, ci=FAKE):
    c = _cache() if c is None else c
    return ssm.lib().rssm_attn_advance(ctypes.byref(d), ctypes.byref(c), cu, acc, ci, None, None)


BAD_DIMS = [
    (dict(batch=-1), INV), (dict(q_tokens=0), INV), (dict(num_q_heads=0), INV),
    (dict(num_kv_heads=0), INV), (dict(num_pages=0), INV), (dict(max_pages=0), INV),
    (dict(num_slots=0), INV), (dict(act_dtype=B.RSSM_E4M3), INV), (dict(act_dtype=9), INV),
    (dict(cache_dtype=B.RSSM_F32), INV), (dict(out_dtype=B.RSSM_E4M3), INV),
    (dict(num_q_heads=9), CFG), (dict(head_dim=96), UNS), (dict(page_size=8), UNS),
    (dict(page_size=48), UNS), (dict(page_size=512), UNS),
    (dict(max_pages=1 << 27), UNS),                    # positions past 2^30
    (dict(num_pages=1 << 27), UNS),                    # cache rows past 2^31
]


@pytest.mark.parametrize("bad,code", BAD_DIMS)
def test_dims(lib, bad, code):
    d = _dims(**bad)
    assert _decode(d) == code
    assert _append(d) == code
    assert _read(d) == code
    assert _advance(d) == code
    assert B.rssm_attn_workspace_size(d) == 0


def test_decode_arguments(lib):
    d = _dims()
    assert B.rssm_attn_workspace_size(d) > 0
    for kw in (dict(q=None), dict(q=FAKE + 2), dict(q_stride=1020), dict(q_stride=1016 - 8),
               dict(ci=None), dict(ws=None), dict(ws=FAKE + 8), dict(o=None), dict(o=FAKE + 8),
               dict(lse=FAKE + 4), dict(window=-1), dict(c=_cache(k=None)),
               dict(c=_cache(v=FAKE + 8)), dict(c=_cache(k_scale=None)),
               dict(c=_cache(page_table=None)), dict(c=_cache(slot_len=None)),
               dict(wsb=B.rssm_attn_workspace_size(d) - 1)):
        assert _decode(d, **kw) == INV, kw
    # 65 queries to a key head
    assert _decode(_dims(num_q_heads=26, q_tokens=5), q_stride=26 * 128) == UNS
    assert _decode(_dims(batch=0), q=None) == B.RSSM_OK


def test_append_read_and_advance_arguments(lib):
    d = _dims()
    for kw in (dict(n=-1), dict(n=5), dict(k=None), dict(v=FAKE + 8), dict(ks=248), dict(vs=260),
               dict(ci=None), dict(cu=FAKE + 4), dict(c=_cache(v_scale=None)), dict(c=_cache(k=None))):
        assert _append(d, **kw) == INV, kw
    assert _append(d, n=0, cu=FAKE, k=None) == B.RSSM_OK
    assert _append(_dims(batch=0), n=0, k=None) == B.RSSM_OK
    assert _append(_dims(batch=0), n=3, cu=FAKE) == INV
    for kw in (dict(n=-1), dict(n=5), dict(k=None), dict(v=FAKE + 8), dict(first=FAKE + 4),
               dict(ci=None), dict(c=_cache(page_table=None))):
        assert _read(d, **kw) == INV, kw
    assert _read(d, n=0, cu=FAKE, k=None) == B.RSSM_OK
    for kw in (dict(c=_cache(slot_len=None)), dict(ci=None), dict(acc=FAKE + 4), dict(cu=FAKE + 4)):
        assert _advance(d, **kw) == INV, kw
    assert _advance(_dims(batch=0), ci=None) == B.RSSM_OK


def test_norm_arguments(lib):
    def call(x=FAKE, res=None, w=FAKE, out=None, y=FAKE, scale=FAKE, **kw):
        n = dict(rows=4, cols=256, scale_group=0, act_dtype=B.RSSM_BF16, out_dtype=B.RSSM_E4M3)
        n.update(kw)
        return ssm.lib().rssm_add_rmsnorm(ctypes.byref(B.NormDims(**n)), x, res, w, 1e-5, out, y,
                                          scale, None)
    for kw, code in ((dict(rows=-1), INV), (dict(cols=0), INV), (dict(cols=32769), UNS),
                     (dict(scale_group=64), UNS), (dict(scale_group=128, cols=200), CFG),
                     (dict(act_dtype=B.RSSM_E4M3), INV), (dict(out_dtype=3), INV),
                     (dict(x=None), INV), (dict(x=FAKE + 8), INV), (dict(res=FAKE + 2), INV),
                     (dict(w=None), INV), (dict(out=FAKE + 4), INV), (dict(y=FAKE + 1), INV),
                     (dict(scale=None), INV), (dict(scale=FAKE + 4), INV)):
        assert call(**kw) == code, kw
    assert call(rows=0, x=None) == B.RSSM_OK


def test_runner_refusals(lib):
    """What the runners turn away before a call: lists and outputs of another type or size (the
    kernels would read or write past them), rows beyond the buffers, replaced buffers."""
    dec = ssm.PagedAttentionDecoder(8, 2, 64, 16, 4, 4, 2, 3, T=2, device="cpu")
    i32 = dict(dtype=torch.int32)
    ci, cu = torch.zeros(3, **i32), torch.zeros(4, **i32)
    bf = dict(dtype=torch.bfloat16)
    q, k = torch.zeros(3, 2, 8, 64, **bf), torch.zeros(3, 2, 2, 64, **bf)
    bad = [lambda: dec.decode(q, ci.long()), lambda: dec.decode(q, torch.zeros(6, **i32)[::2]),
           lambda: dec.decode(q[:2], ci), lambda: dec.decode(q.float(), ci),
           lambda: dec.decode(torch.zeros(4, 2, 8, 64, **bf), torch.zeros(4, **i32)),
           lambda: dec.decode(q, ci, o=torch.zeros(2, 2, 8, 64, **bf)),
           lambda: dec.decode(q, ci, o=torch.zeros(3, 2, 8, 64)),
           lambda: dec.decode(q, ci, lse=torch.zeros(3, 2, 7)),
           lambda: dec.append(k, k[:2], ci), lambda: dec.append(k, k.float(), ci),
           lambda: dec.append(k, k, ci, cu_tokens=cu[:3]), lambda: dec.append(k, k, ci, cu_tokens=cu.long()),
           lambda: dec.advance(ci, num_accepted=torch.zeros(2, **i32)),
           lambda: dec.advance(ci, cu_tokens=cu.long()),
           lambda: dec.read(ci, cu[:3], 5), lambda: dec.read(ci, cu, 5, first=cu[:2]),
           lambda: dec.read(ci, cu, 5, k=torch.zeros(4, 2, 64, **bf))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for name in ("page_table", "slot_len", "k_cache", "workspace", "dev_err", "T", "max_batch"):
        with pytest.raises(AttributeError):
            setattr(dec, name, getattr(dec, name))
    dec.window, dec.scale = 7, 0.5

    norm = ssm.AddRMSNorm(torch.ones(128), 1e-5, 2, out_dtype=torch.float8_e4m3fn, device="cpu")
    x, y = torch.zeros(3, 128, **bf), torch.zeros(3, 128, dtype=torch.float8_e4m3fn)
    bad = [lambda: norm(x), lambda: norm(x, y=y), lambda: norm(x[:2].float()), lambda: norm(x[:, :64]),
           lambda: norm(x[:2], y=y), lambda: norm(x[:2], y=y[:2].view(torch.uint8)),
           lambda: norm(x[:2], x), lambda: norm(x[:2], scale=torch.zeros(1, 1))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(AttributeError):
        norm.weight = torch.zeros(128)
    norm.eps = 1e-6


def test_debug_decode_arguments(lib):
    def call(wait_us, q=FAKE):
        return ssm.lib().rssm_debug_attn_decode(ctypes.byref(_dims()), ctypes.byref(_cache()), 1, 1.0, 0,
                                                q, 1024, FAKE, FAKE, 1 << 40, FAKE, None, -1, wait_us,
                                                None, None)
    assert call(0) == INV and call(2000001) == INV and call(1000, q=None) == INV


def _elsewhere(dec, norm, dev):
    """Calls of a runner of `dev` that each get one tensor of the CPU."""
    def there(*a, **kw):
        return torch.zeros(*a, device=dev, **kw)
    i32, bf = dict(dtype=torch.int32), dict(dtype=torch.bfloat16)
    ci, cu = there(3, **i32), there(4, **i32)
    q, k, kr = there(3, 2, 8, 64, **bf), there(3, 2, 2, 64, **bf), there(5, 2, 64, **bf)
    x = there(2, 128, **bf)
    return [lambda: dec.decode(q.cpu(), ci), lambda: dec.decode(q, ci.cpu()),
            lambda: dec.decode(q, ci, o=q.cpu()), lambda: dec.decode(q, ci, lse=torch.zeros(3, 2, 8)),
            lambda: dec.append(k.cpu(), k, ci), lambda: dec.append(k, k.cpu(), ci),
            lambda: dec.append(k, k, ci.cpu()), lambda: dec.append(k, k, ci, cu_tokens=cu.cpu()),
            lambda: dec.advance(ci.cpu()), lambda: dec.advance(ci, num_accepted=ci.cpu()),
            lambda: dec.advance(ci, cu_tokens=cu.cpu()), lambda: dec.read(ci.cpu(), cu, 5),
            lambda: dec.read(ci, cu.cpu(), 5), lambda: dec.read(ci, cu, 5, first=ci.cpu()),
            lambda: dec.read(ci, cu, 5, k=kr.cpu()), lambda: dec.read(ci, cu, 5, v=kr.cpu()),
            lambda: norm(x.cpu()), lambda: norm(x, x.cpu()), lambda: norm(x, x, residual_out=x.cpu()),
            lambda: norm(x, y=torch.zeros(2, 128, dtype=torch.float8_e4m3fn)),
            lambda: norm(x, scale=torch.zeros(2, 1))]


def _refuses(calls):
    for i, call in enumerate(calls):
        with pytest.raises(ValueError, match="device"):
            call()


def test_runner_refuses_tensors_of_another_device(lib):
    """Without a GPU: runners made on the CPU that stand for ones of GPU 0."""
    dec = ssm.PagedAttentionDecoder(8, 2, 64, 16, 4, 4, 2, 3, T=2, device="cpu")
    norm = ssm.AddRMSNorm(torch.ones(128), 1e-5, 2, out_dtype=torch.float8_e4m3fn, device="cpu")
    dec._index = norm._index = 0
    _refuses(_elsewhere(dec, norm, "cpu"))


@pytest.mark.gpu
def test_gpu_runner_refuses_tensors_of_the_cpu():
    dec = ssm.PagedAttentionDecoder(8, 2, 64, 16, 4, 4, 2, 3, T=2)
    norm = ssm.AddRMSNorm(torch.ones(128), 1e-5, 2, out_dtype=torch.float8_e4m3fn)
    _refuses(_elsewhere(dec, norm, "cuda"))
    ci = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    dec.step(*(torch.zeros(3, 2, h, 64, dtype=torch.bfloat16, device="cuda") for h in (8, 2, 2)), ci)
    norm(torch.zeros(2, 128, dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("kw,records", [
    (dict(num_q_heads=8, cache_dtype=B.RSSM_BF16), 2 + 8),                    # 8 groups a CTA
    (dict(num_q_heads=8), 2 + 16),
    (dict(num_q_heads=32), 2 + 8),                                            # two warps a group
    (dict(num_q_heads=16, q_tokens=4), 2), (dict(num_q_heads=128), 2),        # many queries: the CTAs'
    (dict(num_q_heads=32, cache_dtype=B.RSSM_BF16), 2),
    (dict(num_q_heads=128, act_dtype=B.RSSM_F32, out_dtype=B.RSSM_F32), 2 + 1),
])
def test_workspace_is_what_the_call_s_kernel_uses(lib, kw, records):
    d = _dims(**kw)
    M = d.q_tokens * d.num_q_heads // d.num_kv_heads
    size = B.rssm_attn_workspace_size(d)
    assert 0 < size <= 256 * (4 + records * M * d.head_dim * 4 + 2 * M * 8) + 256
    assert _decode(d, q_stride=d.num_q_heads * 128, wsb=size - 1) == INV


def test_workspace_of_dims_that_only_append(lib):
    """T of a prompt's length: rssm_attn_decode refuses it, no workspace is asked for."""
    d = _dims(q_tokens=4096, num_q_heads=16)
    assert B.rssm_attn_workspace_size(d) == 0 and _decode(d) == UNS
    dec = ssm.PagedAttentionDecoder(16, 2, 64, 16, 4, 4, 2, 1, T=4096, device="cpu")
    assert dec.workspace.numel() <= 16
