"""The linear-attention and rotary entry points reject bad arguments on the host before any
launch, and the frequencies of long contexts (no GPU needed)."""
import ctypes
import math

import pytest

import ssm_linear_attention_gb300 as ssm
from ssm_linear_attention_gb300 import _binding as B
from ssm_linear_attention_gb300 import build as rbuild

INV, UNS, CFG, OK = B.RSSM_ERR_INVALID_ARG, B.RSSM_ERR_UNSUPPORTED, B.RSSM_ERR_CONFIG, B.RSSM_OK
FAKE = 0x10000  # aligned non-null address; never dereferenced (validation fails first)


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return ssm.lib()


def _dims(**kw):
    d = dict(batch=4, num_heads=8, num_k_heads=2, key_dim=128, value_dim=64, num_slots=8,
             state_dtype=B.RSSM_F32, act_dtype=B.RSSM_BF16, out_dtype=B.RSSM_BF16)
    d.update(kw)
    return B.LinattnDims(**d)


def _inputs(**kw):
    i = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, w=None, q_stride=256, k_stride=256, v_stride=512, g_stride=8,
             w_stride=0, scale=1.0)
    i.update(kw)
    return B.LinattnInputs(**i)


def _prompt(d, i=None, n=100, cu=FAKE, resume=None, state=FAKE, ci=FAKE, ws=FAKE, wsb=1 << 40, o=FAKE):
    return ssm.lib().rssm_linattn_prompt(ctypes.byref(d), ctypes.byref(i or _inputs()), n, cu, resume, state, ci, ws,
                                         wsb, o, None, None)


def _step(d, i=None, state=FAKE, ci=FAKE, o=FAKE):
    return ssm.lib().rssm_linattn_step(ctypes.byref(d), ctypes.byref(i or _inputs()), state, ci, o, None, None)


@pytest.mark.parametrize("bad,code", [
    (dict(batch=-1), INV), (dict(num_heads=0), INV), (dict(num_k_heads=0), INV), (dict(num_slots=0), INV),
    (dict(state_dtype=B.RSSM_E4M3), INV), (dict(act_dtype=5), INV), (dict(out_dtype=B.RSSM_E4M3), INV),
    (dict(num_heads=9), CFG), (dict(key_dim=96), UNS), (dict(value_dim=32), UNS), (dict(value_dim=256), UNS),
    (dict(num_heads=16384), UNS), (dict(batch=1 << 27), UNS)])
def test_linear_dims(lib, bad, code):
    assert _prompt(_dims(**bad)) == code
    assert _step(_dims(**bad)) == code
    assert B.rssm_linattn_workspace_size(_dims(**bad), 1000) == 0


BAD_INPUTS = [dict(q=None), dict(k=FAKE + 8), dict(v=None), dict(g=None), dict(g=FAKE + 4), dict(w=FAKE + 4, w_stride=8),
              dict(q_stride=248), dict(q_stride=260), dict(k_stride=0), dict(v_stride=504), dict(g_stride=7),
              dict(g_stride=-8), dict(w=FAKE, w_stride=0), dict(w=FAKE, w_stride=4), dict(q_stride=1 << 40)]


@pytest.mark.parametrize("bad", BAD_INPUTS)
def test_linear_inputs(lib, bad):
    assert _prompt(_dims(), _inputs(**bad)) == INV
    assert _step(_dims(), _inputs(**bad)) == INV


def test_linear_arguments(lib):
    d = _dims()
    for kw in (dict(n=-1), dict(state=None), dict(state=FAKE + 8), dict(ci=None), dict(o=None), dict(cu=FAKE + 4),
               dict(resume=FAKE + 1)):
        assert _prompt(d, **kw) == INV, kw
    for kw in (dict(state=None), dict(ci=FAKE + 4), dict(o=FAKE + 8)):
        assert _step(d, **kw) == INV, kw
    assert _prompt(d, n=101, cu=None) == CFG          # 101 tokens of 4 rows
    assert _prompt(d, n=0, state=None) == OK
    assert _prompt(_dims(batch=0), n=0, ci=None) == OK
    assert _step(_dims(batch=0), ci=None) == OK


def test_linear_null_structs(lib):
    assert ssm.lib().rssm_linattn_prompt(None, None, 1, None, None, None, None, None, 0, None, None, None) == INV
    assert ssm.lib().rssm_linattn_step(ctypes.byref(_dims()), None, FAKE, FAKE, FAKE, None, None) == INV


def _rope(pos=FAKE, ci=None, sl=None, cu=None, freq=FAKE, q=FAKE, qs=1024, k=FAKE, ks=256, qo=FAKE, qos=1024, ko=FAKE,
          kos=256, **kw):
    d = dict(batch=2, n_tokens=10, num_q_heads=8, num_k_heads=2, head_dim=128, rot_dim=64, interleaved=0, num_slots=4,
             act_dtype=B.RSSM_BF16)
    d.update(kw)
    return ssm.lib().rssm_rope(ctypes.byref(B.RopeDims(**d)), freq, 1.0, pos, ci, sl, cu, q, qs, k, ks, qo, qos, ko, kos,
                               None, None)


@pytest.mark.parametrize("bad,code", [
    (dict(n_tokens=-1), INV), (dict(num_q_heads=-1), INV), (dict(num_q_heads=0), INV), (dict(num_k_heads=-1), INV),
    (dict(head_dim=0), INV), (dict(act_dtype=B.RSSM_E4M3), INV), (dict(head_dim=100), UNS), (dict(head_dim=520), UNS),
    (dict(n_tokens=1 << 28), UNS), (dict(rot_dim=0), CFG), (dict(rot_dim=63), CFG), (dict(rot_dim=130), CFG),
    (dict(freq=None), INV), (dict(q=None), INV), (dict(qo=FAKE + 8), INV), (dict(k=None), INV), (dict(ko=None), INV),
    (dict(qs=1016), INV), (dict(qs=1028), INV), (dict(kos=248), INV), (dict(qos=1032), INV),  # in place, other stride
    (dict(pos=FAKE + 4), INV), (dict(pos=None), INV), (dict(pos=None, ci=FAKE), INV),
    (dict(pos=None, ci=FAKE, sl=FAKE, num_slots=0), INV), (dict(pos=None, ci=FAKE, sl=FAKE, batch=3), CFG),
    (dict(pos=None, ci=FAKE, sl=FAKE, cu=FAKE + 4), INV), (dict(pos=None, batch=-1), INV)])
def test_rope_arguments(lib, bad, code):
    assert _rope(**bad) == code


def test_rope_of_nothing(lib):
    assert _rope(n_tokens=0, q=None) == OK
    assert _rope(pos=None, batch=0, n_tokens=0) == OK


def test_frequencies():
    f, m = ssm.rotary_frequencies(8, 10000.0)
    assert m == 1.0 and all(math.isclose(x, 10.0 ** -i, rel_tol=1e-12) for i, x in enumerate(f))
    g, _ = ssm.rotary_frequencies(8, 10000.0, {"type": "linear", "factor": 4})
    assert all(math.isclose(x, y / 4, rel_tol=1e-12) for x, y in zip(g, f))
    g, _ = ssm.rotary_frequencies(128, 10000.0, {"type": "base", "factor": 8.0})
    plain, _ = ssm.rotary_frequencies(128, 10000.0)
    assert g[0] == plain[0] and math.isclose(g[-1], plain[-1] / 8, rel_tol=1e-9)
    g, m = ssm.rotary_frequencies(128, 10000.0, {"type": "yarn", "factor": 8.0, "original": 4096})
    turns = [4096 * x / (2 * math.pi) for x in plain]
    assert math.isclose(m, 0.1 * math.log(8) + 1)
    for x, y, t in zip(g, plain, turns):
        if t > 40:
            assert x == y
        if t < 0.8:
            assert math.isclose(x, y / 8, rel_tol=1e-12)
        assert y / 8 * (1 - 1e-12) <= x <= y
    g, m = ssm.rotary_frequencies(128, 10000.0, {"type": "bands", "factor": 8.0, "original": 4096})
    assert m == 1.0
    for x, y, t in zip(g, plain, turns):
        assert math.isclose(x, y if t >= 4 else y / 8 if t <= 1 else y / 8 + (y - y / 8) * (t - 1) / 3, rel_tol=1e-9)
    for bad in ({"type": "other"}, {"type": "yarn", "factor": 2}, {"factor": 0}, {"type": "linear", "factr": 2},
                {"type": "bands", "factor": 2, "original": 4096, "fast": 1}):
        with pytest.raises(ValueError):
            ssm.rotary_frequencies(128, 10000.0, bad)
    with pytest.raises(ValueError):
        ssm.rotary_frequencies(7)
