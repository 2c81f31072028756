"""rssm_add_rmsnorm against float64.

Tolerances: the sum of squares of n terms runs in float32 over a tree of at most 256
sequential terms, so the inverse root carries at most 2^-24 * 256 / 2 relative in the
worst case and a few 2^-24 on average; with the two products |y - ref| <= 2^-17 |ref| for
a float32 output, plus half a spacing for bf16 (8 significant bits: at most 2^-8 of the value). An 8-bit output must be the
nearest e4m3 value of ref / scale up to 2^-16 of it; scales agree to 2^-16."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    import ssm_linear_attention_gb300 as ssm
    ssm.lib()


def e4m3_table():
    b = torch.arange(256, dtype=torch.uint8).view(FP8).double().numpy()
    return np.unique(b[np.isfinite(b)])


def reference(x, res, w):
    r = x.double() + (0 if res is None else res.double())
    return r, r / (r.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()


def compare(y, scale, ref, group):
    ref = ref.cpu().numpy()
    if y.dtype != FP8:
        tol = 2.0 ** -17 + (2.0 ** -8 if y.dtype == torch.bfloat16 else 0)
        assert np.all(np.abs(y.double().cpu().numpy() - ref) <= tol * np.abs(ref) + 1e-37)
        return
    rows, cols = ref.shape
    rg = ref.reshape(rows, -1, group or cols)
    amax = np.maximum(np.abs(rg).max(-1), 2.0 ** -100)
    sc = scale.double().cpu().numpy()
    assert sc.shape == amax.shape
    assert np.all(np.abs(sc - amax / 448) <= 2.0 ** -16 * amax / 448)
    want = (rg * (448 / amax)[..., None]).reshape(rows, cols)
    grid = e4m3_table()
    i = np.clip(np.searchsorted(grid, want), 1, len(grid) - 1)
    half = np.minimum(np.abs(want - grid[i - 1]), np.abs(want - grid[i]))
    got = y.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= half + 2.0 ** -15 * np.abs(want) + 1e-12)


SHAPES = [(1, 1), (3, 7), (1, 8), (5, 24), (2, 127), (7, 128), (4, 1000), (3, 1001), (1, 4096),
          (33, 2560), (300, 640), (5, 8192), (2, 12288), (1, 16384 + 8), (2, 32768), (3, 32767),
          (1000, 256), (70, 5120)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32, FP8])
def test_norm_matches_float64(rows, cols, act, out):
    import ssm_linear_attention_gb300 as ssm
    g = torch.Generator(device="cuda")
    g.manual_seed(rows * 31 + cols)
    x = torch.randn(rows, cols, generator=g, device="cuda").to(act)
    res = (4 * torch.randn(rows, cols, generator=g, device="cuda")).to(act)
    w = 1 + 0.3 * torch.randn(cols, generator=g, device="cuda")
    for group in ([0, 128] if out == FP8 and cols % 128 == 0 else [0]):
        norm = ssm.AddRMSNorm(w, EPS, rows, act_dtype=act, out_dtype=out, scale_group=group)
        r, ref = reference(x, res, w)
        into = torch.empty_like(res)
        y, scale = norm(x, res, residual_out=into)
        torch.cuda.synchronize()
        assert torch.equal(into, (x.float() + res.float()).to(act))
        compare(y, scale, ref, group)
        # the same without a residual, and in place
        y, scale = norm(x)
        torch.cuda.synchronize()
        compare(y, scale, reference(x, None, w)[1], group)
        inplace = res.clone()
        y1, s1 = norm(x, inplace)
        y1 = y1.clone()
        torch.cuda.synchronize()
        assert torch.equal(inplace, into)
        y2, _ = norm(x, res, residual_out=torch.empty_like(res))
        torch.cuda.synchronize()
        assert torch.equal(y1.view(torch.uint8), y2.view(torch.uint8))


@pytest.mark.parametrize("out", [torch.bfloat16, FP8])
@pytest.mark.parametrize("cols", [256, 250])
def test_zero_tiny_huge_and_nan_rows(out, cols):
    import ssm_linear_attention_gb300 as ssm
    x = torch.zeros(6, cols, device="cuda")
    x[1] = 1e-30
    x[2] = 1e15 * torch.arange(1, cols + 1, device="cuda")
    x[3, 5] = float("nan")
    x[4, 9] = float("inf")
    x[5] = torch.linspace(-3, 3, cols, device="cuda")
    w = torch.ones(cols, device="cuda")
    norm = ssm.AddRMSNorm(w, EPS, 6, act_dtype=torch.float32, out_dtype=out)
    y, scale = norm(x)
    torch.cuda.synchronize()
    val = y.double() * (1 if scale is None else scale.double())
    ref = reference(x, None, w)[1]
    assert bool((val[0] == 0).all())
    assert bool(torch.isnan(val[3]).all())
    # an infinity makes the mean infinite: 0 elsewhere and NaN in its place, the whole row in 8 bits
    assert bool(torch.isnan(val[4]).any())
    if out == FP8:
        assert bool(torch.isnan(val[4]).all())
    for i in (1, 2, 5):
        step = 2.0 ** -8 * ref[i].abs() if out != FP8 else \
            torch.maximum(2.0 ** -4 * ref[i].abs(), ref[i].abs().max() / 448 * 2.0 ** -9)
        assert bool(((val[i] - ref[i]).abs() <= step * 1.01 + 1e-37).all())


def test_wrapper_refusals():
    import ssm_linear_attention_gb300 as ssm
    norm = ssm.AddRMSNorm(torch.ones(64), EPS, 4)
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    for args in ((x.float(),), (x, x[:2]), (x, x.float()), (torch.zeros(5, 64, device="cuda",
                 dtype=torch.bfloat16),), (x.t().contiguous().t(),)):
        with pytest.raises(ValueError):
            norm(*args)
