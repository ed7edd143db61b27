"""fp8_add_rmsnorm_quant (and its UE8M0 form): calls of the C entry points that
the Python binding does not make, and values at the ends of fp32's range."""

import ctypes

import pytest
import torch

from fp8_block_scaled_group128_b200 import binding as fb
from fp8_block_scaled_group128_b200 import synth

import moe_ref as ref
from gpu_util import require_gpu, to_dev

pytestmark = pytest.mark.gpu
FMT = ["fp32", "ue8m0"]
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert fb.get_device_error() == 0


def _fn(fmt):
    return fb.fp8_add_rmsnorm_quant if fmt == "fp32" else fb.fp8_add_rmsnorm_quant_ue8m0


def _inputs(M, K, seed):
    x = to_dev(synth.activations("llama", M, K, seed=seed))
    res = to_dev(synth.activations("deepseek", M, K, seed=seed + 1))
    w = to_dev(synth.uniform_bf16((K,), 0.25, 2.0, seed=seed))
    return x, res, w


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("K", [384, 4096])
@pytest.mark.parametrize("M", [5, 148, 149, 1037])
def test_residual_out_without_a_residual(M, K, fmt):
    """Through the C ABI: with a NULL residual, residual_out is a copy of x (or
    x itself), whatever the number of rows; the other outputs stay."""
    x, _, w = _inputs(M, K, seed=M + K)
    want = _fn(fmt)(x, weight=w, eps=EPS)
    call = getattr(fb.lib(), _fn(fmt).__name__)

    def run(xp, out):
        q, s, y = (torch.zeros_like(t) for t in want[:3])
        args = [ctypes.c_void_p(t if t is None else t.data_ptr()) for t in (xp, None, w, out, y, q, s)]
        status = call(*args[:3], EPS, M, K, *args[3:],
                      ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert status == 0
        for a, b in zip((q, s, y), want):
            assert torch.equal(a, b)

    out = torch.full((M + 1, K), 5.0, dtype=torch.bfloat16, device="cuda")
    run(x, out)
    assert torch.equal(out[:M], x) and bool((out[M] == 5).all())
    same = x.clone()
    run(same, same)
    assert torch.equal(same, x)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M", [6, 200])
def test_norm_beyond_fp32(M, fmt):
    """n beyond fp32 in one place, and a NaN weight in another: those groups'
    scales are NaN in both forms, y is infinite or NaN there, and the other
    groups and the rows without such an n stay."""
    x, res, w = _inputs(M, 640, seed=31)
    w[200], w[630] = 3.0e38, float("nan")
    x[:, 200] = 4 * (x.abs() + res.abs()).amax(dim=1)
    res[:, 200] = 0
    x[1, 200] = 0
    n = ref.norm_rows(x, res, w, EPS)[0]
    big = torch.arange(M, device="cuda") != 1
    assert bool((n[big, 200] > 4e38).all()) and float(n[1, 200]) == 0
    q, s, y, _ = _fn(fmt)(x, residual=res, weight=w, eps=EPS)
    nan = s.isnan() if fmt == "fp32" else s == 255
    hit = torch.zeros(M, 5, dtype=torch.bool, device="cuda")
    hit[:, 4] = True
    hit[big, 1] = True
    assert torch.equal(nan, hit)
    assert bool(y[big, 200].isinf().all()) and bool(y[:, 630].isnan().all())
    for rows, groups in ((big, [0, 2, 3]), (~big, [0, 1, 2, 3])):
        cols = torch.cat([torch.arange(128 * g, 128 * g + 128) for g in groups]).cuda()
        ref.check_norm(n[rows][:, cols], fmt, q[rows][:, cols].contiguous(),
                       s[rows][:, groups], y[rows][:, cols])


def _scaled_rows(copies, K, powers, seed):
    """Rows of both signs up to 2^p, for every p `copies` times, neighbours of
    different p; the first two elements are 2^p and (the smallest bf16) 2^-133."""
    g = torch.Generator().manual_seed(seed)
    v = torch.rand(copies, len(powers), K, generator=g, dtype=torch.float64) * 2 - 1
    v[..., 0] = 1.0
    v *= torch.exp2(torch.tensor(powers, dtype=torch.float64))[None, :, None]
    v[..., 1] = 2.0 ** -133
    return v.view(-1, K).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("eps,powers", [
    (0.0, (-133, -130, -126, -100, -76, -66, -50, 0, 50, 63, 64, 76, 100, 120, 126, 127, 127.99)),
    (2.0 ** -149, (-70, -50, 0, 64, 127)), (1e-6, (-80, -50, 0, 62, 65, 110, 127)),
    (1e20, (-20, 20, 60, 64, 127)), (3e38, (0, 50, 64, 120, 127))])
@pytest.mark.parametrize("copies,K", [(1, 128), (60, 128), (60, 384), (1, 1152), (60, 1152),
                                      (35, 4096), (1, 14336), (35, 14336), (1, 65536)])
def test_squares_beyond_fp32(copies, K, eps, powers, fmt):
    """Finite rows whose squares, or their sum, lie outside the range of fp32,
    next to ordinary ones: the norm is that of the formula."""
    x = _scaled_rows(copies, K, powers, seed=K + copies)
    w = to_dev(synth.uniform_bf16((K,), 0.25, 2.0, seed=K))
    n = ref.norm_rows(x, None, w, eps)[0]
    assert bool(n.isfinite().all()) and bool((n.abs().amax(dim=1) > 0).all())
    q, s, y, _ = _fn(fmt)(x, weight=w, eps=eps)
    ref.check_norm(n, fmt, q, s, y)
    # (x + res is exact here: r = x / 2)
    res = torch.where(x.abs() >= 2.0 ** -120, x * -0.5, torch.zeros_like(x))
    n, r_ref = ref.norm_rows(x, res, w, eps)
    q, s, y, r = _fn(fmt)(x, residual=res, weight=w, eps=eps)
    assert torch.equal(r, r_ref)
    ref.check_norm(n, fmt, q, s, y)


@pytest.mark.parametrize("M", [3, 301])
def test_zero_row_without_eps(M):
    """0 / sqrt(0): NaN, as the formula has it, in that row only."""
    x, _, w = _inputs(M, 768, seed=33)
    x[1] = 0
    q, s, y, _ = fb.fp8_add_rmsnorm_quant(x, weight=w, eps=0.0)
    assert bool(y[1].isnan().all()) and bool(s[1].isnan().all())
    keep = torch.arange(M, device="cuda") != 1
    ref.check_norm(ref.norm_rows(x, None, w, 0.0)[0][keep], "fp32", q[keep], s[keep], y[keep])


@pytest.mark.parametrize("M", [148, 20_000])
@pytest.mark.parametrize("w_one", [True, False])
def test_codes_are_those_of_the_quotient(M, w_one):
    """q is e4m3(n / s) for the fp32 n and the returned s, but where n / s is
    within two fp32 ulps of the middle between two codes. n is known to the bit:
    the rows are small whole numbers, whose squares add up exactly in any order,
    K is a power of two, and the inverse root and both products round once."""
    K = 1024
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randint(-100, 101, (M, K), generator=g, device="cuda").to(torch.bfloat16)
    w = to_dev(synth.uniform_bf16((K,), 0.25, 2.0, seed=41))
    if w_one:
        w = torch.ones_like(w)
    q, s, y, _ = fb.fp8_add_rmsnorm_quant(x, weight=w, eps=0.0)
    mean = (x.double() ** 2).sum(dim=1, keepdim=True) / K
    rstd = (1.0 / mean.sqrt()).float()
    n = (x.float() * rstd) * w.float()
    assert torch.equal(y, n.to(torch.bfloat16))
    amax = n.abs().view(M, K // 128, 128).amax(dim=2)
    assert torch.equal(s, (amax.double() / 448).float())
    v = n.double() / s.double().repeat_interleave(128, dim=1)
    got, want = ref.e4m3_values(q), ref.e4m3_round(v)
    off = got != want
    middle = (got[off] + want[off]) / 2
    ulp = torch.exp2(torch.floor(torch.log2(v[off].abs())) - 23)
    assert bool(((got[off] - want[off]).abs() <= ref.e4m3_step(torch.maximum(got[off].abs(), want[off].abs()))).all())
    assert bool(((v[off] - middle).abs() <= 2 * ulp).all())
