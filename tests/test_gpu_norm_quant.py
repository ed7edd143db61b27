"""fp8_add_rmsnorm_quant (and its UE8M0 form) against the 64-bit norm: the
residual bit for bit, y within half a bf16 step, the scales within the fp32
error of the norm, every code within half an E4M3 step."""

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


def _fn(fmt):
    return fb.fp8_add_rmsnorm_quant if fmt == "fp32" else fb.fp8_add_rmsnorm_quant_ue8m0


def _inputs(M, K, seed):
    x = to_dev(synth.activations("llama", M, K, seed=seed))
    res = to_dev(synth.activations("deepseek", M, K, seed=seed + 1))
    w = to_dev(synth.uniform_bf16((K,), 0.25, 2.0, seed=seed))
    return x, res, w


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,K", [(1, 128), (3, 256), (257, 256), (7, 1152), (9, 1408), (130, 2048),
                                 (1, 4096), (64, 7168), (2, 8320), (5, 14336), (3, 16512),
                                 (2, 40960), (2, 65536), (301, 4096), (1031, 896)])
@pytest.mark.parametrize("with_res", [True, False])
def test_values(M, K, fmt, with_res):
    x, res, w = _inputs(M, K, seed=M + K)
    res = res if with_res else None
    q, s, y, r = _fn(fmt)(x, residual=res, weight=w, eps=EPS)
    n, r_ref = ref.norm_rows(x, res, w, EPS)
    if with_res:
        assert torch.equal(r, r_ref)
    else:
        assert r is None
    ref.check_norm(n, fmt, q, s, y)
    q2, s2, y2, _ = _fn(fmt)(x, residual=res, weight=w, eps=EPS, want_y=False)
    assert y2 is None and torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("fmt", FMT)
def test_no_weight_and_eps(fmt):
    x, res, _ = _inputs(33, 640, seed=4)
    q, s, y, _ = _fn(fmt)(x, residual=res, eps=0.5)
    ref.check_norm(ref.norm_rows(x, res, None, 0.5)[0], fmt, q, s, y)
    ones = torch.ones(640, dtype=torch.bfloat16, device="cuda")
    q2, s2, y2, _ = _fn(fmt)(x, residual=res, weight=ones, eps=0.5)
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(y, y2)


@pytest.mark.parametrize("fmt", FMT)
def test_zero_rows_and_groups(fmt):
    """A row of zeros and a group of zeros: codes are zeros of the element's
    sign, the scale is 0 (UE8M0: the smallest code); nothing is NaN."""
    x, _, w = _inputs(4, 512, seed=5)
    x[1] = 0
    x[2, 128:256] = 0
    x[3, 256:384] = -0.0
    q, s, y, _ = _fn(fmt)(x, weight=w, eps=EPS)
    ref.check_norm(ref.norm_rows(x, None, w, EPS)[0], fmt, q, s, y)
    assert bool((q[1] == 0).all()) and bool((s[1] == 0).all()) and bool((y[1] == 0).all())
    assert bool((q[2, 128:256] == 0).all()) and bool((q[3, 256:384] == 0x80).all())


@pytest.mark.parametrize("fmt", FMT)
def test_small_and_large_values(fmt):
    """Rows scaled by powers of two from 2^-60 (eps decides) to 2^40."""
    x, _, w = _inputs(6, 256, seed=6)
    for i, p in enumerate((-60, -20, -8, 0, 20, 40)):
        x[i] *= 2.0 ** p
    q, s, y, _ = _fn(fmt)(x, weight=w, eps=EPS)
    ref.check_norm(ref.norm_rows(x, None, w, EPS)[0], fmt, q, s, y)


@pytest.mark.parametrize("fmt", FMT)
def test_nan_and_inf_stay_in_their_row(fmt):
    x, res, w = _inputs(5, 384, seed=7)
    x[1, 200] = float("nan")
    x[3, 10] = float("inf")
    q, s, y, r = _fn(fmt)(x, residual=res, weight=w, eps=EPS)
    keep = [0, 2, 4]
    n = ref.norm_rows(x, res, w, EPS)[0]
    ref.check_norm(n[keep], fmt, q[keep], s[keep], y[keep])
    assert bool(y[1].isnan().all()) and bool(((q[1] & 0x7F) == 0x7F).all())
    # the infinity's own element is inf * 0, the others are finite * 0
    assert bool(y[3, 10].isnan()) and bool((y[3, 128:] == 0).all())
    if fmt == "fp32":
        assert bool(s[1].isnan().all()) and bool(s[3, 0].isnan()) and bool((s[3, 1:] == 0).all())


@pytest.mark.parametrize("alias", ["residual", "x"])
def test_residual_in_place(alias):
    x, res, w = _inputs(40, 1280, seed=8)
    want = fb.fp8_add_rmsnorm_quant(x, residual=res, weight=w)
    xc, rc = x.clone(), res.clone()
    q, s, y, r = fb.fp8_add_rmsnorm_quant(xc, residual=rc, weight=w,
                                          residual_out=rc if alias == "residual" else xc)
    assert r.data_ptr() == (rc if alias == "residual" else xc).data_ptr()
    for a, b in zip((q, s, y, r), want):
        assert torch.equal(a, b)


def test_rows_around_the_call_are_left_alone():
    M, K = 5, 768
    x, res, w = _inputs(M + 2, K, seed=9)
    q = torch.full((M + 2, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((M + 2, K // 128), 7.0, device="cuda")
    y = torch.full((M + 2, K), 3.0, dtype=torch.bfloat16, device="cuda")
    ro = torch.full((M + 2, K), 5.0, dtype=torch.bfloat16, device="cuda")
    fb.fp8_add_rmsnorm_quant(x[1:-1], residual=res[1:-1], weight=w, q=q[1:-1], s=s[1:-1],
                             y=y[1:-1], residual_out=ro[1:-1])
    for t, v in ((q, 0x55), (s, 7.0), (y, 3.0), (ro, 5.0)):
        assert bool((t[0] == v).all()) and bool((t[-1] == v).all())


def test_stream_and_graph():
    """On a side stream, and captured and replayed on new inputs."""
    x, res, w = _inputs(16, 2048, seed=10)
    want = fb.fp8_add_rmsnorm_quant(x, residual=res, weight=w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fb.fp8_add_rmsnorm_quant(x, residual=res, weight=w, stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    xs = x.clone()
    with torch.cuda.graph(graph):
        got = fb.fp8_add_rmsnorm_quant(xs, residual=res, weight=w)
    x2 = to_dev(synth.activations("llama", 16, 2048, seed=77))
    xs.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, fb.fp8_add_rmsnorm_quant(x2, residual=res, weight=w)):
        assert torch.equal(a, b)


def test_feeds_the_linear():
    """The codes go straight into fp8_block_gemm: the same product as from
    the quantizer's codes of y, within both quantizations' half steps."""
    x, res, w = _inputs(24, 1024, seed=11)
    wt = to_dev(synth.weights("llama", 256, 1024, seed=11))
    qw, sw = fb.fp8_quant_weight_block128(wt)
    q, s, y, _ = fb.fp8_add_rmsnorm_quant(x, residual=res, weight=w)
    out = fb.fp8_block_gemm(q, s, qw, sw)
    n = ref.norm_rows(x, res, w, EPS)[0]
    wd = ref.dequant_blocks(qw, sw)
    a = ref.dequant_rows(q, s)
    exact = a @ wd.T
    tol = (a.abs() @ wd.abs().T) * ((1024 // 128 + 256) * ref.U32) + exact.abs() * ref.U16
    assert bool(((out.double() - exact).abs() <= tol).all())
    half = torch.maximum(n.abs() * 2.0 ** -4, s.double().repeat_interleave(128, 1) * 2.0 ** -10)
    assert bool(((exact - n @ wd.T).abs() <= (half * 1.01) @ wd.abs().T).all())


def test_refusals():
    x, res, w = _inputs(4, 512, seed=12)
    with pytest.raises(ValueError):
        fb.fp8_add_rmsnorm_quant(x[:, ::2])
    with pytest.raises(ValueError):
        fb.fp8_add_rmsnorm_quant(x.t())
    with pytest.raises(ValueError):
        fb.fp8_add_rmsnorm_quant(x[0])
    with pytest.raises(ValueError):
        fb.fp8_add_rmsnorm_quant(x, residual=res[:2])
    with pytest.raises(TypeError):
        fb.fp8_add_rmsnorm_quant(x, weight=w.float())
    with pytest.raises(TypeError):
        fb.fp8_add_rmsnorm_quant(x.half())
    with pytest.raises(ValueError):
        fb.fp8_add_rmsnorm_quant(x, residual_out=res)
    with pytest.raises(fb.Fp8bsError):
        fb.fp8_add_rmsnorm_quant(x[:, :100].contiguous())
    with pytest.raises(fb.Fp8bsError):
        fb.fp8_add_rmsnorm_quant(x, eps=-1.0)
    empty = fb.fp8_add_rmsnorm_quant(x[:0], residual=res[:0], weight=w)
    assert empty[0].shape == (0, 512)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("with_res", [True, False])
@pytest.mark.parametrize("M,K", [(149, 128), (150, 256), (701, 384), (1000, 1920), (149, 14336),
                                 (200, 25600), (149, 28672), (160, 51200)])
def test_many_rows(M, K, with_res, fmt):
    """The kernel for many rows: short rows that share a block (the last one
    in part), rows up to its shared memory and beyond."""
    x, res, w = _inputs(M, K, seed=3 * M + K)
    res = res if with_res else None
    q, s, y, r = _fn(fmt)(x, residual=res, weight=w, eps=EPS)
    n, r_ref = ref.norm_rows(x, res, w, EPS)
    assert r is None if res is None else torch.equal(r, r_ref)
    ref.check_norm(n, fmt, q, s, y)
    q2, s2, y2, _ = _fn(fmt)(x, residual=res, weight=w, eps=EPS, want_y=False)
    assert y2 is None and torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("fmt", FMT)
def test_many_rows_with_unusual_values(fmt):
    """Zeros, NaN, infinities and weights of 2^-110 (scales whose reciprocal is
    not used) among ordinary rows; the addition in place."""
    x, res, w = _inputs(300, 640, seed=20)
    w[128:256] = 2.0 ** -110
    res[7] = 0
    x[7] = 0
    x[11, 300:] = 0
    res[11, 300:] = -0.0
    x[20, 5] = float("nan")
    x[30, 639] = float("inf")
    ro = res.clone()
    q, s, y, r = _fn(fmt)(x, residual=ro, weight=w, eps=EPS, residual_out=ro)
    n, r_ref = ref.norm_rows(x, res, w, EPS)
    keep = torch.tensor([i for i in range(300) if i not in (20, 30)], device="cuda")
    assert r.data_ptr() == ro.data_ptr() and torch.equal(r[keep], r_ref[keep])
    ref.check_norm(n[keep], fmt, q[keep], s[keep], y[keep])
    assert bool((q[7] == 0).all()) and bool((q[11, 384:] == 0).all())
    assert bool(y[20].isnan().all()) and bool(((q[20] & 0x7F) == 0x7F).all())
    assert bool(y[30, 639].isnan()) and bool((y[30, :512] == 0).all())
    few = _fn(fmt)(x[:40], residual=res[:40], weight=w, eps=EPS)
    assert torch.equal(few[3][:20], r[:20])


def test_many_rows_timeout_is_reported():
    """A wait limit of one cycle: the error is recorded, the next call is right."""
    x, res, w = _inputs(400, 4096, seed=21)
    want = fb.fp8_add_rmsnorm_quant(x, residual=res, weight=w)
    fb.get_device_error()
    try:
        fb.set_wait_limit(1)
        fb.fp8_add_rmsnorm_quant(x, residual=res, weight=w)
        assert fb.get_device_error() == 6
    finally:
        fb.set_wait_limit(0)
    for a, b in zip(fb.fp8_add_rmsnorm_quant(x, residual=res, weight=w), want):
        assert torch.equal(a, b)
    assert fb.get_device_error() == 0


def test_offsets_beyond_32_bits():
    """2.3e9 elements: the last rows as in a call of their own."""
    M, K, n = 280_000, 8192, 200
    base, _, w = _inputs(1000, K, seed=22)
    x = base.repeat(M // 1000, 1)
    x[-n:] = _inputs(n, K, seed=23)[0]
    q, s, y, _ = fb.fp8_add_rmsnorm_quant(x, weight=w)
    tail = fb.fp8_add_rmsnorm_quant(x[-n:], weight=w)
    for a, b in zip((q, s, y), tail):
        assert torch.equal(a[-n:], b)
    assert torch.equal(q[:1000], q[1000:2000])
