"""fp8_add_rmsnorm_quant's kernel for many rows: what lies around the call's
rows, other streams, captured graphs and its place in a chain of launches. Row
lengths with several rows to a block (the last block in part) and with one."""

import pytest
import torch

from fp8_block_scaled_group128_b200 import binding as fb
from fp8_block_scaled_group128_b200 import synth

import moe_ref as ref
from gpu_util import require_gpu, to_dev

pytestmark = pytest.mark.gpu
FMT = ["fp32", "ue8m0"]
SHAPES = [(301, 128), (299, 256), (150, 384), (151, 1024), (149, 4096), (163, 51200)]


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
@pytest.mark.parametrize("with_res", [True, False])
@pytest.mark.parametrize("M,K", SHAPES)
def test_rows_around_the_call_are_left_alone(M, K, with_res, fmt):
    if with_res and K * 4 > 100 * 1024:
        K //= 2   # the longest rows that the kernel takes with a residual
    x, res, w = _inputs(M + 2, K, seed=M)
    q = torch.full((M + 2, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((M + 2, K // 128), 7, dtype=torch.float32 if fmt == "fp32" else torch.uint8, device="cuda")
    y = torch.full((M + 2, K), 3.0, dtype=torch.bfloat16, device="cuda")
    ro = torch.full((M + 2, K), 5.0, dtype=torch.bfloat16, device="cuda")
    keep = x.clone(), res.clone(), w.clone()
    # NaN around the rows read: none of it may reach them
    x[0], x[-1], res[0], res[-1] = (float("nan"),) * 4
    extra = dict(residual=res[1:-1], residual_out=ro[1:-1]) if with_res else {}
    if fmt == "fp32":
        extra["s"] = s[1:-1]
    else:
        extra["s8"] = s[1:-1]
    _fn(fmt)(x[1:-1], weight=w, q=q[1:-1], y=y[1:-1], **extra)
    for t, v in ((q, 0x55), (s, 7), (y, 3.0), (ro, 5.0)):
        assert bool((t[0] == v).all()) and bool((t[-1] == v).all())
    for t, k in zip((x, res, w), keep):
        assert torch.equal(t[1:-1] if t.dim() == 2 else t, k[1:-1] if t.dim() == 2 else k)
    n, r = ref.norm_rows(x[1:-1], res[1:-1] if with_res else None, w, 1e-6)
    ref.check_norm(n, fmt, q[1:-1], s[1:-1], y[1:-1])
    assert not with_res or torch.equal(ro[1:-1], r)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,K", SHAPES[:5])
def test_streams(M, K, fmt):
    """Two streams at once, several calls each."""
    a, b = _inputs(M, K, seed=K), _inputs(M + 40, K, seed=K + 5)
    want = [_fn(fmt)(x, residual=r, weight=w) for x, r, w in (a, b)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[_fn(fmt)(x, residual=r, weight=w, stream=st) for (x, r, w), st in ((a, s1), (b, s2))]
           for _ in range(8)]
    torch.cuda.synchronize()
    for pair in got:
        for outs, right in zip(pair, want):
            for t, v in zip(outs, right):
                assert torch.equal(t, v)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,K", SHAPES[:5])
def test_captured_chain(M, K, fmt):
    """A residual stream through four norms, each reading what the one before it
    wrote, the residual updated in place; captured, and replayed on new inputs."""
    x, res, w = _inputs(M, K, seed=K + 9)

    def chain(x, res):
        outs = []
        for _ in range(4):
            q, s, x, res = _fn(fmt)(x, residual=res, weight=w, residual_out=res)
            outs += [q, s, x]
        return outs + [res]

    torch.cuda.synchronize()
    xs, rs = x.clone(), res.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(xs, rs)
    for seed in (61, 62):
        x2, r2, _ = _inputs(M, K, seed=seed)
        xs.copy_(x2)
        rs.copy_(r2)
        graph.replay()
        torch.cuda.synchronize()
        xc, rc = x2, r2
        for i in range(4):
            n, rc = ref.norm_rows(xc, rc, w, 1e-6)
            ref.check_norm(n, fmt, *got[3 * i:3 * i + 3])
            xc = got[3 * i + 2]
        assert torch.equal(got[-1], rc)
        for t, v in zip(got, chain(x2, r2.clone())):
            assert torch.equal(t, v)
