"""The mixture-of-experts block as a decoder layer runs it: norm and
quantization of the residual stream, the router's product, the choice of the
experts, the expert MLP, and the next layer's norm with the MLP's output as the
addition; eagerly and as one captured graph."""

import pytest
import torch

from fp8_block_scaled_group128_b200 import binding as fb
from fp8_block_scaled_group128_b200 import synth

import moe_ref as ref
from gpu_util import require_gpu, to_dev
from test_gpu_moe_mlp import _experts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert fb.get_device_error() == 0


def _block(x, res, wn, wr, bias, experts, fmt):
    norm, moe = ((fb.fp8_add_rmsnorm_quant, fb.fp8_moe_mlp) if fmt == "fp32" else
                 (fb.fp8_add_rmsnorm_quant_ue8m0, fb.fp8_moe_mlp_ue8m0))
    qa, sa, h, r = norm(x, residual=res, weight=wn)
    logits = (h @ wr.t()).float()
    ids, w = fb.moe_route_topk(logits, 4, scoring="sigmoid", bias=bias, n_group=4, topk_group=2,
                               scale=2.5)
    y = moe(qa, sa, ids, w, *experts)
    nxt = norm(y, residual=r, weight=wn)
    return qa, sa, h, r, logits, ids, w, y, nxt


def _inputs(M, K, I, E, fmt, seed):
    x = to_dev(synth.activations("llama", M, K, seed=seed))
    res = to_dev(synth.activations("deepseek", M, K, seed=seed + 1))
    wn = to_dev(synth.uniform_bf16((K,), 0.5, 1.5, seed=seed))
    wr = to_dev(synth.weights("llama", E, K, seed=seed))
    bias = torch.linspace(-0.1, 0.1, E, device="cuda")
    return x, res, wn, wr, bias, _experts(E, I, K, fmt, seed)


@pytest.mark.parametrize("fmt", ["fp32", "ue8m0"])
@pytest.mark.parametrize("M", [1, 7, 64])
def test_block(M, fmt):
    K, I, E = 1024, 384, 16
    x, res, wn, wr, bias, experts = _inputs(M, K, I, E, fmt, seed=M)
    qa, sa, h, r, logits, ids, w, y, nxt = _block(x, res, wn, wr, bias, experts, fmt)
    n, r_ref = ref.norm_rows(x, res, wn, 1e-6)
    assert torch.equal(r, r_ref)
    ref.check_norm(n, fmt, qa, sa, h)
    ids_ref, w_ref = ref.route(logits, 4, "sigmoid", bias=bias, n_group=4, topk_group=2, scale=2.5)
    assert ids.cpu().tolist() == ids_ref.tolist()
    assert float((w.double().cpu() - torch.from_numpy(w_ref)).abs().max()) <= 2.5 * 128 * ref.U32
    want, tol = ref.moe(qa, sa, ids, w, *experts)
    assert bool(((y.double() - want).abs() <= tol).all())
    n2, r2 = ref.norm_rows(y, r, wn, 1e-6)
    assert torch.equal(nxt[3], r2)
    ref.check_norm(n2, fmt, *nxt[:3])


def test_block_in_a_graph():
    args = _inputs(16, 1024, 384, 16, "fp32", seed=5)
    x = args[0]
    fresh = to_dev(synth.activations("llama", 16, 1024, seed=55))
    first = _block(*args, "fp32")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):      # the router's product warms its library up
        _block(*args, "fp32")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _block(*args, "fp32")
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got[:8], first[:8]):
        assert torch.equal(a, b)
    x.copy_(fresh)
    graph.replay()
    torch.cuda.synchronize()
    want, tol = ref.moe(got[0], got[1], got[5], got[6], *args[5])
    assert bool(((got[7].double() - want).abs() <= tol).all())
    assert not torch.equal(got[7], first[7])


def test_calls_keep_nothing():
    """Outputs die with their last reference, also those of refused calls; given
    outputs are returned as they are."""
    import gc
    import sys
    x, res, wn, wr, bias, experts = _inputs(4, 512, 256, 8, "fp32", seed=9)
    logits = torch.randn(4, 8, device="cuda")
    q, s = fb.fp8_add_rmsnorm_quant(x, residual=res, weight=wn)[:2]
    ids, w = fb.moe_route_topk(logits, 2)
    y = fb.fp8_moe_mlp(q, s, ids, w, *experts)
    again = fb.fp8_add_rmsnorm_quant(x, residual=res, weight=wn, q=q, s=s)
    assert again[0] is q and again[1] is s
    assert fb.moe_route_topk(logits, 2, ids=ids, weights=w)[0] is ids
    assert fb.fp8_moe_mlp(q, s, ids, w, *experts, y=y) is y
    del again
    torch.cuda.synchronize()
    gc.collect()
    used, refs = torch.cuda.memory_allocated(), [sys.getrefcount(t) for t in (x, q, ids, y)]
    for _ in range(50):
        fb.fp8_add_rmsnorm_quant(x, residual=res, weight=wn, q=q)
        fb.moe_route_topk(logits, 2, ids=ids)
        fb.fp8_moe_mlp(q, s, ids, w, *experts)
        fb.fp8_moe_mlp(q, s, ids, w, *experts, y=y)
        for bad in (lambda: fb.fp8_add_rmsnorm_quant(x, residual=res, eps=-1.0, q=q),
                    lambda: fb.moe_route_topk(logits, 9, ids=None),
                    lambda: fb.fp8_moe_mlp(q, s, ids, w, *experts, first_expert=-1, y=y)):
            with pytest.raises(fb.Fp8bsError):
                bad()
        with pytest.raises(TypeError):
            fb.moe_route_topk(logits, "2")
        with pytest.raises(TypeError):
            fb.fp8_add_rmsnorm_quant(x, residual=res, eps="small")
        with pytest.raises(ValueError):
            fb.fp8_add_rmsnorm_quant(x, residual=res, q=q, s=s[:2])
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == used
    assert [sys.getrefcount(t) for t in (x, q, ids, y)] == refs


def test_a_stream_of_the_callers_choice():
    """The current stream, and one that is given: outputs belong to it."""
    x, res, wn, wr, bias, experts = _inputs(16, 512, 256, 8, "fp32", seed=10)
    want = _block(x, res, wn, wr, bias[:8].contiguous(), experts, "fp32")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    q, s, h, r = fb.fp8_add_rmsnorm_quant(x, residual=res, weight=wn, stream=side)
    with torch.cuda.stream(side):
        logits = (h @ wr.t()).float()
        ids, w = fb.moe_route_topk(logits, 4, scoring="sigmoid", bias=bias, n_group=4, topk_group=2,
                                   scale=2.5)
    y = fb.fp8_moe_mlp(q, s, ids, w, *experts, stream=side)
    side.synchronize()
    for a, b in zip((q, s, h, r, ids, w, y), [want[i] for i in (0, 1, 2, 3, 5, 6, 7)]):
        assert torch.equal(a, b)
