"""moe_route_topk against the definition in 64 bits: the same ids everywhere
(ties to the lowest index, dead experts never chosen), weights within fp32
error."""

import numpy as np
import pytest
import torch

from fp8_block_scaled_group128_b200 import binding as fb

import moe_ref as ref
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

# fp32 weights: exponential (2 ulp), the sum of up to 1024 terms (32 chained
# additions per lane and 5 tree levels at most), divisions and the scale: under
# 50 roundings of 2^-24 each, plus the argument's rounding |x - max| <= 88 half
# steps of the exponential
REL = 192 * ref.U32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _logits(M, E, seed, dtype=torch.float32, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, E, generator=g) * spread).to(dtype).cuda()


def _bias(E, seed, size=0.2):
    g = torch.Generator().manual_seed(1000 + seed)
    return (torch.randn(E, generator=g) * size).cuda()


def _check(x, k, **kw):
    ids, w = fb.moe_route_topk(x, k, **kw)
    ids_ref, w_ref = ref.route(x, k, **{"scoring": "softmax", **kw})
    np.testing.assert_array_equal(ids.cpu().numpy(), ids_ref)
    w = w.double().cpu().numpy()
    assert np.all(np.abs(w - w_ref) <= np.abs(w_ref) * REL + 1e-37), np.abs(w - w_ref).max()
    return ids, w


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (1, 8, 2), (5, 8, 8), (33, 31, 5), (6, 32, 32), (17, 60, 4),
                                   (9, 65, 3), (13, 129, 6), (3, 256, 8), (5, 257, 8), (4, 512, 22),
                                   (3, 1000, 32), (2, 1024, 10)])
def test_plain(M, E, k, scoring, renorm, dtype):
    _check(_logits(M, E, seed=M + E, dtype=dtype), k, scoring=scoring, renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,E,k", [(1, 4, 1), (33, 60, 6), (70, 256, 8), (3, 1024, 32)])
def test_bias(M, E, k, dtype):
    _check(_logits(M, E, seed=E, dtype=dtype), k, scoring="sigmoid", bias=_bias(E, E))


@pytest.mark.parametrize("E,ng,kg,k", [(256, 8, 4, 8), (256, 8, 1, 8), (64, 32, 3, 6), (96, 3, 2, 5),
                                       (10, 10, 4, 4), (120, 5, 5, 7), (1024, 16, 2, 32), (84, 7, 3, 1)])
@pytest.mark.parametrize("bias", [True, False])
def test_groups(E, ng, kg, k, bias):
    _check(_logits(41, E, seed=E + ng), k, scoring="sigmoid", n_group=ng, topk_group=kg,
           bias=_bias(E, ng) if bias else None, scale=1.5)


def test_ties_go_to_the_lowest_index():
    """Logits of a few values only, so that most choices are ties."""
    g = torch.Generator().manual_seed(3)
    x = torch.randint(-2, 3, (64, 96), generator=g).float().cuda()
    _check(x, 9)
    _check(x, 9, scoring="sigmoid", bias=torch.zeros(96, device="cuda"))
    _check(x, 9, scoring="sigmoid", n_group=6, topk_group=2)
    _check(torch.zeros(2, 70, device="cuda"), 32)
    z = torch.zeros(1, 40, device="cuda")
    z[0, ::2] = -0.0
    assert fb.moe_route_topk(z, 8)[0].tolist() == [list(range(8))]


def test_close_scores_are_ordered_in_64_bits():
    """Biases that differ by less than a 32-bit sigmoid resolves."""
    x = torch.full((1, 64), 0.3, device="cuda")
    bias = torch.zeros(64, device="cuda")
    bias[7] = 2.0 ** -30
    bias[50] = 2.0 ** -28
    bias[20] = -(2.0 ** -40)
    ids, _ = _check(x, 4, scoring="sigmoid", bias=bias)
    assert ids.tolist() == [[50, 7, 0, 1]]


def test_dead_experts():
    """-inf and NaN logits and biases: never chosen, and -1 where fewer than
    top_k are left, down to a row with none."""
    x = _logits(6, 40, seed=8)
    x[0, :] = -float("inf")
    x[1, 3:] = -float("inf")
    x[2, ::2] = float("nan")
    x[3, :39] = float("nan")
    x[4, 8:] = -float("inf")
    for kw in (dict(), dict(scoring="sigmoid"), dict(renormalize=False),
               dict(scoring="sigmoid", n_group=5, topk_group=2)):
        ids, w = _check(x, 6, **kw)
        assert ids[0].tolist() == [-1] * 6 and not w[0].any()
    bias = _bias(40, 1)
    bias[5] = -float("inf")
    bias[6] = float("nan")
    ids, _ = _check(x, 6, scoring="sigmoid", bias=bias)
    assert not torch.isin(ids, torch.tensor([5, 6], device="cuda", dtype=torch.int32)).any()


def test_wide_logits():
    """Spread over hundreds: weights that underflow and scores that saturate."""
    x = _logits(16, 100, seed=9, spread=60.0)
    _check(x, 5, renormalize=False)
    ids, w = fb.moe_route_topk(x, 5, scoring="sigmoid")
    ids_ref, _ = ref.route(x, 5, "sigmoid")
    np.testing.assert_array_equal(ids.cpu().numpy(), ids_ref)
    assert bool(torch.isfinite(w).all())


def test_many_rows_stream_graph_and_given_outputs():
    x, bias = _logits(4099, 256, seed=10), _bias(256, 10)
    kw = dict(scoring="sigmoid", bias=bias, n_group=8, topk_group=4)
    ids, w = fb.moe_route_topk(x, 8, **kw)
    some = torch.tensor([0, 1, 777, 4095, 4098])
    ids_ref, w_ref = ref.route(x[some.cuda()], 8, **kw)
    np.testing.assert_array_equal(ids[some.cuda()].cpu().numpy(), ids_ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    i2, w2 = fb.moe_route_topk(x, 8, stream=side, **kw)
    side.synchronize()
    assert torch.equal(ids, i2) and torch.equal(w, w2)
    out = torch.full((4101, 8), 99, dtype=torch.int32, device="cuda")
    wo = torch.full((4101, 8), 9.0, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fb.moe_route_topk(x, 8, ids=out[1:-1], weights=wo[1:-1], **kw)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[1:-1], ids) and torch.equal(wo[1:-1], w)
    assert bool((out[0] == 99).all()) and bool((out[-1] == 99).all()) and bool((wo[-1] == 9).all())


def test_refusals():
    x = _logits(3, 16, seed=1)
    with pytest.raises(ValueError):
        fb.moe_route_topk(x, 2, scoring="tanh")
    with pytest.raises(TypeError):
        fb.moe_route_topk(x.half(), 2)
    with pytest.raises(ValueError):
        fb.moe_route_topk(x.t(), 2)
    with pytest.raises(ValueError):
        fb.moe_route_topk(x, 2, scoring="sigmoid", bias=torch.zeros(15, device="cuda"))
    with pytest.raises(TypeError):
        fb.moe_route_topk(x, 2, scoring="sigmoid", bias=torch.zeros(16, device="cuda").bfloat16())
    for kw in (dict(top_k=17), dict(top_k=0), dict(top_k=2, n_group=4),
               dict(top_k=2, bias=torch.zeros(16, device="cuda")),
               dict(top_k=5, scoring="sigmoid", n_group=4, topk_group=1)):
        with pytest.raises(fb.Fp8bsError):
            fb.moe_route_topk(x, **kw)
    with pytest.raises(ValueError):
        fb.moe_route_topk(x, 2, ids=torch.zeros(3, 3, dtype=torch.int32, device="cuda"))
    assert fb.moe_route_topk(x[:0], 2)[0].shape == (0, 2)


@pytest.mark.parametrize("M", [5, 700])
@pytest.mark.parametrize("E,ng,kg,k", [(48, 1, 1, 3), (48, 6, 2, 3), (200, 8, 3, 7), (1024, 32, 5, 9)])
def test_few_and_many_rows(M, E, ng, kg, k):
    """A thread for each expert, or one or two warps for a row; bf16 logits,
    which tie; the weights of one are those of the other."""
    x = _logits(M, E, seed=E + M, dtype=torch.bfloat16)
    kw = dict(scoring="sigmoid", n_group=ng, topk_group=kg, bias=_bias(E, ng))
    _check(x, k, **kw)
    ids, w = fb.moe_route_topk(x, k, **kw)
    more = fb.moe_route_topk(torch.cat([x, x]), k, **kw)
    assert torch.equal(more[0][:M], ids) and torch.equal(more[1][M:], w)


@pytest.mark.parametrize("ng,kg", [(1, 1), (4, 2)])
def test_scores_far_from_zero(ng, kg):
    """Logits down to -700 and up to the largest: scores near 0 and equal to 1."""
    g = torch.Generator().manual_seed(12)
    x = (torch.randn(20, 32, generator=g) * 150).clamp(-690, 1e4)
    x[3] = -80 - 3 * torch.arange(32)
    x[4, :20] = 50 + torch.arange(20)          # 1 in 64 bits: ties
    x[5, 7] = 3e38
    x[6] = torch.linspace(-61, -59, 32)
    bias = torch.zeros(32, device="cuda")
    _check_ids(x.cuda(), 6, scoring="sigmoid", bias=bias, n_group=ng, topk_group=kg)


def _check_ids(x, k, **kw):
    ids, _ = fb.moe_route_topk(x, k, **kw)
    np.testing.assert_array_equal(ids.cpu().numpy(), ref.route(x, k, **kw)[0])


def test_offsets_beyond_32_bits():
    """2.25e9 logits: the last rows as in a call of their own."""
    M, E = 2_200_000, 1024
    base = _logits(2000, E, seed=13, dtype=torch.bfloat16)
    x = base.repeat(M // 2000, 1)
    x[-700:] = _logits(700, E, seed=14, dtype=torch.bfloat16)
    ids, w = fb.moe_route_topk(x, 4)
    tail = fb.moe_route_topk(x[-700:], 4)
    assert torch.equal(ids[-700:], tail[0]) and torch.equal(w[-700:], tail[1])
    assert torch.equal(ids[:2000], ids[2000:4000])
