"""Host-side checks of the mixture-of-experts block's entry points: every
refusal happens before a GPU is touched."""

import ctypes

import pytest
import torch

from fp8_block_scaled_group128_b200 import binding as fb
from fp8_block_scaled_group128_b200.build import build

OK, NULL, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4
P = ctypes.c_void_p(0x1000)
MIS = ctypes.c_void_p(0x1004)    # 4-byte aligned only
MIS2 = ctypes.c_void_p(0x1002)   # 2-byte aligned
MIS1 = ctypes.c_void_p(0x1001)


@pytest.fixture(scope="module")
def lib():
    build()
    return fb.lib()


@pytest.mark.parametrize("name", ["fp8_add_rmsnorm_quant", "fp8_add_rmsnorm_quant_ue8m0"])
def test_norm_refusals(lib, name):
    f = getattr(lib, name)

    def call(x=P, res=P, w=P, eps=1e-6, M=4, K=256, out=P, y=P, q=P, s=P):
        return f(x, res, w, eps, M, K, out, y, q, s, None)

    for K in (0, -128, 100, 65536 + 128):
        assert call(K=K) == SHAPE
    assert call(M=-1) == SHAPE
    assert call(M=1 << 31) == SHAPE
    for eps in (-1e-6, float("nan"), float("inf")):
        assert call(eps=eps) == SHAPE
    for k in ("x", "q", "s"):
        assert call(**{k: None}) == NULL
    for k in ("x", "res", "w", "out", "y", "q"):
        assert call(**{k: MIS}) == ALIGN
    if name.endswith("quant"):
        assert call(s=MIS2) == ALIGN
    assert call(x=None, q=None, s=None, M=0) == OK


def test_route_refusals(lib):
    f = lib.moe_route_topk

    def call(x=P, bf16=0, bias=None, scoring=1, M=4, E=16, k=2, ng=1, kg=1, ids=P, w=P):
        return f(x, bf16, bias, scoring, M, E, k, ng, kg, 1, 1.0, ids, w, None)

    for bad in (dict(M=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=17), dict(E=64, k=33),
                dict(scoring=2), dict(scoring=-1), dict(ng=0), dict(ng=3), dict(E=66, ng=33),
                dict(ng=4, kg=0), dict(ng=4, kg=5), dict(ng=8, kg=1, k=3), dict(ng=4, kg=2, scoring=0),
                dict(bias=P, scoring=0)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(x=None), dict(ids=None), dict(w=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(x=MIS2), dict(x=MIS1, bf16=1), dict(bias=MIS2), dict(ids=MIS2), dict(w=MIS2)):
        assert call(**bad) == ALIGN, bad
    assert call(x=None, ids=None, w=None, M=0) == OK


@pytest.mark.parametrize("name", ["fp8_moe_mlp", "fp8_moe_mlp_ue8m0"])
def test_moe_refusals(lib, name):
    f = getattr(lib, name)
    names = ("qa", "sa", "ids", "weights", "qg", "sg", "qd", "sd", "y")
    big = 1 << 30

    def call(M=4, K=256, I=128, E=4, k=2, first=0, ws=P, size=big, **ptr):
        return f(*[ptr.get(n, P) for n in names], M, K, I, E, k, first, ws, size, None)

    for bad in (dict(M=-1), dict(M=129), dict(K=0), dict(K=100), dict(I=0), dict(I=192), dict(E=0),
                dict(E=1025), dict(k=0), dict(k=33), dict(first=-1), dict(first=1 << 31),
                dict(E=1024, I=1 << 20), dict(E=1024, K=1 << 22)):
        assert call(**bad) == SHAPE, bad
    for n in names:
        assert call(**{n: None}) == NULL, n
    for n in ("qa", "qg", "qd", "y"):
        assert call(**{n: MIS}) == ALIGN, n
    for n in ("ids", "weights"):
        assert call(**{n: MIS2}) == ALIGN, n
    if name == "fp8_moe_mlp":
        for n in ("sa", "sg", "sd"):
            assert call(**{n: MIS2}) == ALIGN, n
    need = lib.fp8bs_moe_workspace_bytes(4, 256, 128, 4, 2)
    assert need > 0
    assert call(size=need - 1) == WORKSPACE
    assert call(ws=None) == WORKSPACE
    assert call(ws=MIS) == WORKSPACE
    assert call(M=0, ws=None, size=0, **{n: None for n in names}) == OK


def test_moe_workspace_query(lib):
    q = lib.fp8bs_moe_workspace_bytes
    assert q(0, 256, 128, 4, 2) == 0
    assert q(129, 256, 128, 4, 2) == 0 and q(4, 100, 128, 4, 2) == 0
    sizes = [q(m, 4096, 2048, 8, 2) for m in (1, 16, 17, 64, 128)]
    assert sizes == sorted(sizes) and sizes[0] > 0


def test_host_tensors_are_refused():
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    u8, f32, i32 = (torch.zeros(2, 256, dtype=d) for d in (torch.uint8, torch.float32, torch.int32))
    with pytest.raises(TypeError):
        fb.fp8_add_rmsnorm_quant(x)
    with pytest.raises(TypeError):
        fb.fp8_add_rmsnorm_quant_ue8m0(x, residual=x)
    with pytest.raises(TypeError):
        fb.moe_route_topk(f32, 2)
    with pytest.raises(TypeError):
        fb.fp8_moe_mlp(u8, f32, i32, f32, u8, f32, u8[None], f32)
