"""fp8_moe_mlp: a token's result beside other tokens and alone. How the work is
cut, and with it the order of the sums, goes by the whole call, so that rows of
different batches agree within the arithmetic's tolerance, not to the bit."""

import pytest
import torch

from fp8_block_scaled_group128_b200 import binding as fb

import moe_ref as ref
from gpu_util import require_gpu
from test_gpu_moe_mlp import FMT, _case, _fn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert fb.get_device_error() == 0


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,K,I,E,k", [(64, 1024, 512, 8, 2), (128, 512, 384, 3, 2), (33, 2048, 128, 24, 6),
                                       (17, 256, 2048, 4, 1)])
def test_rows_alone_and_in_a_batch(M, K, I, E, k, fmt):
    args = _case(M, K, I, E, k, fmt, seed=500 + M)
    y = _fn(fmt)(*args)
    want, tol = ref.moe(*args)
    assert bool(((y.double() - want).abs() <= tol).all())
    for lo, hi in ((0, 1), (M - 1, M), (3, 19), (0, M // 2), (M // 2, M)):
        part = [t[lo:hi].contiguous() for t in args[:4]] + list(args[4:])
        alone = _fn(fmt)(*part)
        # each side is within tol of the 64-bit layer
        assert bool(((alone.double() - y[lo:hi].double()).abs() <= 2 * tol[lo:hi]).all())
        assert bool(((alone.double() - want[lo:hi]).abs() <= tol[lo:hi]).all())


@pytest.mark.parametrize("fmt", FMT)
def test_order_of_the_tokens(fmt):
    """Tokens in another order: the same rows, to the bit (the cut goes by the
    numbers of tokens, and a row's sums have their order of experts and parts)."""
    args = list(_case(96, 768, 384, 6, 3, fmt, seed=540))
    y = _fn(fmt)(*args)
    order = torch.randperm(96, generator=torch.Generator().manual_seed(2)).cuda()
    moved = [t[order].contiguous() for t in args[:4]] + args[4:]
    assert torch.equal(_fn(fmt)(*moved), y[order])
