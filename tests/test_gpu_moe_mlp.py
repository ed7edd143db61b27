"""fp8_moe_mlp (and its UE8M0 form) against the layer in 64 bits on the same
codes. The tolerance is the arithmetic's own: the fp32 products' roundings,
what those can move in h's codes (a step only where a rounding boundary lies
that near), and the output's half bf16 step."""

import pytest
import torch

from fp8_block_scaled_group128_b200 import binding as fb
from fp8_block_scaled_group128_b200 import synth

import moe_ref as ref
from gpu_util import require_gpu, to_dev

pytestmark = pytest.mark.gpu
FMT = ["fp32", "ue8m0"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert fb.get_device_error() == 0


def _fn(fmt):
    return fb.fp8_moe_mlp if fmt == "fp32" else fb.fp8_moe_mlp_ue8m0


def _rows(M, K, fmt, seed):
    x = to_dev(synth.activations("deepseek", M, K, seed=seed))
    return fb.fp8_quant_act_group128(x) if fmt == "fp32" else fb.fp8_quant_act_group128_ue8m0(x)


def _experts(E, I, K, fmt, seed):
    quant = fb.fp8_quant_weight_block128 if fmt == "fp32" else fb.fp8_quant_weight_block128_ue8m0
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for n, k in ((2 * I, K), (K, I)):
        parts = []
        for _ in range(E):
            spread = torch.exp(0.5 * torch.randn(n // 128, k // 128, generator=g, device="cuda"))
            w = torch.randn(n, k, generator=g, device="cuda") / k ** 0.5
            w = w * spread.repeat_interleave(128, 0).repeat_interleave(128, 1)
            parts.append(quant(w.to(torch.bfloat16)))
        out += [torch.stack([q for q, _ in parts]), torch.stack([s for _, s in parts])]
    return out


def _choices(M, E, k, seed, first=0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(M, E, generator=g).argsort(dim=1)[:, :k].to(torch.int32) + first
    w = torch.softmax(torch.randn(M, k, generator=g), dim=1)
    return ids.contiguous().cuda(), w.cuda()


def _check(y, args, first=0):
    want, tol = ref.moe(*args, first=first)
    err = (y.double() - want).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), int((err > tol).sum()))


def _case(M, K, I, E, k, fmt, seed=0):
    qa, sa = _rows(M, K, fmt, seed + 1)
    qg, sg, qd, sd = _experts(E, I, K, fmt, seed + 2)
    ids, w = _choices(M, E, k, seed + 3)
    return qa, sa, ids, w, qg, sg, qd, sd


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,K,I,E,k", [
    (1, 128, 128, 1, 1), (1, 256, 128, 4, 2), (1, 2048, 512, 16, 2), (2, 384, 256, 3, 3),
    (5, 640, 384, 7, 2), (15, 512, 128, 4, 1), (16, 512, 256, 4, 2), (17, 512, 256, 4, 2),
    (33, 256, 640, 5, 4), (64, 1152, 256, 9, 8), (65, 128, 384, 2, 2), (100, 384, 128, 32, 8),
    (127, 256, 256, 3, 1), (128, 512, 384, 4, 2), (128, 256, 128, 1, 1), (13, 2432, 1408, 27, 6),
    (31, 896, 128, 200, 6)])
def test_values(M, K, I, E, k, fmt):
    args = _case(M, K, I, E, k, fmt, seed=M + K)
    _check(_fn(fmt)(*args), args)


@pytest.mark.parametrize("fmt", FMT)
def test_expert_shapes(fmt):
    """DeepSeek-V3's expert sizes, 8 experts, 3 tokens."""
    args = _case(3, 7168, 2048, 8, 2, fmt, seed=31)
    _check(_fn(fmt)(*args), args)


@pytest.mark.parametrize("K,I", [(512, 256), (2048, 512)])
def test_the_tolerance_sees_mistakes(K, I):
    """A choice left out, one block's scale off by a quarter, or two experts
    exchanged, planted in the 64-bit layer, are outside the tolerance."""
    args = _case(6, K, I, 5, 2, "fp32", seed=30)
    y = fb.fp8_moe_mlp(*args).double()
    used = int(args[2][0, 0])

    def seen(i, change):
        t = args[i].clone()
        change(t)
        want, tol = ref.moe(*[t if j == i else a for j, a in enumerate(args)])
        return bool(((y - want).abs() > tol).any())

    assert seen(3, lambda w: w[0, 1].zero_())
    assert seen(5, lambda s: s[used, 0, 1].mul_(1.25))
    assert seen(7, lambda s: s[used, 0, 0].mul_(1.25))
    assert seen(2, lambda i: i[0].copy_(i[0].flip(0)))


@pytest.mark.parametrize("M", [1, 19, 128])
def test_all_tokens_to_one_expert(M):
    args = list(_case(M, 384, 256, 6, 1, "fp32", seed=40 + M))
    args[2] = torch.full((M, 1), 4, dtype=torch.int32, device="cuda")
    _check(fb.fp8_moe_mlp(*args), args)


def test_ids_outside_and_empty_rows():
    """-1, ids below and above the local range, and whole rows without a local
    expert: those rows are zeros."""
    args = list(_case(12, 256, 256, 4, 3, "fp32", seed=50))
    ids = args[2]
    ids[0] = -1
    ids[1] = torch.tensor([-1, 2, -7], dtype=torch.int32)
    ids[2] = torch.tensor([4, 1000, 2 ** 31 - 1], dtype=torch.int32)
    ids[3] = torch.tensor([3, -2 ** 31, 0], dtype=torch.int32)
    args[3][1, 0] = float("nan")    # the weight of no expert is not read into the sum
    y = fb.fp8_moe_mlp(*args)
    clean = list(args)
    clean[3] = args[3].nan_to_num(0.0)
    _check(y, clean)
    assert bool((y[0] == 0).all()) and bool((y[2] == 0).all())
    args[2] = torch.full_like(ids, -1)
    assert bool((fb.fp8_moe_mlp(*args) == 0).all())


@pytest.mark.parametrize("fmt", FMT)
def test_first_expert(fmt):
    """Two ranks with half of the experts each add up to the whole layer."""
    qa, sa, ids, w, qg, sg, qd, sd = args = _case(20, 512, 256, 8, 3, fmt, seed=60)
    parts = []
    for r in range(2):
        h = slice(4 * r, 4 * r + 4)
        part = (qa, sa, ids, w, qg[h], sg[h], qd[h], sd[h])
        y = _fn(fmt)(*part, first_expert=4 * r)
        _check(y, part, first=4 * r)
        parts.append(y.double())
    want, tol = ref.moe(*args)
    size = parts[0].abs() + parts[1].abs()
    assert bool(((parts[0] + parts[1] - want).abs() <= 2 * tol + size * ref.U16).all())


def test_an_expert_named_twice():
    """The weights of a repeated expert add."""
    args = list(_case(9, 256, 128, 5, 4, "fp32", seed=70))
    args[2][:, 1] = args[2][:, 0]
    args[2][3] = 2
    _check(fb.fp8_moe_mlp(*args), args)


def test_weights_of_zero_and_large():
    args = list(_case(7, 256, 128, 5, 2, "fp32", seed=71))
    args[3][0] = 0.0
    args[3][1] = torch.tensor([-3.0, 1e4])
    y = fb.fp8_moe_mlp(*args)
    _check(y, args)
    assert bool((y[0] == 0).all())


def test_zero_token_and_nan_token():
    """A token of zeros gives zeros; a NaN stays in its token's row."""
    args = list(_case(18, 256, 256, 4, 2, "fp32", seed=72))
    args[0][5] = 0
    args[1][5] = 0.0
    args[0][9, 3] = 0x7F
    y = fb.fp8_moe_mlp(*args)
    assert bool((y[5] == 0).all()) and bool(y[9].isnan().all())
    keep = [m for m in range(18) if m != 9]
    part = [a[keep] for a in args[:4]] + args[4:]
    _check(y[keep], part)


def test_ue8m0_nan_scales():
    """Code 255 is NaN: of a token, of gate+up, of down; the other results stay."""
    args = list(_case(18, 256, 256, 4, 2, "ue8m0", seed=81))
    clean = fb.fp8_moe_mlp_ue8m0(*args)
    ids = args[2]
    sa, sg, sd = args[1].clone(), args[5].clone(), args[7].clone()
    sa[9, 1] = 255
    y = fb.fp8_moe_mlp_ue8m0(args[0], sa, *args[2:])
    keep = torch.arange(18, device="cuda") != 9
    assert bool(y[9].isnan().all()) and torch.equal(y[keep], clean[keep])
    hit = (ids == 2).any(dim=1)
    assert bool(hit.any()) and not bool(hit.all())
    for block in (1, 3):   # gate rows 128 to 255, up rows 128 to 255
        s = sg.clone()
        s[2, block, 0] = 255
        y = fb.fp8_moe_mlp_ue8m0(*args[:5], s, *args[6:])
        assert bool(y[hit].isnan().all()) and torch.equal(y[~hit], clean[~hit])
    sd[2, 1, 1] = 255      # output columns 128 to 255
    y = fb.fp8_moe_mlp_ue8m0(*args[:7], sd)
    assert bool(y[hit][:, 128:].isnan().all()) and torch.equal(y[~hit], clean[~hit])
    assert torch.equal(y[:, :128], clean[:, :128])


@pytest.mark.parametrize("fmt", FMT)
def test_h_beyond_fp32(fmt):
    """h of one token overflows: its row is NaN, the others stay."""
    args = list(_case(18, 256, 256, 4, 2, fmt, seed=83))
    run = fb.fp8_moe_mlp if fmt == "fp32" else fb.fp8_moe_mlp_ue8m0
    clean = run(*args)
    args[1] = args[1].clone()
    args[1][5] = 2.0 ** 70 if fmt == "fp32" else 197
    a = ref.dequant_rows(args[0][5:6], args[1][5:6])
    w = ref.dequant_blocks(args[4], args[5])[int(args[2][5, 0])]
    g, u = (a @ w.T).chunk(2, dim=-1)
    assert float((g.clamp(min=0) * u).abs().max()) > 1e40
    y = run(*args)
    assert bool(y[5].isnan().all())
    keep = torch.arange(18, device="cuda") != 5
    assert torch.equal(y[keep], clean[keep])


def test_deterministic_and_batch_rows_agree():
    args = _case(64, 1024, 512, 8, 2, "fp32", seed=73)
    y = fb.fp8_moe_mlp(*args)
    for _ in range(5):
        assert torch.equal(y, fb.fp8_moe_mlp(*args))


def test_workspace_streams_and_two_calls_at_once():
    """A kept workspace full of garbage, and two streams with a workspace each."""
    a = _case(16, 1024, 512, 8, 2, "fp32", seed=74)
    b = _case(40, 768, 384, 6, 3, "fp32", seed=75)
    ya, yb = fb.fp8_moe_mlp(*a), fb.fp8_moe_mlp(*b)
    ws = [torch.full((fb.moe_workspace_bytes(m, k, i, e, t),), 0xFF, dtype=torch.uint8, device="cuda")
          for m, k, i, e, t in ((16, 1024, 512, 8, 2), (40, 768, 384, 6, 3))]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        outs.append((fb.fp8_moe_mlp(*a, workspace=ws[0], stream=s1),
                     fb.fp8_moe_mlp(*b, workspace=ws[1], stream=s2)))
    torch.cuda.synchronize()
    for ga, gb in outs:
        assert torch.equal(ga, ya) and torch.equal(gb, yb)
    # one workspace for calls of other sizes, one after the other
    big = torch.full((max(w.numel() for w in ws),), 0xA5, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(fb.fp8_moe_mlp(*a, workspace=big), ya)
        assert torch.equal(fb.fp8_moe_mlp(*b, workspace=big), yb)


def test_graphs_that_share_a_workspace():
    """Captured and replayed with other tokens and other choices; two graphs
    replayed in turn on one workspace."""
    a = list(_case(8, 512, 256, 8, 2, "fp32", seed=76))
    b = _case(24, 512, 256, 8, 2, "fp32", seed=77)
    ws = torch.empty(fb.moe_workspace_bytes(24, 512, 256, 8, 2), dtype=torch.uint8, device="cuda")
    ya_eager, yb_eager = fb.fp8_moe_mlp(*a), fb.fp8_moe_mlp(*b)
    torch.cuda.synchronize()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        ya = fb.fp8_moe_mlp(*a, workspace=ws)
    with torch.cuda.graph(gb):
        yb = fb.fp8_moe_mlp(*b, workspace=ws)
    for _ in range(3):
        ga.replay()
        gb.replay()
    torch.cuda.synchronize()
    assert torch.equal(ya, ya_eager) and torch.equal(yb, yb_eager)
    ids, w = _choices(8, 8, 2, seed=99)
    qa, sa = _rows(8, 512, "fp32", seed=98)
    for t, n in zip(a[:4], (qa, sa, ids, w)):
        t.copy_(n)
    ga.replay()
    torch.cuda.synchronize()
    _check(ya, a)
    assert torch.equal(ya, fb.fp8_moe_mlp(*a))


def test_rows_behind_the_last_token_are_left_alone():
    args = list(_case(6, 256, 128, 4, 2, "fp32", seed=78))
    y = torch.full((8, 256), 5.0, dtype=torch.bfloat16, device="cuda")
    fb.fp8_moe_mlp(*args, y=y[1:7])
    assert bool((y[0] == 5).all()) and bool((y[7] == 5).all())
    _check(y[1:7], args)


def test_refusals():
    qa, sa, ids, w, qg, sg, qd, sd = args = _case(4, 256, 128, 4, 2, "fp32", seed=79)
    for i, bad in ((0, qa.float()), (1, sa.to(torch.uint8)), (2, ids.long()), (3, w.double()),
                   (4, qg.float()), (5, sg.double())):
        with pytest.raises(TypeError):
            fb.fp8_moe_mlp(*[bad if j == i else t for j, t in enumerate(args)])
    for i, bad in ((0, qa[:3]), (1, sa[:, :1].contiguous()), (2, ids[:3]), (3, w[:, :1].contiguous()),
                   (4, qg[:, :128].contiguous()), (5, sg[:3].contiguous()), (6, qd[0]),
                   (7, sd[:, :1].contiguous()), (4, qg.transpose(1, 2))):
        with pytest.raises(ValueError):
            fb.fp8_moe_mlp(*[bad if j == i else t for j, t in enumerate(args)])
    with pytest.raises(fb.Fp8bsError):
        fb.fp8_moe_mlp(*args, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fb.Fp8bsError):
        fb.fp8_moe_mlp(*args, first_expert=-1)
    big = _case(4, 256, 128, 4, 2, "fp32", seed=80)
    rep = [t.repeat(33, 1) for t in big[:4]]
    with pytest.raises(fb.Fp8bsError):
        fb.fp8_moe_mlp(*rep, *big[4:])
    y = fb.fp8_moe_mlp(qa[:0], sa[:0], ids[:0], w[:0], qg, sg, qd, sd)
    assert y.shape == (0, 256)


@pytest.mark.parametrize("M,K,I,E,k", [
    (1, 512, 8192, 8, 8), (2, 256, 6272, 4, 3), (3, 4096, 384, 5, 5), (1, 8192, 128, 2, 1),
    (128, 128, 128, 64, 32), (128, 256, 384, 1, 1), (97, 640, 384, 2, 1), (40, 256, 128, 1024, 4),
    (128, 1024, 896, 3, 2), (64, 384, 2176, 2, 2)])
def test_results_of_many_parts(M, K, I, E, k):
    """Results summed from many chunks (long K or I with few tokens, more than
    16 parts of an output), experts with two blocks of tokens, as many choices
    and experts as there can be."""
    args = _case(M, K, I, E, k, "fp32", seed=200 + M + I)
    y = fb.fp8_moe_mlp(*args)
    _check(y, args)
    assert torch.equal(y, fb.fp8_moe_mlp(*args))


@pytest.mark.parametrize("M", [1, 24, 128])
def test_bounded_wait_reports_timeout_and_recovers(M):
    """A wait limit of one cycle: the call records the timeout and ends, and the
    next one with the default limit, on the same workspace, is right."""
    args = _case(M, 1024, 512, 4, 2, "fp32", seed=81)
    ws = torch.empty(fb.moe_workspace_bytes(M, 1024, 512, 4, 2), dtype=torch.uint8, device="cuda")
    fb.get_device_error()
    try:
        fb.set_wait_limit(1)
        fb.fp8_moe_mlp(*args, workspace=ws)
        assert fb.get_device_error() == 6
    finally:
        fb.set_wait_limit(0)
    y = fb.fp8_moe_mlp(*args, workspace=ws)
    assert fb.get_device_error() == 0
    _check(y, args)


def test_experts_beyond_32_bit_offsets():
    """80 experts of 7168 x 2048 (2.3 GB of gate+up codes): the last two as in a
    call that has only them."""
    E, K, I = 80, 7168, 2048
    qa, sa = _rows(3, K, "fp32", 301)
    two = _experts(2, I, K, "fp32", 302)
    full = [torch.zeros((E,) + t.shape[1:], dtype=t.dtype, device="cuda") for t in two]
    for f, t in zip(full, two):
        f[E - 2:] = t
    ids = torch.tensor([[E - 1, E - 2], [E - 1, -1], [E - 2, E - 1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.75, 0.25], [1.0, 0.5], [0.5, 0.5]], device="cuda")
    y = fb.fp8_moe_mlp(qa, sa, ids, w, *full)
    part = (qa, sa, ids, w, *two)
    assert torch.equal(y, fb.fp8_moe_mlp(*part, first_expert=E - 2))
    _check(y, part, first=E - 2)


@pytest.mark.parametrize("M,E,k", [(4, 5, 4), (1, 40, 32), (8, 3, 4), (31, 6, 1), (2, 200, 16), (16, 2, 2)])
def test_few_choices(M, E, k):
    """At most 32 choices: repeated experts, ids outside the range, whole rows
    without an expert, in one call."""
    g = torch.Generator().manual_seed(400 + M)
    args = list(_case(M, 384, 256, E, 1, "fp32", seed=90 + M))
    ids = torch.randint(-1, E + 2, (M, k), generator=g).to(torch.int32)
    if M > 2:
        ids[1] = -1
        ids[2] = E - 1
    args[2], args[3] = ids.cuda(), torch.randn(M, k, generator=g).cuda()
    y = fb.fp8_moe_mlp(*args)
    _check(y, args)
    # more of the same tokens: the plan for many choices
    more = [torch.cat([a] * (33 // (M * k) + 1)) for a in args[:4]] + args[4:]
    assert more[2].numel() > 32
    _check(fb.fp8_moe_mlp(*more), more)
    args[2] = torch.full_like(args[2], E)
    assert bool((fb.fp8_moe_mlp(*args) == 0).all())
