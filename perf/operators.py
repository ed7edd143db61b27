"""Cases of the mixture-of-experts block around the fine-grained FP8 linear layer.

Three operators that run one after the other in a decoder layer whose MLP is a
mixture of experts:

* ``norm``: the residual addition, the root-mean-square norm and the 1x128
  quantization of the normed row (fp32 or power-of-two scales);
* ``route``: the choice of the experts of every token from the router's
  logits, and their weights;
* ``moe``: the whole expert MLP (gate+up, SwiGLU, quantization, down, weighted
  sum) for a few tokens.

``run`` computes them with elementary torch operations, or (``own``) by the
library's entry points. ``exact`` states the same definitions again in 64 bits.
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-6
GROUP = 128
E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # One new token of a 4096-wide model: the norm before its linears
        # (latency only).
        dict(name="norm_token_4096", op="norm", M=1, K=4096, fmt="fp32", residual=True, y=True),
        # A decode batch of a 7168-wide mixture-of-experts model with
        # power-of-two scales; the bf16 row goes on to the router.
        dict(name="norm_batch64_7168_ue8m0", op="norm", M=64, K=7168, fmt="ue8m0", residual=True,
             y=True),
        # A prefill chunk of the 4096-wide model.
        dict(name="norm_prefill8192_4096", op="norm", M=8192, K=4096, fmt="fp32", residual=True,
             y=True),
        # An odd number of rows of a 14336-wide activation, codes only, no
        # residual stream.
        dict(name="norm_ragged1037_14336", op="norm", M=1037, K=14336, fmt="fp32", residual=False,
             y=False),
        # One token of a model with 256 experts in 8 groups, of which 4 are
        # eligible, sigmoid scores with a selection bias, 8 choices.
        dict(name="route_token_256", op="route", M=1, E=256, top_k=8, scoring="sigmoid", bias=True,
             n_group=8, topk_group=4, renorm=True, scale=2.5, dtype="fp32", dead=0.0),
        # The same router on a prefill chunk.
        dict(name="route_prefill4096_256", op="route", M=4096, E=256, top_k=8, scoring="sigmoid",
             bias=True, n_group=8, topk_group=4, renorm=True, scale=2.5, dtype="fp32", dead=0.0),
        # Softmax over an odd number of experts, bf16 logits (which tie often),
        # some experts switched off.
        dict(name="route_softmax1021_60", op="route", M=1021, E=60, top_k=4, scoring="softmax",
             bias=False, n_group=1, topk_group=1, renorm=True, scale=1.0, dtype="bf16", dead=0.1),
        # One token of a small mixture-of-experts model (latency).
        dict(name="moe_token_small", op="moe", M=1, K=2048, I=512, E=16, total=16, top_k=2,
             fmt="fp32"),
        # One token through 2 of 8 experts of Llama-3-8B's MLP shape.
        dict(name="moe_token_14336", op="moe", M=1, K=4096, I=14336, E=8, total=8, top_k=2,
             fmt="fp32"),
        # A decode batch on one rank of an expert-parallel group: 32 of 256
        # experts are here, every token chose 8 of the 256.
        dict(name="moe_rank64_7168", op="moe", M=64, K=7168, I=2048, E=32, total=256, top_k=8,
             fmt="fp32"),
        # A larger decode batch over 8 experts, all local, power-of-two scales.
        dict(name="moe_batch128_ue8m0", op="moe", M=128, K=7168, I=2048, E=8, total=8, top_k=2,
             fmt="ue8m0"),
        # Odd sizes throughout.
        dict(name="moe_ragged13_1408", op="moe", M=13, K=2432, I=1408, E=27, total=27, top_k=6,
             fmt="fp32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "route", "moe"])
    if op == "norm":
        K = GROUP * _log_int(rng, 2, 112)
        M = _log_int(rng, 1, min(8192, 8192 * 4096 // K))
        return dict(op=op, M=M, K=K, fmt=rng.choice(["fp32", "ue8m0"]),
                    residual=rng.random() < 0.7, y=rng.random() < 0.6)
    if op == "route":
        M = _log_int(rng, 1, 4096)
        scoring = rng.choice(["softmax", "sigmoid"])
        if scoring == "sigmoid" and rng.random() < 0.5:
            n_group = rng.choice([2, 4, 8])
            per = rng.randint(4, 48)
            topk_group = rng.randint(1, n_group)
            E = n_group * per
            top_k = rng.randint(1, min(12, topk_group * per))
        else:
            n_group = topk_group = 1
            E = _log_int(rng, 4, 512)
            top_k = rng.randint(1, min(12, E))
        return dict(op=op, M=M, E=E, top_k=top_k, scoring=scoring,
                    bias=scoring == "sigmoid" and rng.random() < 0.6, n_group=n_group,
                    topk_group=topk_group, renorm=top_k > 1 and rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["fp32", "bf16"]),
                    dead=rng.choice([0.0, 0.0, 0.2]))
    K = GROUP * _log_int(rng, 4, 56)
    I = GROUP * _log_int(rng, 1, 64)
    room = 32 * 7168 * 2048 // (K * I)
    E = _log_int(rng, 1, max(1, min(64, room)))
    M, ranks = _log_int(rng, 1, 128), rng.choice([1, 1, 2, 8])
    top_k = rng.randint(1, min(8, E * ranks))
    if M * top_k < 4 * ranks:   # too few choices for a rank to see some of them
        ranks, top_k = 1, min(top_k, E)
    return dict(op=op, M=M, K=K, I=I, E=E, total=E * ranks, top_k=top_k,
                fmt=rng.choice(["fp32", "ue8m0"]))


def work(case):
    c = case
    M = c["M"]
    if c["op"] == "norm":
        K = c["K"]
        per_row = 2 * K * (1 + (2 if c["residual"] else 0) + (1 if c["y"] else 0)) + K
        per_row += (K // GROUP) * (4 if c["fmt"] == "fp32" else 1)
        return {"bytes": M * per_row + 2 * K, "flops": 6.0 * M * K}
    if c["op"] == "route":
        item = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": M * (c["E"] * item + 8 * c["top_k"]) + (4 * c["E"] if c["bias"] else 0),
                "flops": 8.0 * M * c["E"]}
    K, I, E = c["K"], c["I"], c["E"]
    share = c["top_k"] / c["total"]
    experts = E * (1.0 - (1.0 - share) ** M)   # experts that some token chose
    pairs = M * c["top_k"] * E / c["total"]    # (token, expert) pairs computed here
    scale = 4 if c["fmt"] == "fp32" else 1
    weights = 3 * I * K + 3 * (I // GROUP) * (K // GROUP) * scale
    tokens = M * (K + (K // GROUP) * scale + 8 * c["top_k"] + 2 * K)
    return {"bytes": experts * weights + tokens, "flops": 6.0 * pairs * I * K}


# ------------------------------------------------------------------ inputs --
def _gen(seed, *salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(hash((int(seed),) + salt) & 0x7FFFFFFFFFFF)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _block_codes(w, fmt):
    """Weights [N, K] -> E4M3 bytes and one scale per 128 x 128 block."""
    N, K = w.shape
    b = w.view(N // GROUP, GROUP, K // GROUP, GROUP)
    amax = b.abs().amax(dim=(1, 3))
    s, stored = _scales(amax, fmt)
    q = (b / s[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(N, K).view(torch.uint8), stored


def prepare(case, seed):
    c = case
    if c["op"] == "norm":
        g = _gen(seed, 1)
        M, K = c["M"], c["K"]
        x = _randn(g, M, K)
        x[:, torch.randperm(K, generator=g, device="cuda")[: max(1, K // 200)]] *= 30.0
        st = dict(c, x=x.to(torch.bfloat16),
                  weight=(1.0 + 0.2 * _randn(g, K)).to(torch.bfloat16), res=None)
        if c["residual"]:
            st["res"] = (2.0 * _randn(g, M, K)).to(torch.bfloat16)
        return st
    if c["op"] == "route":
        g = _gen(seed, 2)
        M, E = c["M"], c["E"]
        logits = 1.5 * _randn(g, M, E) + 0.5 * _randn(g, E)
        if c["dead"] > 0.0:   # experts switched off for everyone
            off = torch.rand(E, generator=g, device="cuda") < c["dead"]
            logits = logits.masked_fill(off, -math.inf)
        logits = logits.to(torch.float32 if c["dtype"] == "fp32" else torch.bfloat16)
        return dict(c, logits=logits, b=0.1 * _randn(g, E) if c["bias"] else None)
    g = _gen(seed, 3)
    M, K, I, E = c["M"], c["K"], c["I"], c["E"]
    x = _randn(g, M, K) * torch.exp(0.5 * _randn(g, M, 1))
    qa, sa = _rows_codes(x, c["fmt"])
    order = torch.rand(M, c["total"], generator=g, device="cuda").argsort(dim=1)
    ids = order[:, : c["top_k"]].to(torch.int32).contiguous()
    weights = torch.softmax(_randn(g, M, c["top_k"]), dim=1)
    qg = torch.empty(E, 2 * I, K, dtype=torch.uint8, device="cuda")
    qd = torch.empty(E, K, I, dtype=torch.uint8, device="cuda")
    sg, sd = [], []
    for e in range(E):
        for q, s, n, k in ((qg, sg, 2 * I, K), (qd, sd, K, I)):
            spread = torch.exp(0.5 * _randn(g, n // GROUP, 1, k // GROUP, 1))
            w = _randn(g, n, k).mul_(1.0 / math.sqrt(k)).view(n // GROUP, GROUP, k // GROUP, GROUP)
            q[e], stored = _block_codes(w.mul_(spread).view(n, k), c["fmt"])
            s.append(stored)
    # on a rank that holds part of the experts: the second share of them
    first = E if c["total"] > E else 0
    return dict(c, qa=qa, sa=sa, ids=ids, weights=weights, qg=qg, sg=torch.stack(sg), qd=qd,
                sd=torch.stack(sd), first=first)


# -------------------------------------------------------------- plain forms --
def _scales(amax, fmt):
    """fp32 scale values (1 for an all-zero group, which then encodes as
    zeros) and the scales as they are stored: fp32 amax / 448, or the code of
    the smallest power of two s with 448 s >= amax."""
    if fmt == "fp32":
        s = amax / E4M3_MAX
        return torch.where(s == 0, torch.ones_like(s), s), s
    m, e = torch.frexp(amax.double() / E4M3_MAX)
    code = torch.where(m > 0.5, e, e - 1) + 127
    code = torch.where(amax == 0, torch.zeros_like(code), code.clamp(0, 254))
    return torch.exp2((code - 127).double()).float(), code.to(torch.uint8)


def _rows_codes(x, fmt):
    """fp32 rows [M, K] -> E4M3 bytes [M, K] and stored scales [M, K / 128]."""
    M, K = x.shape
    b = x.view(M, K // GROUP, GROUP)
    s, stored = _scales(b.abs().amax(dim=2), fmt)
    q = (b / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(M, K).view(torch.uint8), stored


def _scale_values(stored):
    if stored.dtype == torch.float32:
        return stored
    return torch.exp2((stored.to(torch.int32) - 127).double()).float()


def _wide(q, stored):
    """E4M3 bytes [..., N, K] with one scale per 128 x 128 block, in fp32."""
    s = _scale_values(stored)
    N, K = q.shape[-2:]
    w = q.view(torch.float8_e4m3fn).float().view(*q.shape[:-2], N // GROUP, GROUP, K // GROUP, GROUP)
    return w.mul_(s[..., :, None, :, None]).view(*q.shape[:-2], N, K)


def _wide_rows(q, stored):
    s = _scale_values(stored)
    M, K = q.shape
    return (q.view(torch.float8_e4m3fn).float().view(M, K // GROUP, GROUP) * s[..., None]).view(M, K)


def _norm_out(q, s, y, r):
    """Outputs of the norm: 8-bit values as the types that they stand for."""
    s = s if s.dtype == torch.float32 else s.view(torch.float8_e8m0fnu)
    out = {"q": q.view(torch.float8_e4m3fn), "s": s}
    if y is not None:
        out["y"] = y
    if r is not None:
        out["residual"] = r
    return out


def _norm(st):
    r = None
    v = st["x"].float()
    if st["res"] is not None:
        r = (v + st["res"].float()).to(torch.bfloat16)
        v = r.float()
    rstd = torch.rsqrt(v.square().mean(dim=1, keepdim=True) + EPS)
    n = v * rstd * st["weight"].float()
    q, s = _rows_codes(n, st["fmt"])
    return _norm_out(q, s, n.to(torch.bfloat16) if st["y"] else None, r)


def _route(st):
    x = st["logits"].float()
    M, E = x.shape
    dead = torch.isneginf(x) | torch.isnan(x)
    by_score = st["b"] is not None or st["n_group"] > 1
    if by_score:   # the order of close scores is decided in 64 bits
        key = torch.sigmoid(x.double())
        if st["b"] is not None:
            key = key + st["b"].double()
    else:
        key = x
    key = key.masked_fill(dead, -math.inf)
    if st["n_group"] > 1:
        G, per = st["n_group"], E // st["n_group"]
        two = key.view(M, G, per).sort(dim=2, descending=True).values[..., :2]
        total = two[..., 0]
        if per > 1:
            total = total + two[..., 1].masked_fill(torch.isneginf(two[..., 1]), 0.0)
        best = total.sort(dim=1, descending=True, stable=True).indices[:, : st["topk_group"]]
        open_ = torch.zeros(M, G, dtype=torch.bool, device=x.device).scatter_(1, best, True)
        key = key.masked_fill(~open_.repeat_interleave(per, dim=1), -math.inf)
    ranked = key.sort(dim=1, descending=True, stable=True)
    ids = ranked.indices[:, : st["top_k"]]
    none = torch.isneginf(ranked.values[:, : st["top_k"]])
    if st["scoring"] == "sigmoid":
        w = torch.sigmoid(x)
    else:
        top = x.masked_fill(dead, -math.inf).amax(dim=1, keepdim=True)
        w = torch.exp(x - top).masked_fill(dead, 0.0)
        w = w / w.sum(dim=1, keepdim=True)
    w = w.gather(1, ids).masked_fill(none, 0.0)
    if st["renorm"]:
        w = w / (w.sum(dim=1, keepdim=True) + 1e-20)
    return {"ids": ids.masked_fill(none, -1).to(torch.int32), "weights": w * st["scale"]}


def _swiglu(gu):
    g, u = gu.chunk(2, dim=-1)
    return g / (1.0 + torch.exp(-g)) * u


def _moe(st):
    a = _wide_rows(st["qa"], st["sa"])
    M, k = st["ids"].shape
    E, I, fmt = st["E"], st["I"], st["fmt"]
    local = st["ids"].long() - st["first"]
    here = (local >= 0) & (local < E)
    w = st["weights"].masked_fill(~here, 0.0)
    local = local.clamp(0, E - 1)
    if M * k <= E:   # few tokens: one copy of the weights for each choice
        pick = local.view(-1)
        gu = torch.bmm(_wide(st["qg"][pick], st["sg"][pick]),
                       a.repeat_interleave(k, dim=0)[:, :, None])[..., 0]
        h = _wide_rows(*_rows_codes(_swiglu(gu), fmt))
        d = torch.bmm(_wide(st["qd"][pick], st["sd"][pick]), h[:, :, None])[..., 0]
        y = (d.view(M, k, -1) * w[..., None]).sum(dim=1)
    else:            # every expert on every token, weighted
        gu = torch.matmul(a, _wide(st["qg"], st["sg"]).transpose(1, 2))
        h = _wide_rows(*_rows_codes(_swiglu(gu).view(E * M, I), fmt)).view(E, M, I)
        d = torch.bmm(h, _wide(st["qd"], st["sd"]).transpose(1, 2))
        share = torch.zeros(M, E, device=a.device).scatter_add_(1, local, w)
        y = (d * share.t()[..., None]).sum(dim=0)
    return y.to(torch.bfloat16)


def run(state):
    st = state
    if own:
        import fp8_block_scaled_group128_b200 as fb
        if st["op"] == "norm":
            norm = fb.fp8_add_rmsnorm_quant if st["fmt"] == "fp32" else fb.fp8_add_rmsnorm_quant_ue8m0
            q, s, y, r = norm(st["x"], residual=st["res"], weight=st["weight"], eps=EPS,
                              want_y=st["y"])
            return _norm_out(q, s, y, r)
        if st["op"] == "route":
            ids, w = fb.moe_route_topk(st["logits"], st["top_k"], scoring=st["scoring"],
                                       bias=st["b"], n_group=st["n_group"],
                                       topk_group=st["topk_group"], renormalize=st["renorm"],
                                       scale=st["scale"])
            return {"ids": ids, "weights": w}
        moe = fb.fp8_moe_mlp if st["fmt"] == "fp32" else fb.fp8_moe_mlp_ue8m0
        return moe(st["qa"], st["sa"], st["ids"], st["weights"], st["qg"], st["sg"], st["qd"],
                   st["sd"], first_expert=st["first"])
    if st["op"] == "norm":
        return _norm(st)
    if st["op"] == "route":
        return _route(st)
    return _moe(st)


# ----------------------------------------------------------- 64-bit values --
def _grid(v):
    """64-bit values rounded to the nearest E4M3 value (ties to even),
    saturating at 448: steps of 2^(e - 3) in [2^e, 2^(e + 1)), and of 2^-9 below
    2^-6."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3.0)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_rows(n, fmt):
    """64-bit rows -> E4M3 values (64-bit) and scale values [rows, groups]."""
    R, K = n.shape
    amax = n.abs().view(R, K // GROUP, GROUP).amax(dim=2)
    if fmt == "fp32":
        s = amax / E4M3_MAX
    else:
        p = torch.ceil(torch.log2(amax / E4M3_MAX))
        p = torch.where(torch.exp2(p - 1) * E4M3_MAX >= amax, p - 1, p)
        p = torch.where(torch.exp2(p) * E4M3_MAX < amax, p + 1, p)
        s = torch.exp2(torch.where(amax == 0, torch.full_like(p, -127.0), p).clamp(-127, 127))
    div = torch.where(s == 0, torch.ones_like(s), s).repeat_interleave(GROUP, dim=1)
    return _grid(n / div), s


def _value64(bytes_):
    """E4M3 bytes -> 64-bit values from the format's definition."""
    b = torch.arange(256, dtype=torch.float64)
    mant, ex = b % 8, torch.div(b, 8, rounding_mode="floor") % 16
    v = torch.where(ex == 0, mant * 2.0 ** -9, (8.0 + mant) * torch.exp2(ex - 10.0))
    v = torch.where(b >= 128, -v, v).to(bytes_.device)
    return v[bytes_.long()]


def _exact_weight(q, stored):
    s = stored.double() if stored.dtype == torch.float32 else torch.exp2(stored.double() - 127.0)
    s = s.repeat_interleave(GROUP, dim=0).repeat_interleave(GROUP, dim=1)
    return _value64(q).mul_(s)


def _exact_norm(st):
    out = {}
    v = st["x"].double()
    if st["res"] is not None:
        out["residual"] = (v + st["res"].double()).to(torch.bfloat16).double()
        v = out["residual"]
    n = v / torch.sqrt((v * v).sum(dim=1, keepdim=True) / st["K"] + EPS) * st["weight"].double()
    out["q"], out["s"] = _exact_rows(n, st["fmt"])
    if st["y"]:
        out["y"] = n
    return out


def _exact_route(st):
    x = st["logits"].double().cpu().numpy()
    M, E = x.shape
    dead = np.isneginf(x) | np.isnan(x)
    safe = np.where(dead, 0.0, x)
    sig = 1.0 / (1.0 + np.exp(-safe))
    by_score = st["b"] is not None or st["n_group"] > 1
    key = sig if by_score else safe
    if st["b"] is not None:
        key = key + st["b"].double().cpu().numpy()
    key = np.where(dead, -np.inf, key)
    if st["n_group"] > 1:
        G, per = st["n_group"], E // st["n_group"]
        two = -np.sort(-key.reshape(M, G, per), axis=2)[:, :, :2]
        two[:, :, 1:][np.isneginf(two[:, :, 1:])] = 0.0
        rank = np.argsort(-two.sum(axis=2), axis=1, kind="stable")
        closed = np.ones((M, G), bool)
        np.put_along_axis(closed, rank[:, : st["topk_group"]], False, axis=1)
        key = np.where(np.repeat(closed, per, axis=1), -np.inf, key)
    ids = np.argsort(-key, axis=1, kind="stable")[:, : st["top_k"]]
    none = np.isneginf(np.take_along_axis(key, ids, axis=1))
    if st["scoring"] == "sigmoid":
        w = sig
    else:
        top = np.where(dead, -np.inf, x).max(axis=1, keepdims=True)
        w = np.where(dead, 0.0, np.exp(safe - np.where(np.isneginf(top), 0.0, top)))
        total = w.sum(axis=1, keepdims=True)
        w = w / np.where(total == 0.0, 1.0, total)
    w = np.where(none, 0.0, np.take_along_axis(w, ids, axis=1))
    if st["renorm"]:
        w = w / (w.sum(axis=1, keepdims=True) + 1e-20)
    return {"ids": np.where(none, -1, ids).astype(np.int32), "weights": w * st["scale"]}


def _exact_moe(st):
    qa, sa = st["qa"], st["sa"]
    sv = sa.double() if sa.dtype == torch.float32 else torch.exp2(sa.double() - 127.0)
    a = _value64(qa) * sv.repeat_interleave(GROUP, dim=1)
    y = torch.zeros(st["M"], st["K"], dtype=torch.float64, device=a.device)
    ids = st["ids"].long() - st["first"]
    for e in range(st["E"]):
        share = (st["weights"].double() * (ids == e)).sum(dim=1)
        rows = torch.nonzero((ids == e).any(dim=1)).view(-1)
        if rows.numel() == 0:
            continue
        gu = a[rows] @ _exact_weight(st["qg"][e], st["sg"][e]).T
        g, u = gu[:, : st["I"]], gu[:, st["I"]:]
        v, s = _exact_rows(g * torch.sigmoid(g) * u, st["fmt"])
        d = (v * s.repeat_interleave(GROUP, dim=1)) @ _exact_weight(st["qd"][e], st["sd"][e]).T
        y[rows] += share[rows, None] * d
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] == "norm":
        return _exact_norm(st)
    if st["op"] == "route":
        return _exact_route(st)
    return _exact_moe(st)
