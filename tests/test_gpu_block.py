"""Operators around the layer on the GPU against the float64 oracle
(oracle/block.py): grouped routing, the norms around the block, adapters, and a
run of them together with the layer's own steps.

Tolerances come from the arithmetic: `U[t]` is the half step of one rounding to
the element type, EPS = 2^-23 a float32 rounding of either kind (a matrix
instruction may truncate), and each bound counts the roundings on its path.
"""
import math

import numpy as np
import pytest
import torch

import mixture_experts_layer_token_amd as moe
import oracle
from oracle import block
from workloads import to_f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
EPS = 2.0 ** -23


def _randn(gen, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _within(got, ref, bound):
    err = np.abs(to_f64(got) - ref)
    bad = ~(err <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size}, worst {np.nanmax(err / np.maximum(bound, 1e-300)):.3g} bounds"


# ------------------------------------------------------------ grouped routing

def _route(x, w, k, k_max, rule, *, rb=None, sb=None, scale=1.0, router="auto", policy="exact", stream=None, ws=None):
    T, d = x.shape
    E = w.shape[0]
    desc = moe.make_desc(T, d, E, 128, k_max, dtype=x.dtype, routed_scale=scale, router=router, k_policy=policy)
    if ws is None:
        ws = moe.alloc_workspace(desc, moe.MOE_OP_ROUTE_GROUPED, DEV)
    n = max(T * k_max, 1)
    off = torch.full((T + 1,), -7, dtype=torch.int32, device=DEV)
    ids = torch.full((n,), -7, dtype=torch.int32, device=DEV)
    wts = torch.full((n,), -7.0, device=DEV)
    status = torch.full((1,), -7, dtype=torch.int32, device=DEV)
    moe.moe_route_grouped(desc, rule, x, w, rb, sb, k, off, ids, wts, status, ws, stream)
    torch.cuda.synchronize()
    return off.cpu().numpy(), ids.cpu().numpy(), to_f64(wts), int(status)


def _weight_bound(x, w, ref_w, off):
    """Relative error a weight may have: two roundings (its logit's, its own; exp and
    the divisions are float64), and in bf16, where the logits may come from sums of
    64 products in float32, twice the logit's error: at most 66 * 2^-23 (64 additions
    that may truncate, second-order terms) + 2^-24 (a stored slice) of sum |x_i w_i|
    <= |x| |w|; a sigmoid or a softmax moves by at most that factor, and so does the
    sum it is divided by."""
    r = np.zeros(len(off) - 1)
    if x.dtype == torch.bfloat16:
        r = (66 * 2.0 ** -23 + 2.0 ** -24) * np.linalg.norm(to_f64(x), axis=1) * np.linalg.norm(to_f64(w), axis=1).max()
    r = np.repeat(r, np.diff(off))
    return np.abs(ref_w) * (2 * EPS + 2.02 * np.expm1(r)) + 1e-38


def _check_route(x, w, k, k_max, rb=None, sb=None, scale=1.0, router="auto", policy="exact", **kw):
    off, ids, wts, status = _route(x, w, k, k_max, moe.make_route_rule(**kw), rb=rb, sb=sb, scale=scale, router=router,
                                   policy=policy)
    ke, bad = oracle.execution_budgets(to_f64(k), k_max, policy)
    ref = block.route_grouped(to_f64(x), to_f64(w), to_f64(rb), to_f64(sb), ke, scale=scale, **kw)
    A = int(ref["tok_off"][-1])
    assert status == bad
    np.testing.assert_array_equal(off, ref["tok_off"])
    np.testing.assert_array_equal(ids[:A], ref["ids"])
    assert (np.abs(wts[:A] - ref["w"]) <= _weight_bound(x, w, ref["w"], ref["tok_off"])).all()
    assert (ids[A:] == -7).all() and (wts[A:] == -7.0).all()
    return ref


RULES = [
    dict(score="sigmoid", n_group=8, topk_group=4, group_score="top2", renorm=True),
    dict(score="sigmoid", n_group=1, topk_group=1, group_score="max", renorm=False),
    dict(score="softmax", n_group=8, topk_group=3, group_score="max", renorm=False),
    dict(score="softmax", n_group=4, topk_group=4, group_score="top2", renorm=True),
]


@pytest.mark.parametrize("rule", range(len(RULES)))
@pytest.mark.parametrize("dtype,T,d,E,k_max", [
    ("bf16", 1, 256, 64, 8), ("f32", 3, 128, 64, 5), ("bf16", 65, 1152, 256, 8), ("f32", 130, 256, 200, 24),
    ("bf16", 129, 384, 24, 6), ("bf16", 33, 128, 1024, 40), ("f32", 9, 128, 512, 7), ("bf16", 1500, 2048, 256, 8)])
def test_route_grouped(rule, dtype, T, d, E, k_max):
    g = _gen(T + d + E)
    x, w = _randn(g, T, d, dtype=DT[dtype]), _randn(g, E, d, dtype=DT[dtype], std=d ** -0.5)
    k = torch.randint(0, min(k_max, 9) + 1, (T,), generator=g, device=DEV, dtype=torch.int32)
    k[T // 2] = min(k_max, E // 8)
    sb = (torch.rand(E, generator=g, device=DEV) - 0.5) * 0.1
    _check_route(x, w, k, min(k_max, E // 8 * RULES[rule]["topk_group"]) if RULES[rule]["n_group"] == 8 else k_max,
                 sb=sb if rule != 2 else None, rb=sb if rule == 1 else None, scale=2.5, **RULES[rule])


@pytest.mark.parametrize("n_group,keep,E", [(64, 5, 64), (64, 64, 128), (7, 3, 7), (3, 2, 96), (5, 4, 35), (33, 10, 99)])
@pytest.mark.parametrize("gs", ["max", "top2"])
def test_group_shapes(n_group, keep, E, gs):
    g = _gen(E)
    x, w = _randn(g, 40, 128), _randn(g, E, 128, std=0.1)
    k_max = min(6, keep * (E // n_group))
    k = torch.full((40,), k_max, dtype=torch.int32, device=DEV)
    _check_route(x, w, k, k_max, score="sigmoid", n_group=n_group, topk_group=keep, group_score=gs, renorm=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_route_grouped_ties_and_masks(dtype):
    """Equal logits everywhere (a zero token, repeated router rows), experts and
    whole groups out of service, a token with no expert left, forced experts."""
    g = _gen(5)
    E, d = 32, 128
    x = _randn(g, 12, d, dtype=DT[dtype])
    x[3] = 0
    w = _randn(g, E, d, dtype=DT[dtype], std=d ** -0.5)
    w[5:20] = w[4]
    k = torch.tensor([0, 1, 2, 8, 8, 3, 4, 8, 7, 8, 1, 8], dtype=torch.int32, device=DEV)
    inf = math.inf
    masks = {"none": {}, "some": {0: -inf, 9: -inf, 31: -inf}, "group": dict.fromkeys(range(8, 16), -inf),
             "few": dict.fromkeys(range(2, 32), -inf), "all": dict.fromkeys(range(32), -inf),
             "nan": {4: math.nan, 7: -inf}, "forced": {30: inf, 2: inf, 17: inf}, "lowest": {1: -3.0e38, 6: -3.0e38}}
    for name, m in masks.items():
        sb = torch.zeros(E, device=DEV)
        for e, v in m.items():
            sb[e] = v
        for rule in RULES:
            rule = {**rule, "n_group": min(rule["n_group"], 4), "topk_group": min(rule["topk_group"], 2)}
            _check_route(x, w, k, 8, sb=sb, **rule)


def test_route_grouped_values_that_are_no_numbers():
    """A token with a NaN or an infinity is routed by what its scores still say and
    leaves the others as they are."""
    g = _gen(6)
    x, w = _randn(g, 6, 128), _randn(g, 16, 128, std=0.1)
    k = torch.full((6,), 4, dtype=torch.int32, device=DEV)
    x2 = x.clone()
    x2[1, 5] = math.nan
    x2[4, 7] = math.inf
    for score in ("sigmoid", "softmax"):
        rule = moe.make_route_rule(score=score)
        off, ids, wts, _ = _route(x, w, k, 4, rule)
        _, ids2, wts2, _ = _route(x2, w, k, 4, rule)
        keep = np.repeat([True, False, True, True, False, True], 4)
        np.testing.assert_array_equal(ids[keep], ids2[keep])
        np.testing.assert_array_equal(wts[keep], wts2[keep])
        assert (ids2[4:8] == -1).all() and (wts2[4:8] == 0).all()
        if score == "softmax":
            assert (ids2[16:20] == -1).all()


@pytest.mark.parametrize("router", ["float64", "screened"])
@pytest.mark.parametrize("low", [-3.4028234663852886e38, -1e4, -3.0])
def test_route_grouped_large_biases(router, low):
    """Experts pushed away by the type's lowest value or a smaller constant: alone, in a
    whole group, against each other (the sum of two is below float32), and biases so
    large that a float32 key would lose the scores."""
    g = _gen(17)
    x, w = _randn(g, 40, 512, dtype=torch.bfloat16), _randn(g, 64, 512, dtype=torch.bfloat16, std=512 ** -0.5)
    k = torch.randint(0, 9, (40,), generator=g, device=DEV, dtype=torch.int32)
    for away in ([0, 9, 63], list(range(8, 24)) + [3], list(range(64)), list(range(5, 64))):
        sb = (torch.rand(64, generator=g, device=DEV) - 0.5) * 0.1
        sb[away] = low
        for gs in ("top2", "max"):
            _check_route(x, w, k, 8, sb=sb, router=router, score="sigmoid", n_group=8, topk_group=3, group_score=gs,
                         renorm=True)
        _check_route(x, w, k, 8, sb=sb, router=router, score="softmax", n_group=8, topk_group=3, group_score="top2",
                     renorm=False)
    sb = torch.full((64,), 1e4, device=DEV) + (torch.rand(64, generator=g, device=DEV) * 1e-2)
    _check_route(x, w, k, 8, sb=sb, router=router, **RULES[0])


@pytest.mark.parametrize("T", [0, 1])
def test_route_grouped_empty(T):
    x, w = torch.zeros(T, 128, device=DEV), torch.zeros(8, 128, device=DEV)
    k = torch.zeros(T, dtype=torch.int32, device=DEV)
    off, ids, _, status = _route(x, w, k, 2, moe.make_route_rule())
    assert status == 0 and (off == 0).all() and (ids == -7).all()


def test_route_grouped_bad_budgets_and_policies():
    g = _gen(8)
    x, w = _randn(g, 70, 128, dtype=torch.bfloat16), _randn(g, 16, 128, dtype=torch.bfloat16)
    k = torch.randint(0, 5, (70,), generator=g, device=DEV, dtype=torch.int32)
    _check_route(x, w, k, 4, policy="batch_max", **RULES[1])
    k[3], k[69] = -1, 5
    _check_route(x, w, k, 4, **RULES[1])


@pytest.mark.parametrize("T,d,E", [(600, 7168, 256), (2048, 1024, 96), (70, 4096, 512), (64, 128, 8)])
@pytest.mark.parametrize("rule", range(len(RULES)))
def test_route_grouped_routers_agree(T, d, E, rule):
    """The screened router takes the float64 one's decisions, close ones included
    (router rows that repeat, and rows that differ in one last place)."""
    g = _gen(T)
    x, w = _randn(g, T, d, dtype=torch.bfloat16), _randn(g, E, d, dtype=torch.bfloat16, std=d ** -0.5)
    w[E // 2] = w[1]
    w[E - 1] = w[2]
    w[E - 1, :3] += 2.0 ** -8 * w[2, :3]
    sb = torch.zeros(E, device=DEV)
    k = torch.randint(0, 9, (T,), generator=g, device=DEV, dtype=torch.int32).clamp(max=E // 8 * 3)
    kw = dict(sb=sb, scale=2.5)
    a = _route(x, w, k, min(8, E // 8 * 3), moe.make_route_rule(**RULES[rule]), router="float64", **kw)
    b = _route(x, w, k, min(8, E // 8 * 3), moe.make_route_rule(**RULES[rule]), router="screened", **kw)
    np.testing.assert_array_equal(a[0], b[0])
    np.testing.assert_array_equal(a[1], b[1])
    A = int(a[0][-1])
    assert (np.abs(a[2][:A] - b[2][:A]) <= 2 * _weight_bound(x, w, a[2][:A], a[0])).all()


@pytest.mark.parametrize("T,d,E,k_max,rule", [(4200, 1024, 256, 8, 0), (900, 8192, 160, 8, 0), (2100, 2048, 272, 70, 3),
                                              (1100, 1024, 1024, 9, 2)])
def test_route_grouped_large_batches(T, d, E, k_max, rule):
    """AUTO's matrix-instruction logits (T * E * d >= 2^30) against the oracle: scaled
    tokens (wide and narrow radius), equal and nearly equal experts, some out of service."""
    g = _gen(T + E)
    x, w = _randn(g, T, d, dtype=torch.bfloat16), _randn(g, E, d, dtype=torch.bfloat16, std=d ** -0.5)
    x[::7] *= 8
    x[1::7] *= 2.0 ** -6
    x[5] = 0
    w[E // 3] = w[0]
    w[E // 2] = w[2]
    w[E // 2, 5] += 2.0 ** -9
    k = torch.randint(0, k_max + 1, (T,), generator=g, device=DEV, dtype=torch.int32)
    sb = None
    if RULES[rule]["score"] == "sigmoid":
        sb = (torch.rand(E, generator=g, device=DEV) - 0.5) * 0.1
        sb[7] = -math.inf
    _check_route(x, w, k, k_max, sb=sb, scale=2.5, **RULES[rule])


# ---------------------------------------------------------------------- norms

def _norm_bound(v, dv, w, b, kind, eps, off):
    """Bound on the error of norm(v) when v is off by at most dv: the sums of the
    statistics have under 128 roundings on any path (16 chunk elements and up to
    64 of a chunk, 6 steps of the butterfly, 16 waves, the quotient and root)."""
    c = 128 * EPS
    m = v.mean(1, keepdims=True) if kind == "layer" else 0.0
    dm = dv.mean(1, keepdims=True) + c * np.abs(v).mean(1, keepdims=True) if kind == "layer" else 0.0
    u = v - m
    rs = 1.0 / np.sqrt((u * u).mean(1, keepdims=True) + eps)
    du = dv + dm + EPS * np.abs(u)
    dstat = np.sqrt((du * du).mean(1, keepdims=True)) * rs
    wf = np.abs(off + (0.0 if w is None else w)) if w is not None else 1.0
    return wf * rs * (du + np.abs(u) * (2 * dstat + c)) * 1.01 + 4 * EPS * (0.0 if b is None else np.abs(b)), \
        block.norm(v, w, b, kind=kind, eps=eps, w_offset=off)


def _norm_case(seed, dtype, T, d, kind, post, gate, bias, weights=True, resid=True, scale=1.0):
    g = _gen(seed)
    dt = DT[dtype]
    t = {"y": _randn(g, T, d, dtype=dt, std=scale), "resid": _randn(g, T, d, dtype=dt, std=scale) if resid else None}
    for n in ("post_w", "pre_w"):
        t[n] = _randn(g, d, dtype=dt) if weights and (post or n == "pre_w") else None
    for n in ("post_b", "pre_b"):
        t[n] = _randn(g, d, dtype=dt) if bias and (post or n == "pre_b") else None
    t["gate"] = {"none": None, "channel": lambda: _randn(g, d, dtype=dt), "token": lambda: _randn(g, T, dtype=dt),
                 "full": lambda: _randn(g, T, d, dtype=dt)}[gate]
    t["gate"] = t["gate"] and t["gate"]()
    return t


def _norm_check(t, dtype, kind, post, gate, alpha, off, eps, r, x, y64=None, dy=0.0):
    f = {n: to_f64(v) for n, v in t.items()}
    y = f["y"] if y64 is None else y64
    dy = np.zeros_like(y) + dy
    if post:
        dp, p = _norm_bound(y, dy, f["post_w"], f["post_b"], kind, eps, off)
    else:
        dp, p = dy, y
    gt = 1.0 if f["gate"] is None else (f["gate"][:, None] if gate == "token" else f["gate"])
    rr = (0.0 if f["resid"] is None else f["resid"]) + alpha * gt * p
    dr = np.abs(alpha * gt) * dp + 4 * EPS * (np.abs(alpha * gt * p) + np.abs(rr))
    if r is not None:
        _within(r, rr, dr + U[dtype] * (np.abs(rr) + dr) * 1.01 + 1e-40)
    if x is not None:
        dx, xx = _norm_bound(rr, dr, f["pre_w"], f["pre_b"], kind, eps, off)
        _within(x, xx, dx + U[dtype] * (np.abs(xx) + dx) * 1.01 + 1e-40)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype,T,d", [
    ("bf16", 1, 7168), ("bf16", 5, 8), ("bf16", 3, 1), ("f32", 2, 1), ("bf16", 7, 129), ("f32", 9, 1531),
    ("bf16", 64, 2048), ("f32", 33, 2048), ("bf16", 3, 8200), ("f32", 3, 20000), ("bf16", 2, 40001),
    ("bf16", 2, 65536), ("f32", 2, 65535), ("f32", 2, 65536), ("bf16", 300, 520)])
@pytest.mark.parametrize("gate,post,bias", [("none", False, False), ("channel", True, True), ("token", True, False),
                                            ("full", False, True)])
def test_norm(kind, dtype, T, d, gate, post, bias):
    t = _norm_case(T + d, dtype, T, d, kind, post, gate, bias)
    nd = moe.make_norm_desc(T, d, dtype=DT[dtype], kind=kind, eps=1e-5, alpha=0.5, w_offset=1.0, gate=gate, post=post)
    r, x = torch.empty_like(t["y"]), torch.empty_like(t["y"])
    moe.moe_norm(nd, t["y"], t["resid"], t["post_w"], t["post_b"], t["gate"], t["pre_w"], t["pre_b"], r, x)
    _norm_check(t, dtype, kind, post, gate, 0.5, 1.0, 1e-5, r, x)
    # each output alone has the same bits, and so has either written in place
    for only in ("r", "x"):
        o = torch.empty_like(r)
        moe.moe_norm(nd, t["y"], t["resid"], t["post_w"], t["post_b"], t["gate"], t["pre_w"], t["pre_b"],
                     o if only == "r" else None, o if only == "x" else None)
        assert torch.equal(o, r if only == "r" else x)
    y2, r2 = t["y"].clone(), t["resid"].clone()
    moe.moe_norm(nd, y2, r2, t["post_w"], t["post_b"], t["gate"], t["pre_w"], t["pre_b"], r2, y2)
    assert torch.equal(r2, r) and torch.equal(y2, x)
    y2, r2 = t["y"].clone(), t["resid"].clone()
    moe.moe_norm(nd, y2, r2, t["post_w"], t["post_b"], t["gate"], t["pre_w"], t["pre_b"], y2, r2)
    assert torch.equal(y2, r) and torch.equal(r2, x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_parts_left_out(dtype):
    """The plain norm of the residual, no residual, no weights, large and tiny rows."""
    t = _norm_case(3, dtype, 20, 1000, "rms", True, "none", False)
    nd = moe.make_norm_desc(20, 1000, dtype=DT[dtype])
    x = torch.empty_like(t["y"])
    moe.moe_norm(nd, None, t["resid"], None, None, None, t["pre_w"], None, None, x)
    _norm_check({**t, "y": torch.zeros_like(t["y"])}, dtype, "rms", False, "none", 1.0, 0.0, 1e-6, None, x)
    nd = moe.make_norm_desc(20, 1000, dtype=DT[dtype], post=True, alpha=2.0)
    r = torch.empty_like(x)
    moe.moe_norm(nd, t["y"], None, None, None, None, None, None, r, x)
    _norm_check({**t, "resid": None, "post_w": None, "pre_w": None}, dtype, "rms", True, "none", 2.0, 0.0, 1e-6, r, x)
    for scale in (1e-12, 1e12):
        t = _norm_case(4, dtype, 4, 512, "layer", True, "channel", True, scale=scale)
        nd = moe.make_norm_desc(4, 512, dtype=DT[dtype], kind="layer", post=True, gate="channel")
        r, x = torch.empty_like(t["y"]), torch.empty_like(t["y"])
        moe.moe_norm(nd, t["y"], t["resid"], t["post_w"], t["post_b"], t["gate"], t["pre_w"], t["pre_b"], r, x)
        _norm_check(t, dtype, "layer", True, "channel", 1.0, 0.0, 1e-6, r, x)


def test_norm_rows_do_not_meet():
    """A row of infinities or NaN leaves its neighbours' bits alone; a row of zeros
    stays finite."""
    t = _norm_case(5, "bf16", 6, 768, "rms", True, "none", False)
    nd = moe.make_norm_desc(6, 768, post=True)
    out = []
    for bad in (False, True):
        y = t["y"].clone()
        y[3] = 0
        if bad:
            y[1], y[4, 5] = math.inf, math.nan
        r, x = torch.empty_like(y), torch.empty_like(y)
        moe.moe_norm(nd, y, t["resid"], t["post_w"], None, None, t["pre_w"], None, r, x)
        out.append((r, x))
    for a, b in zip(*out):
        assert torch.equal(a[[0, 2, 3, 5]], b[[0, 2, 3, 5]])
        assert torch.isfinite(a).all() and torch.isnan(b[4]).all()


def _combine_case(seed, dtype, T, d, k_max, shared, holes):
    g = _gen(seed)
    k = torch.randint(0, k_max + 1, (T,), generator=g, device=DEV, dtype=torch.int32)
    off = torch.zeros(T + 1, dtype=torch.int32, device=DEV)
    off[1:] = torch.cumsum(k, 0)
    A, cap = int(off[-1]), max(T * k_max, 1)
    inv = torch.full((cap,), 1 << 30, dtype=torch.int32, device=DEV)
    inv[:A] = torch.randperm(A, generator=g, device=DEV).int()
    if holes and A > 4:
        inv[torch.randint(0, A, (3,), generator=g, device=DEV)] = -1
    return dict(y_perm=_randn(g, cap, d, dtype=DT[dtype]), y_shared=_randn(g, T, d, dtype=DT[dtype]) if shared else None,
                tok_off=off, w=torch.rand(cap, generator=g, device=DEV), inv=inv)


@pytest.mark.parametrize("dtype,T,d,k_max,shared", [
    ("bf16", 1, 7168, 8, True), ("bf16", 37, 256, 3, False), ("f32", 20, 2048, 8, True), ("bf16", 9, 4096, 20, True),
    ("f32", 5, 16512, 2, False), ("bf16", 4, 65536, 4, True), ("f32", 3, 65536, 3, True), ("bf16", 260, 128, 33, True)])
@pytest.mark.parametrize("kind,post,gate", [("rms", True, "channel"), ("layer", False, "token"), ("rms", False, "none")])
def test_combine_norm(dtype, T, d, k_max, shared, kind, post, gate):
    c = _combine_case(T * k_max + d, dtype, T, d, k_max, shared, True)
    t = _norm_case(d, dtype, T, d, kind, post, gate, kind == "layer")
    desc = moe.make_desc(T, d, max(k_max, 2), 128, k_max, dtype=DT[dtype])
    nd = moe.make_norm_desc(T, d, dtype=DT[dtype], kind=kind, post=post, gate=gate, alpha=0.75)
    r, x = torch.empty_like(t["y"]), torch.empty_like(t["y"])
    args = (c["y_perm"], c["y_shared"], c["tok_off"], c["w"], c["inv"])
    ops = (t["post_w"], t["post_b"], t["gate"], t["pre_w"], t["pre_b"])
    moe.moe_combine_norm(desc, nd, *args, t["resid"], *ops, r, x)
    h = {n: None if v is None else v.cpu().numpy() if v.dtype == torch.int32 else to_f64(v) for n, v in c.items()}
    y = block.combine(h["y_perm"], h["y_shared"], h["tok_off"], h["w"], h["inv"], T, d)
    ay = block.combine(np.abs(h["y_perm"]), None if h["y_shared"] is None else np.abs(h["y_shared"]), h["tok_off"],
                       h["w"], h["inv"], T, d)
    _norm_check(t, dtype, kind, post, gate, 0.75, 0.0, 1e-6, r, x, y64=y, dy=(k_max + 2) * EPS * ay)
    r2 = t["resid"].clone()
    x2 = torch.empty_like(x)
    moe.moe_combine_norm(desc, nd, *args, r2, *ops, r2, x2)
    assert torch.equal(r2, r) and torch.equal(x2, x)


def test_combine_norm_is_combine_then_add():
    """Without norms and residual it is moe_combine bit for bit."""
    c = _combine_case(1, "bf16", 50, 1024, 9, True, True)
    desc = moe.make_desc(50, 1024, 16, 128, 9)
    a, b = (torch.empty(50, 1024, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    moe.moe_combine(desc, c["y_perm"], c["y_shared"], c["tok_off"], c["w"], c["inv"], a)
    moe.moe_combine_norm(desc, moe.make_norm_desc(50, 1024), c["y_perm"], c["y_shared"], c["tok_off"], c["w"], c["inv"],
                         None, None, None, None, None, None, b, None)
    assert torch.equal(a, b)


# ------------------------------------------------------------------- adapters

def _adapt_case(seed, dtype, T, K, N, R, L, G=1, k_max=1, mapped=False, order="random"):
    g = _gen(seed)
    dt = DT[dtype]
    rows = T * k_max
    t = dict(a=_randn(g, L, G, R, K, dtype=dt, std=K ** -0.5), b=_randn(g, L, G, N, R, dtype=dt),
             ranks=torch.randint(0, R + 1, (L,), generator=g, device=DEV, dtype=torch.int32),
             scales=_randn(g, L), adapter_ids=torch.randint(-1, L + 1, (T,), generator=g, device=DEV, dtype=torch.int32),
             row_tok=None, x_rows=None, expert_off=None)
    if order == "one":
        t["adapter_ids"][:] = L - 1
    elif order == "none":
        t["adapter_ids"][:] = -1
    elif order == "runs":
        t["adapter_ids"] = t["adapter_ids"].sort().values.contiguous()
    t["ranks"][-1] = R
    if G > 1 or mapped:
        k = torch.randint(0, k_max + 1, (T,), generator=g, device=DEV).clamp(max=G)
        hit = torch.rand(T, G, generator=g, device=DEV).argsort(1).argsort(1) < k[:, None]
        tok = hit.t().nonzero()[:, 1].int()
        t["row_tok"] = torch.full((rows,), 1 << 29, dtype=torch.int32, device=DEV)
        t["row_tok"][:tok.numel()] = tok
        t["expert_off"] = torch.zeros(G + 1, dtype=torch.int32, device=DEV)
        t["expert_off"][1:] = torch.cumsum(hit.sum(0), 0)
    if mapped:
        t["x_rows"] = t["row_tok"]
    t["x"] = _randn(g, T if mapped else rows, K, dtype=dt)
    t["y"] = _randn(g, rows, N, dtype=dt)
    return t


def _adapt(t, out, dtype, T, ws=None, stream=None):
    L, G, R, K = t["a"].shape
    rows, N = t["y"].shape
    ad = moe.make_adapter_desc(T, rows, K, N, R, L, G, dtype=DT[dtype])
    if ws is None:
        ws = moe.alloc_adapt_workspace(ad, DEV)
    if ws is not None:
        ws.view(torch.int32).fill_(0x7fc0_7fc0)  # NaN wherever a part that was not written is read
    moe.moe_adapt(ad, t["x"], t["x_rows"], t["a"], t["b"], t["ranks"], t["scales"], t["adapter_ids"], t["row_tok"],
                  t["expert_off"], t["y"], out, ws, stream)
    return out


def _adapt_ref(t, dtype):
    f = {n: None if v is None else v.cpu().numpy() if v.dtype == torch.int32 else to_f64(v) for n, v in t.items()}
    kw = dict(ranks=f["ranks"], row_tok=f["row_tok"], x_rows=f["x_rows"], expert_off=f["expert_off"])
    ref = block.adapt(f["y"], f["x"], f["a"], f["b"], f["adapter_ids"], scales=f["scales"], **kw)
    mag = block.adapt(np.zeros_like(f["y"]), np.abs(f["x"]), np.abs(f["a"]), np.abs(f["b"]), f["adapter_ids"],
                      scales=np.abs(f["scales"]), **kw)
    # the first product's K roundings, the second's R (twice: value and remainder),
    # the scale's, and in bf16 what value and remainder together leave out, 2^-16
    K, R = t["a"].shape[3], t["a"].shape[2]
    d = mag * ((K + 2 * R + 4) * EPS + (2.0 ** -16 if dtype == "bf16" else 0.0))
    return ref, d + (U[dtype] * 1.01) * (np.abs(ref) + d) + 1e-40


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,N,R,L,G,k_max,mapped,order", [
    (1, 8, 8, 8, 1, 1, 1, False, "one"), (1, 2048, 1032, 16, 4, 1, 1, False, "one"),
    (17, 136, 72, 24, 5, 1, 1, False, "random"), (33, 520, 264, 128, 3, 1, 1, False, "random"),
    (100, 256, 512, 64, 40, 1, 1, False, "random"), (300, 128, 2056, 40, 6, 1, 1, False, "runs"),
    (64, 128, 128, 16, 3, 1, 1, False, "none"), (50, 256, 128, 16, 3, 9, 4, False, "random"),
    (40, 128, 256, 32, 4, 64, 6, True, "random"), (9, 1000, 24, 8, 2, 1024, 3, False, "random"),
    (70, 64, 64, 16, 6, 1, 1, True, "random"), (5, 4096, 64, 72, 2, 3, 2, False, "one"),
    (8200, 72, 1032, 16, 5, 1, 1, False, "random"), (33000, 16, 1032, 8, 3, 1, 1, False, "runs"),
    (2100, 40, 264, 24, 3, 5, 5, True, "random"), (20, 7168, 512, 96, 2, 1, 1, False, "random")])
def test_adapt(dtype, T, K, N, R, L, G, k_max, mapped, order):
    t = _adapt_case(T + K + R, dtype, T, K, N, R, L, G, k_max, mapped, order)
    ref, bound = _adapt_ref(t, dtype)
    n = len(t["y"]) if t["expert_off"] is None else int(t["expert_off"][-1])
    out = torch.full_like(t["y"], 7.0)
    _adapt(t, out, dtype, T)
    _within(out[:n], ref[:n], bound[:n])
    assert (out[n:] == 7.0).all()
    # rows without an adapter keep y's bits; in place gives the same
    tok = torch.arange(len(out), device=DEV) if t["row_tok"] is None else t["row_tok"].long()
    own = t["adapter_ids"][tok[:n]]
    free = (own < 0) | (own >= L)
    assert torch.equal(out[:n][free], t["y"][:n][free])
    y = t["y"].clone()
    _adapt({**t, "y": y}, y, dtype, T)
    assert torch.equal(y[:n], out[:n]) and torch.equal(y[n:], t["y"][n:])


def test_adapt_requests_do_not_meet():
    """Adapters, stored ranks and rows that hold NaN or infinities change only the
    rows that use them."""
    t = _adapt_case(11, "bf16", 64, 128, 192, 16, 4)
    t["adapter_ids"][:] = torch.arange(64, device=DEV) % 4
    t["ranks"][:] = torch.tensor([16, 5, 16, 0], device=DEV)
    good = _adapt(t, torch.empty_like(t["y"]), "bf16", 64)
    bad = {n: v.clone() if v is not None else None for n, v in t.items()}
    bad["a"][0], bad["b"][0] = math.nan, math.inf
    bad["a"][1, 0, 5:], bad["b"][1, 0, :, 5:] = math.inf, math.nan
    bad["a"][3], bad["b"][3] = math.nan, math.nan
    bad["x"][2], bad["y"][6, 3] = math.nan, math.inf
    got = _adapt(bad, torch.empty_like(t["y"]), "bf16", 64)
    rows = torch.arange(64, device=DEV)
    same = (rows % 4 != 0) & (rows != 2) & (rows != 6)
    assert torch.equal(got[same], good[same])
    assert torch.isnan(got[2]).all() and torch.isnan(got[4]).any()
    assert torch.isinf(got[6, 3]) and torch.equal(got[6, 4:], good[6, 4:])


def test_adapt_ids_and_maps_out_of_range():
    t = _adapt_case(12, "f32", 20, 64, 64, 8, 3, mapped=True)
    t["adapter_ids"][:] = 1
    t["expert_off"][1] = 18
    t["row_tok"] = torch.arange(20, dtype=torch.int32, device=DEV)
    t["x_rows"] = t["row_tok"].clone()
    t["row_tok"][3], t["x_rows"][5], t["x_rows"][6] = 20, -1, 20
    t["adapter_ids"][8], t["adapter_ids"][9] = -2, 1 << 30
    ref, bound = _adapt_ref(t, "f32")
    out = _adapt(t, torch.empty_like(t["y"]).fill_(7.0), "f32", 20)
    _within(out[:18], ref[:18], bound[:18])
    for r in (3, 5, 6, 8, 9):
        assert torch.equal(out[r], t["y"][r])
    assert (out[18:] == 7.0).all()


# --------------------------------------------------- streams, graphs, together

def test_other_stream_and_two_graphs_on_one_workspace():
    """Captured calls replay with new budgets, inputs and ids, in turn with each
    other on the same workspaces and with eager work between, and every replay
    has the eager call's bits."""
    g = _gen(21)
    T, d, E, k_max, L, R = 50, 512, 64, 6, 3, 16
    desc = moe.make_desc(T, d, E, 128, k_max)
    rule = moe.make_route_rule(n_group=8, topk_group=4)
    nd = moe.make_norm_desc(T, d, post=True)
    ad = moe.make_adapter_desc(T, T, d, d, R, L)
    ws, wa = moe.alloc_workspace(desc, moe.MOE_OP_ROUTE_GROUPED, DEV), moe.alloc_adapt_workspace(ad, DEV)
    w, a, b = _randn(g, E, d, dtype=torch.bfloat16), _randn(g, L, 1, R, d, dtype=torch.bfloat16), \
        _randn(g, L, 1, d, R, dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32, device=DEV)

    def buffers():
        return dict(x=torch.zeros(T, d, dtype=torch.bfloat16, device=DEV), k=torch.zeros(T, **i32), ad=torch.zeros(T, **i32),
                    off=torch.zeros(T + 1, **i32), ids=torch.zeros(T * k_max, **i32), wts=torch.zeros(T * k_max, device=DEV),
                    st=torch.zeros(1, **i32), r=torch.zeros(T, d, dtype=torch.bfloat16, device=DEV),
                    n=torch.zeros(T, d, dtype=torch.bfloat16, device=DEV), o=torch.zeros(T, d, dtype=torch.bfloat16, device=DEV))

    def calls(s, stream=None):
        moe.moe_norm(nd, s["x"], s["x"], None, None, None, None, None, s["r"], s["n"], stream)
        moe.moe_route_grouped(desc, rule, s["n"], w, None, None, s["k"], s["off"], s["ids"], s["wts"], s["st"], ws, stream)
        moe.moe_adapt(ad, s["n"], None, a, b, None, None, s["ad"], None, None, s["r"], s["o"], wa, stream)

    sets = [buffers(), buffers()]
    graphs = []
    for s in sets:
        calls(s)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            calls(s)
        graphs.append(gr)
    side = torch.cuda.Stream()
    for step in range(4):
        want = []
        for s in sets:
            s["x"].copy_(_randn(g, T, d, dtype=torch.bfloat16))
            s["k"].copy_(torch.randint(0, k_max + 1, (T,), generator=g, **i32))
            s["ad"].copy_(torch.randint(-1, L, (T,), generator=g, **i32))
            e = buffers()
            for n in ("x", "k", "ad"):
                e[n].copy_(s[n])
            torch.cuda.synchronize()
            if step % 2:
                calls(e, side)
                side.synchronize()
            else:
                calls(e)
            want.append(e)
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for s, e in zip(sets, want):
            A = int(e["off"][-1])
            for n in ("off", "st", "r", "n", "o"):
                assert torch.equal(s[n], e[n]), (step, n)
            assert torch.equal(s["ids"][:A], e["ids"][:A]) and torch.equal(s["wts"][:A], e["wts"][:A])


@pytest.mark.parametrize("adapters,shared_adapters", [(0, 0), (3, 0), (0, 2), (3, 2)])
def test_block_together(adapters, shared_adapters):
    """One block in serving order against the float64 oracle of its steps, the
    layer's own tolerance on the output, and its graph against the eager call."""
    g = _gen(31)
    T, d, E, I, Is, k_max, R = 48, 256, 16, 128, 128, 4, 16
    bf = torch.bfloat16
    desc = moe.make_desc(T, d, E, I, k_max, I_shared=Is, routed_scale=2.5)
    rule = moe.make_route_rule(n_group=4, topk_group=2)
    before = moe.make_norm_desc(T, d)
    behind = moe.make_norm_desc(T, d, post=True, gate="channel", alpha=0.5)
    layer = moe.BlockLayer(desc, rule, before, behind, adapters=adapters, shared_adapters=shared_adapters, rank=R, device=DEV)
    y, resid = _randn(g, T, d, dtype=bf), _randn(g, T, d, dtype=bf)
    w_r, sb = _randn(g, E, d, dtype=bf, std=d ** -0.5), (torch.rand(E, generator=g, device=DEV) - 0.5) * 0.1
    sb[3] = -math.inf
    k = torch.randint(0, k_max + 1, (T,), generator=g, device=DEV, dtype=torch.int32)
    wg, wu = (_randn(g, E, I, d, dtype=bf, std=d ** -0.5) for _ in range(2))
    wd = _randn(g, E, d, I, dtype=bf, std=I ** -0.5)
    sh = [_randn(g, Is, d, dtype=bf, std=d ** -0.5), _randn(g, Is, d, dtype=bf, std=d ** -0.5),
          _randn(g, d, Is, dtype=bf, std=Is ** -0.5)]
    pre_w, post_w, gate, next_w = (_randn(g, d, dtype=bf) for _ in range(4))

    def stack(L, G, K):
        return (_randn(g, L, G, R, K, dtype=bf, std=K ** -0.5), _randn(g, L, G, d, R, dtype=bf, std=0.2), None,
                torch.rand(L, generator=g, device=DEV), torch.randint(-1, L, (T,), generator=g, device=DEV, dtype=torch.int32))

    ra = stack(adapters, E, I) if adapters else None
    sa = stack(shared_adapters, 1, Is) if shared_adapters else None
    r, x = torch.empty(T, d, dtype=bf, device=DEV), torch.empty(T, d, dtype=bf, device=DEV)
    run = lambda: layer.run(y, resid, pre_w, w_r, sb, k, wg, wu, wd, r, x, shared=sh, behind_post_w=post_w,
                            behind_gate=gate, next_w=next_w, adapters=ra, shared_adapters=sa)
    run()
    torch.cuda.synchronize()

    f = to_f64
    # the layer's own rounding points: x and resid in bf16, then H and Y
    mid, xin = f(layer.resid), f(layer.x)
    want_mid, want_x = block.norm_chain(f(y), f(resid), pre=(f(pre_w), None))
    np.testing.assert_allclose(mid, want_mid, rtol=2 * U["bf16"], atol=1e-6)
    np.testing.assert_allclose(xin, want_x, rtol=2 * U["bf16"], atol=1e-6)
    rt = block.route_grouped(xin, f(w_r), None, f(sb), f(k).astype(int), score="sigmoid", n_group=4, topk_group=2, scale=2.5)
    A = len(rt["ids"])
    np.testing.assert_array_equal(layer.ids[:A].cpu().numpy(), rt["ids"])
    out = np.zeros((T, d))
    sig = lambda z: z / (1 + np.exp(-z))

    def expert(v, g_, u_, d_, lora):
        h = sig(g_ @ v) * (u_ @ v)
        o = d_ @ h
        if lora is not None:
            a_, b_, s_ = lora
            o = o + s_ * (b_ @ (a_ @ h))
        return o

    pick = lambda st, t, e: None if st is None or int(st[4][t]) < 0 else (
        f(st[0][int(st[4][t]), e]), f(st[1][int(st[4][t]), e]), float(st[3][int(st[4][t])]))
    for t in range(T):
        for j in range(rt["tok_off"][t], rt["tok_off"][t + 1]):
            e = rt["ids"][j]
            out[t] += rt["w"][j] * expert(xin[t], f(wg[e]), f(wu[e]), f(wd[e]), pick(ra, t, e))
        out[t] += expert(xin[t], *map(f, sh), pick(sa, t, 0))
    want_r, want_next = block.norm_chain(out, mid, post=(f(post_w), None), gate=f(gate), pre=(f(next_w), None), alpha=0.5)
    for got, want in ((r, want_r), (x, want_next)):
        assert np.linalg.norm(f(got) - want) <= 1e-2 * np.linalg.norm(want)

    r1, x1 = r.clone(), x.clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        run()
    for _ in range(3):
        r.zero_()
        x.zero_()
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(r, r1) and torch.equal(x, x1)
    assert torch.isfinite(r).all()
