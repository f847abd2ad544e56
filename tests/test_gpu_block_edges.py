"""Edges of the operators around the layer on the GPU.  Tolerances as in
test_gpu_block.py.  AUTO takes the screened routing of bf16 batches from T * E * d =
3 * 2^28 on."""
import math

import numpy as np
import pytest
import torch

import mixture_experts_layer_token_amd as moe
from tests.test_gpu_block import (DEV, DT, EPS, RULES, U, _adapt, _adapt_ref, _check_route, _gen, _norm_case, _randn,
                                  _route)
from workloads import to_f64

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- adapters

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,R", [(16, 72, 8), (40, 264, 24), (33, 136, 64), (32, 200, 128), (9000, 1032, 16),
                                   (9000, 1032, 128)])
def test_adapt_products_that_are_infinite(dtype, T, N, R):
    """An infinite or very large A x and infinite entries of B give what the
    definition gives: infinities of the product's sign, NaN only where it has one."""
    g = _gen(T + N)
    dt, K = DT[dtype], 64
    t = dict(x=_randn(g, T, K, dtype=dt), a=_randn(g, 3, 1, R, K, dtype=dt, std=K ** -0.5),
             b=_randn(g, 3, 1, N, R, dtype=dt), ranks=torch.tensor([1, 1, R], dtype=torch.int32, device=DEV),
             scales=torch.tensor([1.0, 0.5, -2.0], device=DEV),
             adapter_ids=torch.full((T,), 2, dtype=torch.int32, device=DEV), row_tok=None, x_rows=None,
             expert_off=None, y=_randn(g, T, N, dtype=dt))
    for at in (0, T - 16):
        ids, x = t["adapter_ids"][at:at + 16], t["x"][at:at + 16]
        ids[:10] = 0
        ids[10:12] = 1
        x[0, 5], x[1, 5] = math.inf, -math.inf
        # A x = 2^127 (2 - 2^-7) + 2^120 3/4: finite, above half a step behind bf16's largest value
        x[2] = 0
        x[2, 0], x[2, 1] = 2.0 ** 127 * (2 - 2.0 ** -7), 2.0 ** 120 * 0.75
        x[3] = -x[2]
        x[4], x[5] = 0, 0
        x[4, 0] = 1.5                              # A x is a bf16 value: no remainder
        x[5, 0], x[5, 1] = 1.0, 2.0 ** -8 * 1.75   # rounded up: a remainder of the other sign
        x[6], x[7] = -x[5], 0
        x[7, 0], x[7, 1] = 1.0, 2.0 ** -8 * 0.5
    t["a"][0, 0, 0] = 0
    t["a"][0, 0, 0, :2] = 1.0
    t["a"][0, 0, 0, 5] = 0.25
    t["b"][0, 0, :, 0] *= 2.0 ** -30
    t["b"][0, 0, 3, 0], t["b"][0, 0, 4, 0], t["b"][0, 0, N - 1, 0] = math.inf, -math.inf, math.inf
    t["b"][0, 0, 6, 0] = 0
    t["b"][1, 0, 5, 0] = -math.inf
    t["b"][2, 0, 7, R - 1], t["b"][2, 0, 9, 2] = math.inf, -math.inf
    with np.errstate(invalid="ignore"):
        ref, bound = _adapt_ref(t, dtype)
    assert np.isnan(ref[0, 6]) and np.isposinf(ref[5, 3]) and np.isneginf(ref[6, 3]) and np.isfinite(ref[2, 0])
    got = to_f64(_adapt(t, torch.empty_like(t["y"]), dtype, T))
    sure = np.isfinite(ref)
    np.testing.assert_array_equal(got[~sure], ref[~sure])
    assert (np.abs(got[sure] - ref[sure]) <= bound[sure]).all()
    y = t["y"].clone()
    np.testing.assert_array_equal(to_f64(_adapt({**t, "y": y}, y, dtype, T)), got)


# ------------------------------------------------------------ grouped routing

@pytest.mark.parametrize("rule", [0, 1, 3])
@pytest.mark.parametrize("xs,ws", [(0, 0), (-75, 58), (-80, 58), (58, -80), (-66, 0), (-110, 40)])
def test_route_grouped_scales_at_the_ends_of_float32(rule, xs, ws):
    """Tokens or router rows whose squares are below float32, with the others so
    large that the products are not: equal experts are ordered by their exact logits all
    the same."""
    g = _gen(41)
    T, d, E = 96, 512, 64
    x, w = _randn(g, T, d, dtype=torch.bfloat16), _randn(g, E, d, dtype=torch.bfloat16)
    # in each 64 values x reads the same from behind and w is its own negative from
    # behind, so that these products add to 0 (and to float32 roundings); the small
    # rest, eight in the middle, is the logit, the same for both experts of a pair
    flip = torch.arange(d, device=DEV).view(-1, 64).flip(1).reshape(-1)
    at = torch.arange(d, device=DEV) % 64
    x, w = torch.where(at < 32, x, x[:, flip]), torch.where(at < 32, w, -w[:, flip])
    rest = (at >= 28) & (at < 36)
    w[:, rest] = _randn(g, E, d // 8, dtype=torch.bfloat16, std=2.0 ** -9)
    w[E // 2:, rest] = w[:E // 2, rest]
    x, w = x * 2.0 ** xs, w * 2.0 ** ws
    k = torch.full((T,), 8, dtype=torch.int32, device=DEV)
    _check_route(x, w, k, 8, router="screened", **RULES[rule])


def _wide_tokens(g, T, d, E):
    """Ordinary tokens, tokens of a norm in the thousands whose logits stay small (the
    large part meets pairs w, -w), and tokens of a norm that saturates the scores."""
    x, w = _randn(g, T, d, dtype=torch.bfloat16), _randn(g, E, d, dtype=torch.bfloat16, std=(d // 2) ** -0.5)
    w[:, 1:d // 2:2] = -w[:, 0:d // 2:2]
    x[:, 1:d // 2:2] = x[:, 0:d // 2:2]
    x[1::4, :d // 2] *= 2.0 ** 10
    x[2::8] *= 2.0 ** 9
    w[E // 3] = w[0]
    w[E // 2] = w[2]
    w[E // 2, d - 1] *= 1 + 2.0 ** -7
    return x, w


@pytest.mark.parametrize("rule", range(len(RULES)))
@pytest.mark.parametrize("T,d,E", [(70, 2048, 256), (37, 1024, 40), (21, 2048, 320), (19, 1024, 1024), (65, 4096, 128)])
def test_route_grouped_every_logit_exact(rule, T, d, E):
    """Tokens whose logits are too uncertain to screen (|x| |w| 8e-6 > 1/16) between
    ordinary ones."""
    g = _gen(T + E)
    x, w = _wide_tokens(g, T, d, E)
    radius = 66 * 2.0 ** -23 * torch.linalg.vector_norm(x.double(), dim=1) * torch.linalg.vector_norm(w.double(), dim=1).max()
    assert (radius > 0.1).sum() >= T // 4 and (radius < 0.03).sum() >= T // 2
    k = torch.randint(0, 6, (T,), generator=g, device=DEV, dtype=torch.int32)
    sb = None if RULES[rule]["score"] == "softmax" else (torch.rand(E, generator=g, device=DEV) - 0.5) * 0.1
    _check_route(x, w, k, 5, sb=sb, scale=2.5, router="screened", **RULES[rule])


@pytest.mark.parametrize("rule", range(len(RULES)))
@pytest.mark.parametrize("router,T,d,E", [("screened", 70, 2048, 256), ("screened", 33, 1024, 1024), ("float64", 40, 512, 64),
                                          ("auto", 3100, 1024, 256)])
def test_route_grouped_router_biases_that_are_not_finite(rule, router, T, d, E):
    """-inf: score 0, of all experts too; +inf: score 1 (a softmax has none then); NaN: out
    of service; ordinary and wide tokens."""
    g = _gen(T + E)
    x, w = _wide_tokens(g, T, d, E)
    k = torch.randint(0, 6, (T,), generator=g, device=DEV, dtype=torch.int32)
    sb = None if RULES[rule]["score"] == "softmax" else (torch.rand(E, generator=g, device=DEV) - 0.5) * 0.1
    for bias in ({E // 4: -math.inf, E - 1: -math.inf}, {E // 4: math.inf}, {1: math.nan, 3: -math.inf},
                 dict.fromkeys(range(E), -math.inf), dict.fromkeys(range(3, E), -math.inf)):
        rb = torch.zeros(E, device=DEV)
        rb[list(bias)] = torch.tensor(list(bias.values()), device=DEV)
        with np.errstate(invalid="ignore"):
            _check_route(x, w, k, 5, sb=sb, rb=rb, router=router, **RULES[rule])


@pytest.mark.parametrize("rule", range(len(RULES)))
@pytest.mark.parametrize("E", [64, 256, 320, 1024])
def test_route_grouped_screened_values_that_are_no_numbers(rule, E):
    """bf16 tokens and router rows with NaN or infinities: the screened router's ids are
    the float64 one's, and ordinary tokens keep theirs."""
    g = _gen(E)
    T, d = 40, 512
    x, w = _randn(g, T, d, dtype=torch.bfloat16), _randn(g, E, d, dtype=torch.bfloat16, std=d ** -0.5)
    k = torch.full((T,), 5, dtype=torch.int32, device=DEV)
    x[3, 9], x[8, 500], x[13, 0], x[13, 1] = math.nan, math.inf, math.inf, -math.inf
    x[20] = math.inf
    x[30, 4] = 3.3e38
    for bad_row in (False, True):
        if bad_row:
            w[5, 7], w[E - 2, 8] = math.nan, math.inf
        a, b = (_route(x, w, k, 5, moe.make_route_rule(**RULES[rule]), scale=2.5, router=r) for r in ("float64", "screened"))
        np.testing.assert_array_equal(a[0], b[0])
        np.testing.assert_array_equal(a[1], b[1])
        # radius of the ordinary tokens: 8e-6 * 23 * 1.3, twice, and both sides' roundings
        np.testing.assert_allclose(a[2], b[2], rtol=6e-4, atol=1e-38)
        assert (b[1][15:20] == -1).all()  # a NaN in the token leaves no score a number


@pytest.mark.parametrize("dtype,T,d,E,router,bias,rule", [
    ("f32", 4099, 256, 250, "auto", True, 4), ("f32", 2113, 384, 264, "auto", False, 2),
    ("bf16", 2100, 256, 272, "float64", True, 0), ("bf16", 4099, 1024, 256, "auto", True, 3),
    ("bf16", 1090, 768, 1000, "float64", False, 1), ("f32", 16385, 128, 8, "float64", True, 1)])
def test_route_grouped_large_batches_in_float64(dtype, T, d, E, router, bias, rule):
    """The 32 x 64 tiles of the float64 logits (from 256 tiles on), at sizes off the tile."""
    g = _gen(T + E)
    rule = (RULES + [dict(score="sigmoid", n_group=5, topk_group=2, group_score="top2", renorm=True)])[rule]
    assert -(-T // 64) * -(-E // 32) >= 256
    x, w = _randn(g, T, d, dtype=DT[dtype]), _randn(g, E, d, dtype=DT[dtype], std=d ** -0.5)
    w[E // 3], w[E - 1] = w[0], w[2]
    k = torch.randint(0, 7, (T,), generator=g, device=DEV, dtype=torch.int32)
    sb = (torch.rand(E, generator=g, device=DEV) - 0.5) * 0.1 if bias else None
    if bias:
        sb[1] = -math.inf
    _check_route(x, w, k, 6, sb=sb, scale=2.5, router=router, **rule)


# ---------------------------------------- more rows than one grid dimension holds

MANY = 2 ** 26 + 3  # workgroups of 64 threads: 2^32 threads and some


def test_norm_of_many_rows():
    y = torch.empty(MANY, 8, dtype=torch.bfloat16, device=DEV)
    y.normal_(generator=_gen(51))
    w = _randn(_gen(52), 8, dtype=torch.bfloat16)
    x = torch.full_like(y, 7.0)
    moe.moe_norm(moe.make_norm_desc(MANY, 8), None, y, None, None, None, w, None, None, x)
    for lo in range(0, MANY, 1 << 24):
        v = y[lo:lo + (1 << 24)].double()
        ref = v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * w.double()
        # 24 roundings on any path of eight values, the rounding to bf16
        bound = ref.abs() * (24 * EPS + U["bf16"] * 1.01) + 1e-40
        assert ((x[lo:lo + (1 << 24)].double() - ref).abs() <= bound).all()


def test_combine_norm_of_many_rows():
    T, d = MANY, 128
    yp = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    yp.normal_(generator=_gen(53))
    off = torch.arange(T + 1, dtype=torch.int32, device=DEV)
    inv = torch.arange(T, dtype=torch.int32, device=DEV).flip(0).contiguous()
    wts = torch.rand(T, generator=_gen(54), device=DEV)
    r = torch.full_like(yp, 7.0)
    moe.moe_combine_norm(moe.make_desc(T, d, 1, 128, 1), moe.make_norm_desc(T, d), yp, None, off, wts, inv, None, None,
                         None, None, None, None, r, None)
    for lo in range(0, T, 1 << 22):
        n = min(1 << 22, T - lo)
        ref = wts[lo:lo + n, None].double() * yp[T - lo - n:T - lo].flip(0).double()
        assert ((r[lo:lo + n].double() - ref).abs() <= ref.abs() * (2 * EPS + U["bf16"] * 1.01) + 1e-40).all()


@pytest.mark.parametrize("gate", ["channel", "token", "full"])
@pytest.mark.parametrize("d", [16, 9])
def test_norm_operands_of_many_rows(gate, d):
    """Every operand of the rows behind the first launch's 2^21: the bits of a call on
    those rows alone."""
    T, n = (1 << 21) + 5, 9
    t = _norm_case(57 + d, "bf16", T, d, "layer", True, gate, True)
    out = [torch.full_like(t["y"], 7.0) for _ in range(2)]
    call = lambda T, t, o: moe.moe_norm(
        moe.make_norm_desc(T, d, kind="layer", post=True, gate=gate, alpha=0.5), t["y"], t["resid"], t["post_w"],
        t["post_b"], t["gate"], t["pre_w"], t["pre_b"], *o)
    call(T, t, out)
    rows = {k: v[-n:].clone() if v is not None and (k in ("y", "resid") or (k == "gate" and gate != "channel")) else v
            for k, v in t.items()}
    last = [torch.empty_like(rows["y"]) for _ in range(2)]
    call(n, rows, last)
    for a, b in zip(out, last):
        assert torch.equal(a[-n:], b)


@pytest.mark.parametrize("gate", ["none", "token", "full"])
def test_combine_norm_operands_of_many_rows(gate):
    T, d, n = (1 << 21) + 5, 128, 9
    t = _norm_case(58, "bf16", T, d, "rms", True, gate, False)
    g = _gen(59)
    off = torch.arange(T + 1, dtype=torch.int32, device=DEV)
    inv = torch.randperm(T, generator=g, device=DEV).int()
    wts, yp, ysh = torch.rand(T, generator=g, device=DEV), t.pop("y"), _randn(g, T, d, dtype=torch.bfloat16)
    call = lambda T, yp, ysh, off, wts, inv, resid, gt, o: moe.moe_combine_norm(
        moe.make_desc(T, d, 1, 128, 1), moe.make_norm_desc(T, d, post=True, gate=gate), yp, ysh, off, wts, inv, resid,
        t["post_w"], None, gt, t["pre_w"], None, *o)
    out = [torch.full_like(ysh, 7.0) for _ in range(2)]
    call(T, yp, ysh, off, wts, inv, t["resid"], t["gate"], out)
    last = [torch.empty(n, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    own = yp[inv[-n:].long()].contiguous()
    c = lambda v: None if v is None else v[-n:].clone()
    call(n, own, c(ysh), off[:n + 1].clone(), c(wts), torch.arange(n, dtype=torch.int32, device=DEV), c(t["resid"]),
         c(t["gate"]), last)
    for a, b in zip(out, last):
        assert torch.equal(a[-n:], b)


@pytest.mark.parametrize("router", ["float64", "screened"])
def test_route_grouped_of_many_tokens(router):
    T, d, E = MANY, 128, 8
    x = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    x.normal_(generator=_gen(55))
    w = _randn(_gen(56), E, d, dtype=torch.bfloat16, std=d ** -0.5)
    k = torch.ones(T, dtype=torch.int32, device=DEV)
    desc = moe.make_desc(T, d, E, 128, 1, router=router)
    off = torch.empty(T + 1, dtype=torch.int32, device=DEV)
    ids = torch.full((T,), -7, dtype=torch.int32, device=DEV)
    wts = torch.full((T,), -7.0, device=DEV)
    st = torch.empty(1, dtype=torch.int32, device=DEV)
    rule = moe.make_route_rule(renorm=False)
    moe.moe_route_grouped(desc, rule, x, w, None, None, k, off, ids, wts, st,
                          moe.alloc_workspace(desc, moe.MOE_OP_ROUTE_GROUPED, DEV))
    assert torch.equal(off, torch.arange(T + 1, dtype=torch.int32, device=DEV)) and int(st) == 0
    assert int(ids.min()) >= 0 and int(ids.max()) < E
    for lo in (0, 2 ** 25 - 50, 2 ** 26 - 50, T - 100):
        part = x[lo:lo + 100].contiguous()
        _, want, ww, _ = _route(part, w, k[:100], 1, rule, router="float64")
        np.testing.assert_array_equal(ids[lo:lo + 100].cpu().numpy(), want)
        # |x| |w| is below 14 * 1.5: radius 1.7e-4, twice
        np.testing.assert_allclose(to_f64(wts[lo:lo + 100]), ww, rtol=4e-4)


# ----------------------------------------------------------------- BlockLayer

def _block_case(g, T, d, E, I, Is, k_max, L, R):
    bf = torch.bfloat16
    stack = lambda G, K: (_randn(g, L, G, R, K, dtype=bf, std=K ** -0.5), _randn(g, L, G, d, R, dtype=bf, std=0.2), None,
                          None, torch.randint(-1, L, (T,), generator=g, device=DEV, dtype=torch.int32))
    return dict(y=_randn(g, T, d, dtype=bf), resid=_randn(g, T, d, dtype=bf), pre_w=_randn(g, d, dtype=bf),
                w_router=_randn(g, E, d, dtype=bf, std=d ** -0.5), select_bias=None,
                k=torch.randint(0, k_max + 1, (T,), generator=g, device=DEV, dtype=torch.int32),
                w_gate=_randn(g, E, I, d, dtype=bf, std=d ** -0.5), w_up=_randn(g, E, I, d, dtype=bf, std=d ** -0.5),
                w_down=_randn(g, E, d, I, dtype=bf, std=I ** -0.5),
                shared=[_randn(g, Is, d, dtype=bf, std=d ** -0.5), _randn(g, Is, d, dtype=bf, std=d ** -0.5),
                        _randn(g, d, Is, dtype=bf, std=Is ** -0.5)],
                adapters=stack(E, I), shared_adapters=stack(1, Is))


def test_block_layer_made_and_run_on_other_streams():
    """A layer made on a busy stream and run on another, given or current, has what it
    needs; the results are those of a layer made and run on the default stream."""
    g = _gen(61)
    T, d, E, I, Is, k_max, L, R = 700, 256, 16, 128, 256, 4, 3, 8
    args = _block_case(g, T, d, E, I, Is, k_max, L, R)
    make = lambda: moe.BlockLayer(moe.make_desc(T, d, E, I, k_max, I_shared=Is), moe.make_route_rule(),
                                  moe.make_norm_desc(T, d), moe.make_norm_desc(T, d, post=True), adapters=L,
                                  shared_adapters=L, rank=R, device=DEV)
    out = lambda: [torch.zeros(T, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    want = make().run(**args, resid_out=(o := out())[0], x_out=o[1])
    torch.cuda.synchronize()
    busy, side = torch.cuda.Stream(), torch.cuda.Stream()
    for given in (True, False):
        got = out()
        torch.cuda.synchronize()
        with torch.cuda.stream(busy):
            torch.cuda._sleep(20_000_000)
            layer = make()
        if given:
            layer.run(**args, resid_out=got[0], x_out=got[1], stream=side)
        else:
            with torch.cuda.stream(side):
                layer.run(**args, resid_out=got[0], x_out=got[1])
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_block_layer_with_layer_norms_and_biases():
    """Weights and biases of all four norms reach their step: the layer's buffers and
    outputs have the bits of the single calls on the same inputs."""
    g = _gen(62)
    T, d, E, I, k_max = 50, 256, 8, 128, 3
    args = {**_block_case(g, T, d, E, I, 128, k_max, 1, 8), "shared": None, "adapters": None, "shared_adapters": None}
    desc = moe.make_desc(T, d, E, I, k_max)
    before = moe.make_norm_desc(T, d, kind="layer", post=True, gate="token")
    behind = moe.make_norm_desc(T, d, kind="layer", post=True, gate="channel", alpha=0.5)
    layer = moe.BlockLayer(desc, moe.make_route_rule(), before, behind, device=DEV)
    vec = {n: _randn(g, d, dtype=torch.bfloat16) for n in (
        "pre_w", "pre_b", "before_post_w", "before_post_b", "behind_post_w", "behind_post_b", "next_w", "next_b")}
    g1, g2 = _randn(g, T, dtype=torch.bfloat16), _randn(g, d, dtype=torch.bfloat16)
    r, x, r1, x1 = (torch.zeros(T, d, dtype=torch.bfloat16, device=DEV) for _ in range(4))
    layer.run(**{**args, **vec}, before_gate=g1, behind_gate=g2, resid_out=r, x_out=x)
    moe.moe_norm(before, args["y"], args["resid"], vec["before_post_w"], vec["before_post_b"], g1, vec["pre_w"],
                 vec["pre_b"], r1, x1)
    assert torch.equal(layer.resid, r1) and torch.equal(layer.x, x1)
    moe.moe_combine_norm(desc, behind, layer.y, None, layer.tok_off, layer.w, layer.inv, layer.resid, vec["behind_post_w"],
                         vec["behind_post_b"], g2, vec["next_w"], vec["next_b"], r1, x1)
    assert torch.equal(r, r1) and torch.equal(x, x1)
