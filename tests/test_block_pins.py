"""Pins of the float64 oracle of the operators around the layer (oracle/block.py),
and the refusals of their entry points.  No GPU needed."""
import ctypes
import math

import numpy as np
import pytest
import torch

import mixture_experts_layer_token_amd as moe
import oracle
from mixture_experts_layer_token_amd import _lib
from oracle import block


def _rng(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


def test_softmax_without_groups_is_the_plain_router():
    x, w = _rng(9, 32), _rng(12, 32, seed=1)
    k = np.array([0, 1, 2, 3, 12, 5, 4, 2, 1])
    a = oracle.route(x, w, None, k, 12, 1.5)
    b = block.route_grouped(x, w, None, None, k, score="softmax", scale=1.5)
    np.testing.assert_array_equal(a["ids"], b["ids"])
    np.testing.assert_array_equal(a["tok_off"], b["tok_off"])
    np.testing.assert_allclose(a["w"], b["w"], rtol=1e-6)


def test_groups_bias_and_ties_hand_worked():
    # logits 0, ln 3, -ln 3, 0 | 0, 0, ln 3, ln 3: sigmoids 1/2, 3/4, 1/4, 1/2 | 1/2, 1/2, 3/4, 3/4
    l3 = math.log(3.0)
    x, w = np.eye(1), np.array([[0, l3, -l3, 0, 0, 0, l3, l3]]).T
    one = dict(score="sigmoid", n_group=2, topk_group=1)
    r = block.route_grouped(x, w, None, None, [3], group_score="top2", **one)  # 5/4 < 3/2
    assert r["ids"].tolist() == [6, 7, 4]
    np.testing.assert_allclose(r["w"], [3 / 8, 3 / 8, 1 / 4], rtol=1e-7)
    r = block.route_grouped(x, w, None, None, [2], group_score="max", **one)  # 3/4 = 3/4: the lower group
    assert r["ids"].tolist() == [1, 0]
    # the bias decides and does not weigh
    b = np.array([0, 0, 0.6, 0, -np.inf, 0, 0, -np.inf])
    r = block.route_grouped(x, w, None, b, [4], group_score="top2", renorm=False, **one)
    assert r["ids"].tolist() == [2, 1, 0, 3]
    np.testing.assert_allclose(r["w"], [1 / 4, 3 / 4, 1 / 2, 1 / 2], rtol=1e-7)
    # two experts in service in the only kept group: the rest of the slots stay empty
    b = np.array([-np.inf] * 4 + [-np.inf, 0, 0, -np.inf])
    r = block.route_grouped(x, w, None, b, [3], group_score="top2", **one)
    assert r["ids"].tolist() == [6, 5, -1]
    np.testing.assert_allclose(r["w"], [3 / 5, 2 / 5, 0], rtol=1e-7)
    r = block.route_grouped(x, w, None, np.full(8, -np.inf), [2], group_score="max", **one)
    assert r["ids"].tolist() == [-1, -1] and not r["w"].any()


def test_norms_against_torch():
    v, w, b = _rng(5, 24), _rng(24, seed=1), _rng(24, seed=2)
    t = torch.from_numpy
    ref = torch.nn.functional.layer_norm(t(v), (24,), t(1 + w), t(b), 1e-5).numpy()
    np.testing.assert_allclose(block.norm(v, w, b, kind="layer", eps=1e-5, w_offset=1.0), ref, rtol=1e-12, atol=1e-12)
    rms = v / np.sqrt(np.mean(v * v, axis=1)[:, None] + 1e-5)
    np.testing.assert_allclose(block.norm(v, eps=1e-5), rms, rtol=1e-14)
    r, x = block.norm_chain(v, w[None], post=(None, None), gate=b, alpha=0.5, pre=(w, b), eps=1e-5)
    np.testing.assert_allclose(r, w + 0.5 * b * rms, rtol=1e-13)
    np.testing.assert_allclose(x, block.norm(r, w, b, eps=1e-5), rtol=1e-14)


def test_adapters_are_merged_weights():
    L, G, R, K, N, rows = 3, 2, 4, 8, 6, 7
    a, b = _rng(L, G, R, K), _rng(L, G, N, R, seed=1)
    w, x = _rng(G, N, K, seed=2), _rng(rows, K, seed=3)
    off, tok = np.array([0, 4, 6]), np.array([2, 0, 1, 3, 0, 2, 1])
    ids, scales = np.array([1, 2, -1, 0]), np.array([0.5, 2.0, 1.0])
    g = [0, 0, 0, 0, 1, 1]
    y = np.stack([w[g[r]] @ x[r] for r in range(6)] + [np.full(N, 9.0)])
    out = block.adapt(y, x, a, b, ids, scales=scales, row_tok=tok, expert_off=off)
    for r in range(6):
        i = ids[tok[r]]
        m = w[g[r]] + (scales[i] * b[i, g[r]] @ a[i, g[r]] if i >= 0 else 0)
        np.testing.assert_allclose(out[r], m @ x[r], rtol=1e-12)
    assert (out[6] == 9.0).all()


# ------------------------------------------------------------------ refusals

P = ctypes.c_void_p
FAKE = [P((i + 1) << 24) for i in range(20)]  # never dereferenced: every call below is refused first


def _desc(**kw):
    base = dict(T=4, d=128, E=8, I=128, k_max=2, I_shared=0, dtype=moe.MOE_BF16, path=0, router=0, routed_scale=1.0,
                k_policy=0, k_granule=1)
    base.update(kw)
    return _lib.moe_desc(**base)


def _rule(**kw):
    base = dict(score=0, n_group=4, topk_group=2, group_score=1, renorm=1)
    base.update(kw)
    return _lib.moe_route_rule(**base)


@pytest.mark.parametrize("rule,desc,code", [
    (dict(score=2), {}, 3), (dict(score=-1), {}, 3), (dict(group_score=2), {}, 3), (dict(renorm=2), {}, 3),
    (dict(n_group=0), {}, 2), (dict(n_group=3), {}, 2), (dict(topk_group=0), {}, 2), (dict(topk_group=5), {}, 2),
    (dict(n_group=128, topk_group=64), dict(E=128), 2), (dict(topk_group=1), dict(k_max=3), 2),
    ({}, dict(router=moe.MOE_ROUTER_FUSED), 3), ({}, dict(router=moe.MOE_ROUTER_SCREENED, dtype=0), 3),
    ({}, dict(E=0), 2), ({}, {}, 4)])
def test_route_grouped_refuses(rule, desc, code):
    lib = _lib.load()
    d, r = _desc(**desc), _rule(**rule)
    call = lambda *a, ws=None, n=0: lib.moe_route_grouped(ctypes.byref(d), ctypes.byref(r), *a, ws, n, None)
    assert call(*FAKE[:9]) == code
    if code == 4:
        assert call(*FAKE[:9], ws=P(1 << 20), n=16) == 4
        assert call(None, *FAKE[1:9], ws=P(1 << 20), n=1 << 30) == 1
        assert call(FAKE[0], None, *FAKE[2:9], ws=P(1 << 20), n=1 << 30) == 1
        assert call(P((1 << 24) + 2), *FAKE[1:9], ws=P(1 << 20), n=1 << 30) == 5
        assert call(*FAKE[:9], ws=P((1 << 20) + 16), n=1 << 30) == 5
        assert lib.moe_route_grouped(ctypes.byref(d), None, *FAKE[:9], None, 0, None) == 1


def _nd(**kw):
    base = dict(T=4, d=128, dtype=1, kind=0, post=1, gate_mode=0, eps=1e-6, alpha=1.0, w_offset=0.0)
    base.update(kw)
    return _lib.moe_norm_desc(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 3), (dict(kind=2), 3), (dict(gate_mode=4), 3), (dict(gate_mode=-1), 3), (dict(post=2), 3),
    (dict(T=-1), 2), (dict(d=0), 2), (dict(d=65537), 2), (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2),
    (dict(eps=float("inf")), 2), (dict(alpha=float("inf")), 2), (dict(w_offset=float("nan")), 2),
    (dict(gate_mode=1), 1)])
def test_norm_refuses(kw, code):
    lib, y = _lib.load(), FAKE
    nd = _nd(**kw)
    assert lib.moe_norm(ctypes.byref(nd), y[0], y[1], y[2], None, None, y[3], None, y[4], y[5], None) == code
    d = _desc(dtype=nd.dtype if nd.dtype in (0, 1) else 1)
    assert lib.moe_combine_norm(ctypes.byref(d), ctypes.byref(nd), *y[:6], y[6], None, None, y[7], None, y[8], y[9],
                                None) == code


def test_norm_refuses_buffers():
    lib, y = _lib.load(), FAKE
    call = lambda nd, *a: lib.moe_norm(ctypes.byref(nd), *a, None)
    off = lambda p, n: P(p.value + n)
    assert lib.moe_norm(None, *y[:9], None) == 1
    assert call(_nd(), y[0], y[1], None, None, None, None, None, None, None) == 1       # no output
    assert call(_nd(), None, None, None, None, None, None, None, None, y[2]) == 1       # no input
    assert call(_nd(), None, y[1], None, None, None, None, None, None, y[2]) == 2       # post norm without y
    assert call(_nd(post=0), None, y[1], None, None, None, None, None, y[3], y[2]) == 2  # resid_out without y
    assert call(_nd(), y[0], y[1], None, None, y[2], None, None, y[3], None) == 1       # a gate that no mode asks for
    assert call(_nd(), off(y[0], 2), y[1], None, None, None, None, None, y[3], None) == 5
    assert call(_nd(), y[0], y[1], off(y[2], 8), None, None, None, None, y[3], None) == 5
    assert call(_nd(), y[0], y[1], None, None, None, None, None, y[3], y[3]) == 2       # both outputs in one
    assert call(_nd(), y[0], y[1], None, None, None, None, None, off(y[0], 256), None) == 2
    assert call(_nd(), y[0], y[1], None, None, None, None, None, None, off(y[1], 1008)) == 2
    assert call(_nd(), y[0], y[1], None, None, None, y[3], None, None, y[3]) == 2       # weight overwritten
    assert call(_nd(T=0), None, None, None, None, None, None, None, None, None) == 0
    nd = _nd()
    comb = lambda d, *a: lib.moe_combine_norm(ctypes.byref(d), ctypes.byref(nd), *a, None)
    rest = [None, None, None, None, None, y[8], None]
    assert comb(_desc(T=3), *y[:6], *rest) == 2
    assert comb(_desc(d=256), *y[:6], *rest) == 2
    assert comb(_desc(dtype=0), *y[:6], *rest) == 2
    assert comb(_desc(), None, *y[1:6], *rest) == 1
    assert comb(_desc(), y[0], y[1], None, *y[3:6], *rest) == 1
    assert comb(_desc(), y[8], *y[1:6], *rest) == 2                                     # output over y_perm
    assert comb(_desc(), y[0], y[8], *y[2:6], *rest) == 2


def _ad(**kw):
    base = dict(T=16, rows=16, K=64, N=64, R=8, L=4, G=1, dtype=1)
    base.update(kw)
    return _lib.moe_adapter_desc(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), 3), (dict(T=-1), 2), (dict(rows=-1), 2), (dict(T=1 << 23, rows=(1 << 22) + 1), 2), (dict(K=4), 2), (dict(K=65544), 2), (dict(K=65), 2),
    (dict(N=12), 2), (dict(R=4), 2), (dict(R=12), 2), (dict(R=136), 2), (dict(L=0), 2), (dict(G=0), 2),
    (dict(G=1025), 2), (dict(T=15), 2), (dict(G=2), 1), ({}, 4)])
def test_adapt_refuses(kw, code):
    lib, y = _lib.load(), FAKE
    d = _ad(**kw)
    n = ctypes.c_size_t(0)
    assert lib.moe_adapt_workspace_size(ctypes.byref(d), ctypes.byref(n)) in ((code,) if code in (2, 3) and kw != dict(T=15) else (0,))
    call = lambda x=y[0], xr=None, a=y[1], b=y[2], ids=y[3], tok=None, off=None, yi=y[4], yo=y[5], ws=None, n=0: \
        lib.moe_adapt(ctypes.byref(d), x, xr, a, b, None, None, ids, tok, off, yi, yo, ws, n, None)
    assert call() == code
    if code != 4:
        return
    for name in ("x", "a", "b", "ids", "yi", "yo"):
        assert call(**{name: None}) == 1, name
    shift = lambda p, k: P(p.value + k)
    for name in ("x", "a", "b", "yi", "yo"):
        assert call(**{name: shift(y[9], 8)}) == 5, name
    assert call(yo=shift(y[4], 64)) == 2
    assert call(yo=y[0]) == 2 and call(yo=y[1]) == 2 and call(yo=y[2]) == 2
    assert call(ws=P(1 << 20), n=8) == 4
    assert call(ws=P((1 << 20) + 64), n=1 << 20) == 5
    assert lib.moe_adapt(None, *[None] * 12, 0, None) == 1
    empty = _ad(rows=0)
    assert lib.moe_adapt(ctypes.byref(empty), *[None] * 12, 0, None) == 0


def test_bindings_refuse_tensors():
    nd = moe.make_norm_desc(2, 64)
    cpu = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_norm(nd, cpu, cpu, None, None, None, None, None, cpu, None)
    with pytest.raises(TypeError, match="torch tensor"):
        moe.moe_norm(nd, [1.0], cpu, None, None, None, None, None, cpu, None)
    desc = moe.make_desc(2, 128, 8, 128, 2)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_route_grouped(desc, moe.make_route_rule(), cpu, cpu, None, None, cpu, cpu, cpu, cpu, None, None)
    with pytest.raises(KeyError):
        moe.make_route_rule(score="tanh")
    with pytest.raises(ValueError, match="no shared expert"):
        moe.BlockLayer(desc, moe.make_route_rule(), nd, nd, shared_adapters=2, device="cpu")


def test_workspace_of_grouped_routing():
    d = _desc(T=64, d=256, E=8)
    n = ctypes.c_size_t(0)
    lib = _lib.load()
    assert lib.moe_workspace_size(ctypes.byref(d), moe.MOE_OP_ROUTE_GROUPED, ctypes.byref(n)) == 0
    need = n.value
    assert need > 0 and need % 256 == 0
    assert lib.moe_workspace_size(ctypes.byref(d), moe.MOE_OP_FORWARD, ctypes.byref(n)) == 0 and n.value >= need
    assert lib.moe_workspace_size(ctypes.byref(d), 8, ctypes.byref(n)) == 3
