"""Edges of the few-token layer and the 4-bit weights on the GPU: logits that tie or are no
numbers, groups that do not fill a tile, the largest sizes.  Tolerances as in test_gpu_few.py."""
import math

import numpy as np
import pytest
import torch

import mixture_experts_layer_token_amd as moe
from oracle import moe_oracle, quant
from perf import more_operators
from tests.test_gpu_few import DEV, DT, EPS, U, Case, Weight, _gen, _k, _layer_ref, _randn, _to_elt, _within
from workloads import to_f64

pytestmark = pytest.mark.gpu


# -------------------------------------------------------------------- routing

def _counts_of_route(c, x, k, router=None, bias=None):
    """moe_route's choices: per expert, and of each token."""
    desc = c.desc()
    i32 = dict(dtype=torch.int32, device=DEV)
    off, status = torch.empty(c.T + 1, **i32), torch.empty(1, **i32)
    ids, w = torch.full((c.T * c.k_max,), -1, **i32), torch.empty(c.T * c.k_max, device=DEV)
    moe.moe_route(desc, x, c.router if router is None else router, bias, k, off, ids, w, status,
                  moe.alloc_workspace(desc, moe.MOE_OP_ROUTE, DEV))
    ids, off = ids.cpu().numpy(), off.cpu().numpy()
    return np.bincount(ids[ids >= 0], minlength=c.E), [ids[off[t]:off[t + 1]] for t in range(c.T)]


@pytest.mark.parametrize("E", [2, 8, 61, 64, 100, 128, 256, 600])
@pytest.mark.parametrize("T", [1, 8, 16])
@pytest.mark.parametrize("tie", ["zeros", "twins", "apart", "bias", "bias63"])
def test_forward_few_ties_go_to_the_lower_expert(E, T, tie):
    """Exactly tied logits: tokens of zeros, equal router rows side by side and 64 apart,
    equal and -inf biases; the best of them with and without the experts 63, 127, .."""
    k_max = min(E, 7)
    c = Case(E + T, "bf16", T, 128, E, 128, 0, k_max)
    if tie == "zeros":
        c.x[::2] = 0
    elif tie == "twins":
        c.router[1::2] = c.router[0::2][:E // 2].clone()
    elif tie == "apart":
        at = torch.arange(E, device=DEV) % min(64, (E + 1) // 2)
        c.router = c.router[at].contiguous()
    else:
        c.x.zero_()
        c.bias = torch.tensor([0.0, -math.inf, 2.0, 1.0] if tie == "bias" else [-math.inf, 1.0, 0.0, 2.0],
                              device=DEV)[torch.arange(E, device=DEV) % 4].contiguous()
        if E == 2:
            c.bias = torch.zeros(2, device=DEV)
    c.check(_k(c, k_max, 1, max(1, k_max // 2)))


@pytest.mark.parametrize("dtype,group", [("f32", 0), ("bf16", 64), ("f32", 32)])
@pytest.mark.parametrize("E", [8, 64, 130])
def test_forward_few_ties_of_other_types(dtype, group, E):
    c = Case(E, dtype, 9, 256, E, 128, 128, 5, group, bool(group))
    c.x[3:6] = 0
    c.router[1::2] = c.router[0::2][:E // 2].clone()
    c.check(_k(c, 5, 3))


@pytest.mark.parametrize("E", [8, 40, 64, 200, 600])
@pytest.mark.parametrize("T,group", [(1, 0), (5, 0), (16, 0), (5, 64)])
def test_forward_few_routes_tokens_that_are_no_numbers(E, T, group):
    """A token with a NaN has NaN for every logit: they tie.  It runs the experts that
    moe_route gives it, without an always-on expert too its outputs are NaN, and the other
    tokens' stay right."""
    k_max, d = min(E, 4), 256
    c = Case(E + T, "bf16", T, d, E, 128, 0, k_max, group, bool(group))
    k, bad = _k(c, k_max), T // 2
    x = c.x.clone()
    x[bad, 9] = math.nan
    out, stats, status = c.forward(k, x=x)
    counts, ids = _counts_of_route(c, x, k)
    st = stats.cpu().numpy()
    np.testing.assert_array_equal(st[:E], counts)
    assert st[E] == (counts > 0).sum() and st[E + 1] == T * k_max and int(status) == 0
    assert ids[bad].tolist() == list(range(k_max)) and out[bad].isnan().all()
    r = moe_oracle.route(to_f64(c.x), to_f64(c.router), None, [k_max] * T, k_max)
    routes = [(j // k_max, int(e), float(w)) for j, (e, w) in enumerate(zip(r["ids"], r["w"])) if j // k_max != bad]
    keep = [t for t in range(T) if t != bad]
    if keep:
        ref, tol = _layer_ref(to_f64(c.x), routes, c.w, None, c.dt, group, T, d)
        _within(out[keep], ref[keep], tol[keep])


# ------------------------------------------------------------- 4-bit weights

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("K", [8, 72, 136, 1000, 1032])
def test_pack_cases_return_the_groups_of_k(monkeypatch, dtype, zeros, group, K):
    """A pack's scales and zero points as [G, N, ceil(K / group)], whatever fills up the
    stored tiles of 128 inputs: the measured calls' outputs are the plain form's."""
    case = dict(op="pack", dtype=dtype, G=2, N=21, K=K, group=group, zeros=zeros)
    want = more_operators.run(more_operators.prepare(case, 7))
    monkeypatch.setattr(more_operators, "own", True)
    got = more_operators.run(more_operators.prepare(case, 7))
    assert got[1].shape == (2, 21, -(-K // group)) and (got[2] is None) == (not zeros)
    for a, b in zip(got, want):
        assert a is None and b is None or a.dtype == b.dtype and torch.equal(a, b)


@pytest.mark.parametrize("dtype,group,zeros", [("bf16", 32, True), ("f32", 128, False)])
def test_q4_more_matrices_than_a_grid_has_rows(dtype, group, zeros):
    """65,600 matrices: packed, re-laid and widened by workgroups that take two of them."""
    G, N, K = 65600, 2, 40
    ng = -(-K // group)
    w = _randn(_gen(1), G, N, K, dtype=DT[dtype])
    q = moe.q4_pack(w, group=group, zeros=zeros)
    out = torch.full_like(w, math.nan)
    moe.moe_q4_unpack(q, out)
    at = [0, 1, 63, 65534, 65535, 65536, 65599]
    codes, s, z = quant.q4_quantise(to_f64(w[at]), group, zeros, _to_elt(dtype))
    np.testing.assert_array_equal(to_f64(q.scales[at])[:, :ng, :N], np.swapaxes(s, 1, 2))
    ref = quant.q4_values(codes, s, z, group)
    _within(out[at], ref, U[DT[dtype]] * np.abs(ref))
    # back from row-major codes: the same bytes
    step = q.scales[:, :ng, :N].transpose(1, 2)
    zp = q.zeros[:, :ng, :N].transpose(1, 2) if zeros else None
    wide = lambda t: t.double().repeat_interleave(group, -1)[..., :K]
    c = torch.where(wide(step) == 0, 0.0, out.double() / wide(step)).round() + (wide(zp) if zeros else 8)
    c = c.to(torch.uint8)
    rm = c[..., 0::2] | (c[..., 1::2] << 4)
    r = moe.q4_tile(rm, step.contiguous(), zp.contiguous() if zeros else None, group=group)
    assert torch.equal(r.scales, q.scales) and (not zeros or torch.equal(r.zeros, q.zeros))
    back = torch.full_like(w, math.nan)
    moe.moe_q4_unpack(r, back)
    assert torch.equal(back, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K,N", [(2, 65536, 40), (20, 14336, 300), (1, 16392, 4100), (5, 136, 262144),
                                      (700, 520, 70), (1000, 72, 8300), (65536, 8, 3)])
def test_q4_linear_at_its_limits(dtype, rows, K, N):
    g = _gen(rows + K)
    w = Weight(g, 1, N, K, DT[dtype], 64, True)
    x = _randn(g, rows, K, dtype=DT[dtype])
    y = torch.full((rows, N), math.nan, dtype=DT[dtype], device=DEV)
    moe.moe_q4_linear(w.arg, x, y)
    xa = to_f64(x)
    ref = xa @ w.val[0].T
    tol = w.order(K) * EPS * (np.abs(xa) @ w.mag[0].T)
    _within(y, ref, tol + U[DT[dtype]] * (np.abs(ref) + tol))


@pytest.mark.parametrize("dtype,group", [("bf16", 0), ("f32", 0), ("bf16", 64), ("f32", 32)])
@pytest.mark.parametrize("T,d,E,I,Is,k_max", [(3, 65536, 3, 128, 0, 2), (16, 16384, 4, 128, 256, 2),
                                              (2, 128, 2, 65536, 0, 2), (10, 256, 5, 14336, 128, 3)])
def test_forward_few_at_its_limits(dtype, group, T, d, E, I, Is, k_max):
    c = Case(T + d, dtype, T, d, E, I, Is, k_max, group, bool(group))
    c.check(_k(c, k_max, 1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E", [8, 40, 200, 600])
@pytest.mark.parametrize("where", ["row", "bias", "x"])
@pytest.mark.parametrize("value", [math.nan, -math.nan, math.inf, -math.inf])
def test_forward_few_routes_like_moe_route_whatever_the_logits(dtype, E, where, value):
    """NaN of either sign and infinities in one expert's router row or bias, or in one token."""
    c = Case(E, dtype, 5, 256, E, 128, 0, 4)
    k, x = _k(c, 4), c.x
    if where == "row":
        t, at = c.router, (3, 7)
    elif where == "bias":
        t, at = torch.zeros(E, device=DEV), (3,)
        c.bias = t
    else:
        t, at = c.x.clone(), (2, 3)
        x = t
    t[at] = math.nan if math.isnan(value) else value
    if math.copysign(1.0, value) < 0 and math.isnan(value):
        bits = t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)
        bits[at] = -(1 << 22) if t.dtype == torch.float32 else -(1 << 6)
        assert t[at].isnan() and bits[at] < 0
    stats = c.forward(k, x=x)[1].cpu().numpy()
    counts, _ = _counts_of_route(c, x, k, None, c.bias)
    np.testing.assert_array_equal(stats[:E], counts)
