"""The few-token layer and the 4-bit weights on the GPU against the float64 oracle
(oracle/moe_oracle.py, oracle/quant.py), and a run of them with the layer's steps.

Tolerances come from the arithmetic: `U[t]` is the half step of one rounding to the
element type, EPS = 2^-23 a float32 rounding of either kind (a matrix instruction may
truncate), and each bound counts the roundings on its path.
"""
import math

import numpy as np
import pytest
import torch

import mixture_experts_layer_token_amd as moe
import oracle
from oracle import moe_oracle, quant
from workloads import to_f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
EPS = 2.0 ** -23


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(gen, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)


def _within(got, ref, bound, what=""):
    err = np.abs(to_f64(got) - ref)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}{int(bad.sum())} of {bad.size}, worst "
                           f"{np.nanmax(err / np.maximum(bound, 1e-300)):.3g} bounds, first {np.argwhere(bad)[0]}")


class Weight:
    """A stack of matrices as the kernels take it, with its float64 values and, for the
    bounds, `mag` >= |weight| of every product that the kernel sums: |W| itself, or for
    codes s (|16 + q| + |16 + z|), what is summed and subtracted again."""

    def __init__(self, gen, G, N, K, dtype, group=0, zeros=False, std=None, layout="rowmajor"):
        std = K ** -0.5 if std is None else std
        self.group = group
        if not group:
            w = _randn(gen, G, N, K, dtype=dtype, std=std)
            self.arg = moe.pack_weights(w) if layout == "blocked" else w
            self.val = to_f64(w)
            self.mag = np.abs(self.val)
            return
        ng = -(-K // group)
        rm = torch.randint(0, 256, (G, N, K // 2), generator=gen, device=DEV, dtype=torch.uint8)
        s = ((torch.rand(G, N, ng, generator=gen, device=DEV) + 0.5) * (std / 4.8)).to(dtype)
        z = torch.randint(0, 16, (G, N, ng), generator=gen, device=DEV, dtype=torch.uint8) if zeros else None
        self.arg = moe.q4_tile(rm, s, z, group=group)
        self.rm = (rm, s, z)
        self.codes = quant.q4_unpair(to_f64(rm))
        zz = None if z is None else to_f64(z)
        self.val = quant.q4_values(self.codes, to_f64(s), zz, group)
        self.mag = quant.q4_values(self.codes + 32 + (16 if z is None else 2 * np.repeat(zz, group, -1)[..., :K]),
                                   to_f64(s), zz, group)  # s (q + z + 32) in either case

    def order(self, K):
        """Roundings of a sum over K: its additions, and for codes each group's three more."""
        return K + 16 + (3 * (-(-K // self.group)) if self.group else 0)


def _silu(v):
    return v / (1.0 + np.exp(-v))


def _ffn(x, e, ws, w, dtype, q4):
    """Rows x [n, d] through expert e with weights w [n]: value and error bound before
    the outputs' own rounding.  H is rounded to bf16, in float32 kept as it is."""
    wg, wu, wd = ws
    d, I = wg.val.shape[2], wg.val.shape[1]
    ax = np.abs(x)
    g, u = x @ wg.val[e].T, x @ wu.val[e].T
    dg = wg.order(d) * EPS * (ax @ wg.mag[e].T)
    du = wu.order(d) * EPS * (ax @ wu.mag[e].T)
    s = _silu(g)
    h = w[:, None] * s * u
    # |SiLU'| <= 1.1; six roundings of SiLU, the product and the weight (1 ulp exp: 2 more)
    dh = np.abs(w)[:, None] * (1.1 * dg * (np.abs(u) + du) + (np.abs(s) + 1.1 * dg) * du) + (8 * EPS + U[dtype]) * np.abs(h)
    dh += 2.0 ** -126
    y = h @ wd.val[e].T
    dy = dh @ np.abs(wd.val[e]).T + wd.order(I) * EPS * ((np.abs(h) + dh) @ wd.mag[e].T)
    return y, dy


def _layer_ref(x, routes, ws, sh, dtype, q4, T, d):
    """routes: (token, expert, weight); returns out and its bound."""
    out, tol = np.zeros((T, d)), np.zeros((T, d))
    for e in sorted({r[1] for r in routes}):
        rows = [(t, w) for t, f, w in routes if f == e]
        at = [t for t, _ in rows]
        y, dy = _ffn(x[at], e, ws, np.array([w for _, w in rows]), dtype, q4)
        for i, t in enumerate(at):
            out[t] += y[i]
            tol[t] += dy[i]
    if sh is not None:
        y, dy = _ffn(x, 0, sh, np.ones(T), dtype, q4)
        out, tol = out + y, tol + dy
    # the routing weights' own error (float32 softmax, 8 roundings) and the final rounding
    n = 1 + len({r[1] for r in routes})
    return out, tol * 1.01 + (n + 8) * EPS * np.abs(out) + U[dtype] * (np.abs(out) + tol) + 2.0 ** -126


class Case:
    def __init__(self, seed, dtype, T, d, E, I, Is, k_max, group=0, zeros=False, layout="rowmajor", std=None):
        g = self.gen = _gen(seed)
        self.dt, self.T, self.d, self.E, self.I, self.Is, self.k_max, self.group = DT[dtype], T, d, E, I, Is, k_max, group
        self.x = _randn(g, T, d, dtype=self.dt)
        mk = lambda G, N, K: Weight(g, G, N, K, self.dt, group, zeros, std, layout)
        self.w = [mk(E, I, d), mk(E, I, d), mk(E, d, I)]
        self.sh = [mk(1, Is, d), mk(1, Is, d), mk(1, d, Is)] if Is else None
        self.args = [w.arg for w in self.w] + ([w.arg for w in self.sh] if Is else [None] * 3)
        self.router = _randn(g, E, d, dtype=self.dt, std=d ** -0.5)
        self.bias = None
        self.layout = layout

    def desc(self, **kw):
        return moe.make_desc(self.T, self.d, self.E, self.I, self.k_max, I_shared=self.Is, dtype=self.dt,
                             weight_layout=self.layout, **kw)

    def outputs(self):
        return (torch.full((self.T, self.d), math.nan, dtype=self.dt, device=DEV),
                torch.full((self.E + 2,), -7, dtype=torch.int32, device=DEV),
                torch.full((1,), -7, dtype=torch.int32, device=DEV))

    def forward(self, k, ws=None, stream=None, x=None, **kw):
        desc = self.desc(**kw)
        if ws is None:
            ws = moe.alloc_workspace(desc, moe.MOE_OP_FEW, DEV)
            ws.fill_(0xA5)
        out, stats, status = self.outputs()
        moe.moe_forward_few(desc, self.x if x is None else x, self.router, self.bias, k, *self.args, out, stats, status,
                            ws, stream)
        return out, stats, status

    def check(self, k, scale=1.0, policy="exact", granule=1):
        out, stats, status = self.forward(k, routed_scale=scale, k_policy=policy, k_granule=granule)
        torch.cuda.synchronize()
        ke, bad = oracle.execution_budgets(to_f64(k), self.k_max, policy, granule)
        r = oracle.route(to_f64(self.x), to_f64(self.router), to_f64(self.bias), ke, self.k_max, scale)
        p = oracle.permute(r["tok_off"], r["ids"], self.E)
        st = stats.cpu().numpy()
        np.testing.assert_array_equal(st[:self.E], p["counts"])
        assert st[self.E] == p["n_active"] and st[self.E + 1] == len(r["ids"]) and int(status) == bad
        tok = np.repeat(np.arange(self.T), np.diff(r["tok_off"]).astype(int))
        routes = list(zip(tok.tolist(), np.asarray(r["ids"]).tolist(), np.asarray(r["w"]).tolist()))
        ref, tol = _layer_ref(to_f64(self.x), routes, self.w, self.sh, self.dt, self.group, self.T, self.d)
        _within(out, ref, tol)
        rel = np.linalg.norm(to_f64(out) - ref) / max(np.linalg.norm(ref), 1e-300)
        assert rel <= (1e-2 if self.dt == torch.bfloat16 else 1e-5), rel
        return out


def _k(case, *choices):
    pick = torch.tensor(choices, dtype=torch.int32, device=DEV)
    return pick[torch.arange(case.T, device=DEV) % len(pick)].contiguous()


# ------------------------------------------------------------- 4-bit weights

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("G,N,K", [(1, 16, 128), (2, 5, 40), (1, 33, 264), (3, 18, 1000)])
def test_q4_tile_and_unpack(dtype, zeros, group, G, N, K):
    w = Weight(_gen(N + K), G, N, K, DT[dtype], group, zeros)
    q = w.arg
    nt, kt, ng = -(-N // 16), -(-K // 128), -(-K // group)
    got = q.codes.cpu().numpy().reshape(G, -1)
    for g in range(G):
        np.testing.assert_array_equal(got[g], quant.q4_tile(w.codes[g], N, K))
    s = to_f64(q.scales)
    np.testing.assert_array_equal(s[:, :ng, :N], np.swapaxes(to_f64(w.rm[1]), 1, 2))
    assert (s[:, ng:] == 0).all() and (s[:, :, N:] == 0).all() and s.shape == (G, kt * 128 // group, nt * 16)
    out = torch.full((G, N, K), math.nan, dtype=DT[dtype], device=DEV)
    moe.moe_q4_unpack(q, out)
    ref = torch.from_numpy(w.val).float().to(DT[dtype])  # 13- or 29-bit products: float32 rounds those of float32
    if dtype == "bf16":
        assert torch.equal(out.cpu(), ref)
    else:
        _within(out, w.val, U[torch.float32] * np.abs(w.val))


def _to_elt(dtype):
    return lambda v: torch.from_numpy(np.asarray(v)).to(DT[dtype]).double().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("G,N,K", [(1, 16, 128), (2, 37, 520), (1, 1, 8), (5, 50, 96)])
def test_q4_pack(dtype, zeros, group, G, N, K):
    g = _gen(K)
    w = _randn(g, G, N, K, dtype=DT[dtype])
    w[0, 0, :] = 0                                        # a group of zeros
    if N > 8:
        w[0, 1] = torch.arange(K, device=DEV).to(DT[dtype]) % 15 - 7.0   # codes at their borders: amax 7
        w[0, 2] = (torch.arange(K, device=DEV) % 29 - 14.0) / 2          # every quotient a tie
        w[0, 3] = w[0, 3].abs() + 3                       # one-sided
        w[0, 4] = -(w[0, 4].abs())
        w[0, 5] *= 2.0 ** -120
        w[0, 6] *= 2.0 ** 100
        w[0, 7] = 2.0 ** -133                             # the scale's last places
    q = moe.q4_pack(w, group=group, zeros=zeros)
    codes, s, z = quant.q4_quantise(to_f64(w), group, zeros, _to_elt(dtype))
    ng = -(-K // group)
    np.testing.assert_array_equal(to_f64(q.scales)[:, :ng, :N], np.swapaxes(s, 1, 2))
    if zeros:
        np.testing.assert_array_equal(q.zeros.cpu().numpy()[:, :ng, :N], np.swapaxes(z, 1, 2))
    out = torch.empty_like(w)
    moe.moe_q4_unpack(q, out)
    ref = quant.q4_values(codes, s, z, group)
    _within(out, ref, U[DT[dtype]] * np.abs(ref) + 2.0 ** -150 if dtype == "f32" else U[DT[dtype]] * np.abs(ref) + 2.0 ** -134)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("zeros", [False, True])
def test_q4_pack_every_magnitude(dtype, zeros):
    """Codes of many values, ties among them, at the scales where 1 / s ends and beyond."""
    w = torch.cat([_randn(_gen(5), 600, 512, dtype=DT[dtype]),
                   (_randn(_gen(6), 56, 512).double() * 2.0 ** -torch.arange(94, 150, device=DEV)[:, None].double()).to(DT[dtype])])
    w[600:, ::5] = w[600:, :1] / 2
    q = moe.q4_pack(w, group=64, zeros=zeros)
    codes, s, z = quant.q4_quantise(to_f64(w)[None], 64, zeros, _to_elt(dtype))
    np.testing.assert_array_equal(to_f64(q.scales)[:, :, :656], np.swapaxes(s, 1, 2))
    np.testing.assert_array_equal(q.codes.cpu().numpy(), quant.q4_tile(codes[0], 656, 512))


def test_q4_pack_values_that_are_no_numbers():
    for bad in (math.nan, math.inf, -math.inf):
        for zeros in (False, True):
            w = _randn(_gen(3), 20, 256)
            w[4, 130] = bad
            q = moe.q4_pack(w, group=64, zeros=zeros)
            out = torch.empty_like(w)
            moe.moe_q4_unpack(q, out)
            assert out[4, 128:192].isnan().all()
            out[4, 128:192] = 0
            assert out.isfinite().all()


def _linear(q, x):
    y = torch.full((x.shape[0], q.desc.N), math.nan, dtype=x.dtype, device=DEV)
    moe.moe_q4_linear(q, x, y)
    return y


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True), (128, False)])
@pytest.mark.parametrize("rows,K,N", [(1, 128, 16), (1, 2048, 512), (3, 1000, 37), (16, 264, 130), (17, 8, 1),
                                      (33, 4096, 100), (64, 712, 256), (100, 512, 48),
                                      (5, 136, 16500), (20, 1000, 16385), (40, 264, 20001), (70, 8, 16399),
                                      (2, 136, 24600), (20, 264, 8200), (20, 520, 4100), (64, 136, 4100),
                                      (64, 136, 8200), (16, 136, 8200)])
def test_q4_linear(dtype, group, zeros, rows, K, N):
    g = _gen(rows + K)
    w = Weight(g, 1, N, K, DT[dtype], group, zeros)
    x = _randn(g, rows, K, dtype=DT[dtype])
    y = _linear(w.arg, x)
    xa = to_f64(x)
    ref = xa @ w.val[0].T
    tol = w.order(K) * EPS * (np.abs(xa) @ w.mag[0].T)
    _within(y, ref, tol + U[DT[dtype]] * (np.abs(ref) + tol))
    if dtype == "f32" and K >= 512:
        assert np.linalg.norm(to_f64(y) - ref) <= 2e-6 * np.linalg.norm(ref)


def test_q4_linear_rows_are_independent():
    """Values that are no numbers, and huge ones, stay in their row; rows behind the
    last are not written."""
    g = _gen(9)
    for dtype, N in (("bf16", 50), ("f32", 50), ("bf16", 16450), ("bf16", 8200), ("f32", 8200)):
        w = Weight(g, 1, N, 384, DT[dtype], 64, True)
        x = _randn(g, 20, 384, dtype=DT[dtype])
        a = _linear(w.arg, x)
        x2 = x.clone()
        x2[3, 7], x2[11, 380], x2[17, 100] = math.nan, math.inf, -math.inf
        y = torch.full((30, N), 5.0, dtype=DT[dtype], device=DEV)
        moe.moe_q4_linear(w.arg, x2, y)
        keep = [r for r in range(20) if r not in (3, 11, 17)]
        assert torch.equal(y[keep], a[keep]) and (y[20:] == 5.0).all()
        x64 = to_f64(x2)
        with np.errstate(invalid="ignore"):
            ref = np.stack([(x64[r] * w.val[0]).sum(1) for r in (3, 11, 17)])
        got = to_f64(y[[3, 11, 17]])
        assert np.isnan(got[0]).all() and not np.isfinite(got).any()
        np.testing.assert_array_equal(got, ref)  # infinities keep the sign of the weight


# ------------------------------------------------------------ few-token layer

SHAPES = [
    # dtype, T, d, E, I, Is, k_max
    ("bf16", 1, 128, 2, 128, 0, 1), ("bf16", 1, 2048, 32, 768, 0, 8), ("f32", 16, 256, 8, 512, 0, 2),
    ("bf16", 3, 7168, 6, 256, 256, 4), ("f32", 5, 1152, 61, 640, 384, 6), ("bf16", 16, 512, 100, 128, 128, 33),
    ("bf16", 7, 384, 1024, 128, 0, 64), ("f32", 2, 7296, 4, 128, 128, 2), ("bf16", 9, 7296, 3, 128, 0, 3),
    ("bf16", 16, 4096, 8, 1408, 0, 2), ("f32", 1, 640, 600, 256, 128, 5), ("f32", 16, 128, 1024, 128, 128, 64),
    ("bf16", 8, 128, 1024, 128, 0, 64), ("bf16", 16, 128, 1024, 128, 128, 64),
    ("bf16", 3, 4096, 6, 128, 128, 2),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("layout", ["rowmajor", "blocked"])
def test_forward_few(shape, layout):
    dtype, T, d, E, I, Is, k_max = shape
    c = Case(T + d + E, dtype, T, d, E, I, Is, k_max, layout=layout)
    c.bias = _randn(c.gen, E, std=0.5)
    c.check(_k(c, k_max, 0, max(1, k_max // 2), 1), scale=1.5)
    c.bias = None
    c.check(_k(c, k_max))


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("group,zeros", [(32, True), (32, False), (64, True), (128, False), (128, True), (64, False)])
def test_forward_few_q4(shape, group, zeros):
    dtype, T, d, E, I, Is, k_max = shape
    if E * d * I > 2 ** 26:
        E, k_max = 8, min(k_max, 8)
    c = Case(T + d + E, dtype, T, d, E, I, Is, k_max, group, zeros)
    c.check(_k(c, k_max, 0, 1))


def test_forward_few_budgets():
    """No budget at all (with and without the always-on expert), invalid ones, both other
    policies."""
    for Is in (0, 128):
        c = Case(4, "bf16", 6, 256, 16, 128, Is, 4)
        out = c.check(_k(c, 0))
        if not Is:
            assert (out == 0).all()
        c.check(torch.tensor([-1, 4, 5, 0, 2, 1 << 30], dtype=torch.int32, device=DEV))
        c.check(_k(c, 1, 3), policy="batch_max")
        c.check(_k(c, 1, 3, 0), policy="round_up", granule=2)


def test_forward_few_no_tokens():
    c = Case(5, "bf16", 0, 128, 8, 128, 0, 2)
    out, stats, status = c.forward(torch.empty(0, dtype=torch.int32, device=DEV))
    assert (stats == 0).all() and int(status) == 0
    moe.moe_experts_few(c.desc(), c.x, torch.zeros(1, dtype=torch.int32, device=DEV),
                        torch.empty(0, dtype=torch.int32, device=DEV), torch.empty(0, device=DEV), *c.args, out,
                        moe.alloc_workspace(c.desc(), moe.MOE_OP_FEW, DEV))
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype,group", [("bf16", 0), ("f32", 0), ("bf16", 64), ("f32", 32)])
def test_forward_few_is_deterministic_and_takes_any_workspace(dtype, group):
    c = Case(6, dtype, 11, 1024, 24, 384, 256, 6, group, bool(group))
    k = _k(c, 6, 3, 0, 5)
    a = c.check(k)
    ws = moe.alloc_workspace(c.desc(), moe.MOE_OP_FEW, DEV)
    for fill in (0, 0xFF, 0x7F):
        ws.fill_(fill)
        b = c.forward(k, ws)[0]
        b2 = c.forward(k, ws)[0]
        assert torch.equal(a, b) and torch.equal(a, b2)


def test_forward_few_agrees_with_forward():
    """Against moe_forward on the same inputs, whose H and expert outputs are rounded: two
    more roundings on the way."""
    c = Case(7, "bf16", 13, 1024, 32, 512, 512, 8)
    k = _k(c, 8, 4, 0)
    a, sa, _ = c.forward(k)
    b, sb, _ = moe.forward(c.x, c.router, None, k, *c.args[:3], [t[0] for t in c.args[3:]], k_max=8)
    assert torch.equal(sa, sb)
    assert float((a.double() - b.double()).norm() / b.double().norm()) < 4 * 2.0 ** -8


def test_forward_few_values_that_are_no_numbers():
    """A token with a NaN leaves the others' outputs right (it takes other experts, so that
    the sums over the list are split elsewhere: another order, within the same bound), and a
    weight that only one token's experts hold leaves them as they are, bit for bit."""
    for dtype in ("bf16", "f32"):
        c = Case(8, dtype, 5, 256, 40, 128, 128, 3)
        k = _k(c, 3)
        a = c.forward(k)[0]
        x2 = c.x.clone()
        x2[2, 9] = math.nan
        b = c.forward(k, x=x2)[0]
        keep = [0, 1, 3, 4]
        r = moe_oracle.route(to_f64(c.x), to_f64(c.router), None, [3] * 5, 3)
        ids = np.asarray(r["ids"]).reshape(5, 3)
        routes = [(j // 3, int(e), float(w)) for j, (e, w) in enumerate(zip(r["ids"], r["w"]))]
        ref, tol = _layer_ref(to_f64(c.x), routes, c.w, c.sh, c.dt, 0, 5, 256)
        _within(a, ref, tol)
        _within(b[keep], ref[keep], tol[keep])
        assert b[2].isnan().all()
        only = [e for e in ids[0] if e not in ids[1:]]
        assert only
        for i, (n, v) in enumerate([(5, math.inf), (77, math.nan)]):
            c.args[2][only[0], n, 3] = v
            b = c.forward(k)[0]
            rest = [j for j in range(256) if j not in (5, 77)]
            # the outputs of a row with such a weight are summed again, without the matrix
            # instruction: the same products in another order
            assert torch.equal(a[:, rest], b[:, rest])
            _within(b[1:], to_f64(a[1:]), 2 * (640 + 16) * EPS * 8 + 2 * U[c.dt] * np.abs(to_f64(a[1:])))
            assert not b[0, 5].isfinite() and (i == 0 or b[0, 77].isnan())
        c.args[2][only[0], 5, 3] = 0.0
        c.args[2][only[0], 77, 3] = 0.0
        c.args[0][only[0], 5, 3] = math.inf  # a row of H
        b = c.forward(k)[0]
        assert torch.equal(a[1:], b[1:]) and not b[0].isfinite().any()


# ---------------------------------------------------------------- given routes

def _experts(c, off, ids, w, ws=None):
    out = torch.full((c.T, c.d), math.nan, dtype=c.dt, device=DEV)
    desc = c.desc()
    if ws is None:
        ws = moe.alloc_workspace(desc, moe.MOE_OP_FEW, DEV)
        ws.fill_(0x5A)
    moe.moe_experts_few(desc, c.x, off, ids, w, *c.args, out, ws)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("dtype,group", [("bf16", 0), ("f32", 0), ("bf16", 128), ("f32", 64)])
def test_experts_few(dtype, group):
    """Holes, ids out of range, an expert named twice, tokens without routes."""
    c = Case(10, dtype, 7, 384, 20, 256, 128, 6, group, False)
    rows = [[3, 19, 0], [], [-1, 5, 20, 7], [5, 5, 5, 2], [-1, -1], [1 << 30, 4], [0, 1, 2, 3, 4, 5]]
    ids = sum(rows, [])
    off = torch.tensor(np.cumsum([0] + [len(r) for r in rows]), dtype=torch.int32, device=DEV)
    pad = 7 * 6 - len(ids)
    w = _randn(c.gen, 7 * 6)
    out = _experts(c, off, torch.tensor(ids + [9] * pad, dtype=torch.int32, device=DEV), w)
    wl, at, routes = to_f64(w), 0, {}
    for t, r in enumerate(rows):
        for e in r:
            if 0 <= e < 20:
                routes[t, e] = routes.get((t, e), 0.0) + wl[at]
            at += 1
    ref, tol = _layer_ref(to_f64(c.x), [(t, e, v) for (t, e), v in routes.items()], c.w, c.sh, c.dt, group, 7, 384)
    # the weights of an expert named twice or more: two float32 additions, on any size of sum
    tol = tol + 4 * EPS * 6 * np.abs(ref).max()
    _within(out, ref, tol)


@pytest.mark.parametrize("T", [6, 12])
@pytest.mark.parametrize("dtype,group,zeros", [("bf16", 64, True), ("bf16", 32, False), ("f32", 128, True)])
def test_experts_few_q4_values_that_are_no_numbers(T, dtype, group, zeros):
    """Tokens and scales that are no numbers stay with the tokens that they belong to."""
    d = 384
    c = Case(14, dtype, T, d, 8, 256, 128, 2, group, zeros)
    off = torch.arange(T + 1, dtype=torch.int32, device=DEV) * 2
    ids = torch.tensor([[t % 4, 4 + t % 2] for t in range(T)], dtype=torch.int32, device=DEV).flatten()
    w = torch.rand(2 * T, generator=c.gen, device=DEV) + 0.5
    a = _experts(c, off, ids, w)
    wl = to_f64(w)
    routes = [(t, e, wl[2 * t + j]) for t in range(T) for j, e in enumerate((t % 4, 4 + t % 2))]
    ref, tol = _layer_ref(to_f64(c.x), routes, c.w, c.sh, c.dt, group, T, d)
    _within(a, ref, tol)
    keep = c.x.clone()
    c.x[2, 9], c.x[3, 380] = math.nan, math.inf
    b = _experts(c, off, ids, w)
    rest = [t for t in range(T) if t not in (2, 3)]
    assert torch.equal(a[rest], b[rest]) and b[2].isnan().all() and not b[3].isfinite().any()
    c.x.copy_(keep)
    # expert 1's down scale of output 7, then a gate scale of one of its columns
    mine, others = [t for t in range(T) if t % 4 == 1], [t for t in range(T) if t % 4 != 1]
    cols = [n for n in range(d) if n != 7]
    c.args[2].scales[1, 1, 7] = math.nan
    b = _experts(c, off, ids, w)
    assert b[mine, 7].isnan().all() and torch.equal(a[:, cols], b[:, cols])
    _within(b[others], ref[others], tol[others])
    c.args[2].scales[1, 1, 7] = 0.0
    c.args[0].scales[1, 0, 3] = math.inf
    b = _experts(c, off, ids, w)
    assert not b[mine].isfinite().any()
    assert torch.equal(a[others][:, cols], b[others][:, cols])


def test_experts_few_behind_grouped_routing():
    """moe_route_grouped, moe_q4_linear beside it and moe_adapt on its output, one stream."""
    c = Case(11, "bf16", 4, 512, 64, 256, 0, 8, 64, True)
    desc, rule = c.desc(), moe.make_route_rule(score="sigmoid", n_group=8, topk_group=2)
    sb = _randn(c.gen, 64, std=0.05)
    sb[10:14] = -math.inf
    k = _k(c, 8, 0, 5)
    i32 = dict(dtype=torch.int32, device=DEV)
    off, ids, w, status = torch.empty(5, **i32), torch.empty(32, **i32), torch.empty(32, device=DEV), torch.empty(1, **i32)
    proj = Weight(c.gen, 1, 192, 512, c.dt, 64, True)
    ad = moe.make_adapter_desc(4, 4, 512, 192, 8, 2, dtype=c.dt)
    a, b = _randn(c.gen, 2, 1, 8, 512, dtype=c.dt, std=0.05), _randn(c.gen, 2, 1, 192, 8, dtype=c.dt)
    own = torch.tensor([0, 1, -1, 0], **i32)
    y, out = torch.empty(4, 192, dtype=c.dt, device=DEV), torch.empty(4, 512, dtype=c.dt, device=DEV)
    moe.moe_route_grouped(desc, rule, c.x, c.router, None, sb, k, off, ids, w, status,
                          moe.alloc_workspace(desc, moe.MOE_OP_ROUTE_GROUPED, DEV))
    moe.moe_experts_few(desc, c.x, off, ids, w, *c.args, out, moe.alloc_workspace(desc, moe.MOE_OP_FEW, DEV))
    moe.moe_q4_linear(proj.arg, out, y)
    y0 = y.clone()
    moe.moe_adapt(ad, out, None, a, b, None, None, own, None, None, y, y, moe.alloc_adapt_workspace(ad))
    torch.cuda.synchronize()
    o = off.cpu().numpy()
    routes = [(t, int(ids[j]), float(w[j])) for t in range(4) for j in range(o[t], o[t + 1]) if int(ids[j]) >= 0]
    ref, tol = _layer_ref(to_f64(c.x), routes, c.w, None, c.dt, 64, 4, 512)
    _within(out, ref, tol)
    oa = to_f64(out)
    pr = oa @ proj.val[0].T
    pt = proj.order(512) * EPS * (np.abs(oa) @ proj.mag[0].T)
    _within(y0, pr, pt + U[c.dt] * (np.abs(pr) + pt))
    assert torch.equal(y[2], y0[2])
    aa, ba = to_f64(a), to_f64(b)
    for r in (0, 1, 3):
        i = int(own[r])
        v = aa[i, 0] @ oa[r]
        full = to_f64(y0[r]) + ba[i, 0] @ v
        slack = 600 * EPS * (np.abs(ba[i, 0]) @ (np.abs(aa[i, 0]) @ np.abs(oa[r]))) + 2.0 ** -16 * (np.abs(ba[i, 0]) @ np.abs(v))
        _within(y[r], full, slack + U[c.dt] * (np.abs(full) + slack))


# ---------------------------------------------------------- streams and graphs

def test_few_graph_replays_with_other_inputs():
    """Two captured layers and a linear that share a workspace (one stream), replayed
    between eager runs, with budgets and activations that change."""
    c = Case(12, "bf16", 8, 1024, 32, 384, 128, 6)
    c4 = Case(13, "bf16", 8, 1024, 32, 384, 128, 6, 64, True)
    proj = Weight(c.gen, 1, 500, 1024, c.dt, 128, False)
    k = _k(c, 6, 2, 0)
    desc = c.desc()
    ws = moe.alloc_workspace(desc, moe.MOE_OP_FEW, DEV)
    o1, s1, t1 = c.outputs()
    o2, s2, t2 = c.outputs()
    y = torch.empty(8, 500, dtype=c.dt, device=DEV)
    x = c.x.clone()

    def step():
        moe.moe_forward_few(desc, x, c.router, None, k, *c.args, o1, s1, t1, ws)
        moe.moe_forward_few(desc, o1, c.router, None, k, *c4.args, o2, s2, t2, ws)
        moe.moe_q4_linear(proj.arg, o2, y)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(5):
        x.copy_(_randn(c.gen, 8, 1024, dtype=c.dt))
        k.copy_(torch.randint(0, 7, (8,), generator=c.gen, device=DEV, dtype=torch.int32))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (o1, s1, o2, s2, y)]
        for t in (o1, o2, y):
            t.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (o1, s1, o2, s2, y)):
            assert torch.equal(a, b)


def test_few_on_two_streams_at_once():
    """Calls with their own workspaces on two streams, many in flight."""
    cs = [Case(20 + i, "bf16", 3, 2048, 16, 512, 0, 4, 0 if i else 128) for i in range(2)]
    ks = [_k(c, 4, 3) for c in cs]
    want = [c.forward(k)[0] for c, k in zip(cs, ks)]
    streams = [torch.cuda.Stream() for _ in cs]
    wss = [moe.alloc_workspace(c.desc(), moe.MOE_OP_FEW, DEV) for c in cs]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for c, k, s, ws in zip(cs, ks, streams, wss):
            with torch.cuda.stream(s):
                got.append(c.forward(k, ws, s)[0])
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 2])
