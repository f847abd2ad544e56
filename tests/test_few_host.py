"""Host side of the few-token layer and the 4-bit weights: sizes, refusals, the oracle's
pins.  No GPU needed: nothing is launched."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import mixture_experts_layer_token_amd as moe
from mixture_experts_layer_token_amd import _lib
from oracle import quant

P = ctypes.c_void_p
FAKE = [P((i + 1) << 32) for i in range(16)]  # never dereferenced: every call is refused first
OK, NULL, SHAPE, UNSUPPORTED, WORKSPACE, ALIGN = 0, 1, 2, 3, 4, 5


def _few_size(desc):
    n = ctypes.c_size_t(0)
    return _lib.load().moe_workspace_size(ctypes.byref(desc), moe.MOE_OP_FEW, ctypes.byref(n)), n.value


def _desc(T=4, d=256, E=8, I=128, k_max=2, **kw):
    return moe.make_desc(T, d, E, I, k_max, **kw)


def test_workspace():
    st, n = _few_size(_desc())
    assert st == OK and n % 256 == 0 and n >= 4 * 2 * 128 * 2
    assert n <= moe.workspace_size(_desc(), moe.MOE_OP_FORWARD)
    assert _few_size(_desc(T=0))[0] == OK
    assert _few_size(_desc(T=16))[0] == OK and _few_size(_desc(T=17))[0] == SHAPE
    assert _few_size(_desc(E=128, k_max=64))[0] == OK and _few_size(_desc(E=128, k_max=65))[0] == SHAPE
    # one expert's six weights in codes keep float32 H in three parts
    f = _few_size(_desc(dtype=torch.float32))[1]
    assert f >= 4 * 2 * 128 * 6


def _forward(desc, q4=None, ws=P(1 << 20), n=1 << 40, **kw):
    names = ("x", "w_router", "bias", "k", "gate", "up", "down", "s_gate", "s_up", "s_down")
    a = [kw.get(v, FAKE[i]) for i, v in enumerate(names)]
    return _lib.load().moe_forward_few(ctypes.byref(desc), *a, q4, kw.get("out", FAKE[11]), None, None, ws, n, None)


def _experts(desc, q4=None, ws=P(1 << 20), n=1 << 40, **kw):
    names = ("x", "tok_off", "ids", "w", "gate", "up", "down", "s_gate", "s_up", "s_down")
    a = [kw.get(v, FAKE[i]) for i, v in enumerate(names)]
    return _lib.load().moe_experts_few(ctypes.byref(desc), *a, q4, kw.get("out", FAKE[11]), ws, n, None)


def _q4(group=64, zeros=True, n=6):
    q = _lib.moe_few_q4()
    q.group = group
    for i in range(n):
        q.scales[i] = (i + 20) << 32
        q.zeros[i] = (i + 30) << 32 if zeros else None
    return q


@pytest.mark.parametrize("call", [_forward, _experts])
def test_few_refusals(call):
    d, sh = _desc(), _desc(I_shared=128)
    off = P((1 << 33) + 8)
    for name in ("x", "gate", "up", "down", "out") + (("w_router", "k") if call is _forward else ("tok_off", "ids", "w")):
        assert call(d, **{name: None}) == NULL, name
    for name in ("s_gate", "s_up", "s_down"):
        assert call(sh, **{name: None}) == NULL, name
    for name in ("x", "gate", "up", "down", "out"):
        assert call(d, **{name: off}) == ALIGN, name
    assert call(sh, s_up=off) == ALIGN
    assert call(_desc(T=17)) == SHAPE and call(_desc(E=100, k_max=65)) == SHAPE
    assert call(d, out=FAKE[0]) == SHAPE                       # in place
    assert call(d, out=P((1 << 32) + 1024)) == SHAPE           # in part
    assert call(d, ws=None) == WORKSPACE
    n = _few_size(d)[1]
    assert call(d, n=n - 1) == WORKSPACE and call(d, ws=P((1 << 20) + 16), n=n) == ALIGN
    for g in (0, 16, 96, 256, -32):
        assert call(d, q4=_q4(g)) == UNSUPPORTED
    q = _q4()
    q.scales[1] = None
    assert call(d, q4=q) == NULL
    q = _q4()
    q.zeros[2] = None
    assert call(d, q4=q) == NULL                               # some with zero points, some without
    q = _q4()
    q.scales[2] = (1 << 40) + 4
    assert call(d, q4=q) == ALIGN
    q = _q4(n=3)
    assert call(sh, q4=q) == NULL                              # the always-on expert's scales


def _qd(G=1, N=64, K=256, group=64, zeros=0, dtype=moe.MOE_BF16):
    return _lib.moe_q4_desc(G, N, K, group, zeros, dtype)


def _bytes(qd):
    n = [ctypes.c_size_t(0) for _ in range(3)]
    st = _lib.load().moe_q4_bytes(ctypes.byref(qd), *(ctypes.byref(v) for v in n))
    return st, tuple(v.value for v in n)


def test_q4_sizes():
    assert _bytes(_qd()) == (OK, (4 * 2 * 1024, 4 * 64 * 2, 0))
    assert _bytes(_qd(G=3, N=65, K=264, group=32, zeros=1, dtype=moe.MOE_F32)) == \
        (OK, (3 * 5 * 3 * 1024, 3 * 12 * 80 * 4, 3 * 12 * 80))
    assert _bytes(_qd(G=0))[0] == OK
    for kw, code in [(dict(G=-1), SHAPE), (dict(G=1 << 20), SHAPE), (dict(N=0), SHAPE), (dict(N=262145), SHAPE),
                     (dict(K=0), SHAPE), (dict(K=4), SHAPE), (dict(K=100), SHAPE), (dict(K=65544), SHAPE),
                     (dict(group=0), UNSUPPORTED), (dict(group=256), UNSUPPORTED), (dict(zeros=2), UNSUPPORTED),
                     (dict(dtype=2), UNSUPPORTED)]:
        assert _bytes(_qd(**kw))[0] == code, kw


@pytest.mark.parametrize("zeros", [0, 1])
def test_q4_refusals(zeros):
    lib, qd = _lib.load(), _qd(zeros=zeros)
    w, c, s, y = FAKE[0], FAKE[1], FAKE[2], FAKE[4]
    z, no = (FAKE[3], None) if zeros else (None, FAKE[3])
    off = P((1 << 34) + 4)
    z_code = NULL if zeros else UNSUPPORTED
    b = ctypes.byref
    pack = lambda w=w, c=c, s=s, z=z, qd=qd: lib.moe_q4_pack(b(qd), w, c, s, z, None)
    unpack = lambda w=w, c=c, s=s, z=z, qd=qd: lib.moe_q4_unpack(b(qd), c, s, z, w, None)
    tile = lambda w=w, c=c, s=s, z=z, qd=qd: lib.moe_q4_tile(b(qd), w, FAKE[5], FAKE[6] if zeros else None, c, s, z, None)
    lin = lambda w=w, c=c, s=s, z=z, qd=qd: lib.moe_q4_linear(b(qd), 4, w, c, s, z, y, None)
    for f in (pack, unpack, tile, lin):
        assert f(w=None) == NULL and f(c=None) == NULL and f(s=None) == NULL and f(z=no) == z_code
        assert f(w=off) == ALIGN and f(c=off) == ALIGN and f(s=off) == ALIGN
        assert f(qd=_qd(K=12, zeros=zeros)) == SHAPE
        if zeros:
            assert f(z=off) == ALIGN
    for f in (pack, unpack, tile):
        assert f(c=w) == SHAPE and f(s=P((1 << 32) + 16)) == SHAPE
        assert f(w=None, c=None, qd=_qd(G=0, zeros=zeros)) == OK
    assert lib.moe_q4_linear(b(qd), -1, w, c, s, z, y, None) == SHAPE
    assert lib.moe_q4_linear(b(qd), 65537, w, c, s, z, y, None) == SHAPE
    assert lib.moe_q4_linear(b(_qd(G=2, zeros=zeros)), 1, w, c, s, z, y, None) == SHAPE
    assert lib.moe_q4_linear(b(qd), 0, None, None, None, None, None, None) == OK
    assert lib.moe_q4_linear(b(qd), 4, w, c, s, z, w, None) == SHAPE
    assert lib.moe_q4_linear(b(qd), 4, w, c, s, z, P((2 << 32) + 512), None) == SHAPE


def test_binding_refuses():
    cpu = torch.zeros(64, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.q4_pack(cpu.t())
    with pytest.raises(ValueError):
        moe.q4_tile(torch.zeros(4, dtype=torch.uint8), torch.zeros(1))
    with pytest.raises(ValueError, match="scales"):
        moe.q4_tile(torch.zeros(16, 128, dtype=torch.uint8), torch.zeros(16, 3))
    with pytest.raises(moe.MoeError):
        moe.alloc_q4(1, 16, 100, device="cpu")
    q = moe.alloc_q4(2, 20, 136, group=32, zeros=True, device="cpu")
    assert q.codes.numel() == 2 * 2 * 2 * 1024 and q.scales.shape == q.zeros.shape == (2, 8, 32)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_q4_unpack(q, torch.zeros(2, 20, 136))
    with pytest.raises(ValueError, match="x: shape"):
        moe.moe_q4_linear(q, torch.zeros(3, 128), torch.zeros(3, 20))


def test_few_weights_must_match(monkeypatch):
    """Kinds, shapes, groups and zero points of 4-bit weights beside each other."""
    monkeypatch.setattr(moe._Args, "__call__", lambda self, t, name, dtype=None, numel=0: None if t is None else 1 << 20)
    d = _desc(I_shared=384)
    mk = lambda G, N, K, **kw: moe.alloc_q4(G, N, K, device="cpu", **{"group": 64, **kw})
    good = [mk(8, 128, 256), mk(8, 128, 256), mk(8, 256, 128), mk(1, 384, 256), mk(1, 384, 256), mk(1, 256, 384)]
    args, q4 = moe._few_weights(moe._Args(), d, good)
    assert args == [1 << 20] * 6 and q4.group == 64 and q4.zeros[0] is None
    for i, w in [(1, mk(8, 256, 128)), (2, mk(8, 128, 256)), (3, mk(1, 128, 256)), (1, mk(4, 128, 256)),
                 (2, mk(8, 256, 128, group=32)), (4, mk(1, 384, 256, zeros=True)),
                 (0, mk(8, 128, 256, dtype=torch.float32))]:
        with pytest.raises(ValueError):
            moe._few_weights(moe._Args(), d, good[:i] + [w] + good[i + 1:])
    with pytest.raises(TypeError):
        moe._few_weights(moe._Args(), d, good[:1] + [torch.zeros(1)] + good[2:])


# ------------------------------------------------------------- pins of the oracle

def _rne(q: Fraction) -> int:
    return round(q)  # ties to even


@pytest.mark.parametrize("zeros", [False, True])
def test_quantise_against_rational_arithmetic(zeros):
    """Codes by exact fractions from the stored scale; the scale by hand for float64."""
    rng = np.random.default_rng(4)
    w = np.round(rng.normal(size=(6, 40)) * 64) / 64
    w[1] = np.abs(w[1])
    w[2] = 0
    codes, s, z = quant.q4_quantise(w, 32, zeros, lambda v: v.astype(np.float32).astype(np.float64))
    for n in range(6):
        for g, (a, e) in enumerate([(0, 32), (32, 40)]):
            v = [Fraction(float(x)) for x in w[n, a:e]]
            sc = Fraction(float(s[n, g]))
            if zeros:
                want = (max(max(v), 0) - min(min(v), 0)) / 15
            else:
                want = max(abs(x) for x in v) / 7
            assert abs(sc - want) <= abs(want) * Fraction(1, 2 ** 24)
            if sc == 0:
                assert (codes[n, a:e] == (0 if zeros else 8)).all()
                continue
            zp = min(max(_rne(-min(min(v), Fraction(0)) / sc), 0), 15) if zeros else 8
            assert not zeros or z[n, g] == zp
            for k, x in enumerate(v):
                assert codes[n, a + k] == min(max(_rne(x / sc) + zp, 0 if zeros else 1), 15)


def test_quantised_values_are_near():
    """No value moves by more than half a step, but for those that the border cuts."""
    rng = np.random.default_rng(5)
    w = rng.normal(size=(20, 256))
    for zeros in (False, True):
        codes, s, z = quant.q4_quantise(w, 64, zeros, lambda v: v)
        err = np.abs(quant.q4_values(codes, s, z, 64) - w)
        step = np.repeat(s, 64, -1)
        assert (err <= (1.0 if zeros else 0.5) * step * (1 + 1e-12)).all()
        assert (codes.min() >= (0 if zeros else 1)) and codes.max() <= 15


def test_values_and_order_by_hand():
    codes = np.array([[0, 15, 8, 3, 1, 2]])
    assert quant.q4_values(codes, np.array([[2.0, 0.5]]), None, 4).tolist() == [[-16, 14, 0, -10, -3.5, -3]]
    assert quant.q4_values(codes, np.array([[2.0, 0.5]]), np.array([[1, 2]]), 4).tolist() == [[-2, 28, 14, 4, -0.5, 0]]
    assert quant.q4_unpair(np.array([[0xF0, 0x38, 0x21]])).tolist() == codes.tolist()
    t = quant.q4_tile(np.arange(16 * 128).reshape(16, 128) % 16, 16, 128).view(np.uint32)
    assert t.size == 256
    # row 0, inputs 0..7 hold 0..7: pairs (0,1) (2,3) .. in the halves of the word
    assert t[0] == 0x75316420
    one = np.zeros((33, 200), dtype=int)
    one[32, 199] = 5  # third row tile, second input tile: input 71 of it, word i = 2, lanes 0..
    b = quant.q4_tile(one, 33, 200).view(np.uint32)
    at = (2 * 2 + 1) * 256 + ((71 // 8 % 4) * 16 + 0) * 4 + 71 // 32
    assert b[at] == 5 << (4 * 3 + 16) and np.count_nonzero(b) == 1
