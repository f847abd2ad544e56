"""Host side of the few-token layer's refusals of overlapping buffers.  No GPU needed: every
call is refused before anything is launched."""
import ctypes

import pytest

from mixture_experts_layer_token_amd import _lib
from tests.test_few_host import FAKE, SHAPE, _desc, _experts, _few_size, _forward, _q4

P = ctypes.c_void_p


def _at(base, off):
    return P(base.value + off)


@pytest.mark.parametrize("call", [_forward, _experts])
@pytest.mark.parametrize("four", [False, True])
def test_out_must_not_overlap_what_the_call_reads(call, four):
    """Weights, their scales and zero points (by their last bytes) and the workspace, where an
    output would be written over the list that other workgroups still read."""
    d = _desc(T=4, d=256, E=8, I=128, I_shared=384)
    out_b = 4 * 256 * 2
    q4 = _q4(group=32) if four else None
    shapes = [(8, 128, 256), (8, 128, 256), (8, 256, 128), (1, 384, 256), (1, 384, 256), (1, 256, 384)]
    for i, (G, N, K) in enumerate(shapes):
        n = G * N * K
        w = FAKE[4 + i]
        size = n // 2 if four else 2 * n
        for at in (0, size // 32 * 16, size - 16, 16 - out_b):
            assert call(d, q4=q4, out=_at(w, at)) == SHAPE, (i, at)
        if four:
            for base, size in (((i + 20) << 32, n // 32 * 2), ((i + 30) << 32, n // 32)):
                assert call(d, q4=q4, out=P(base + size - 16)) == SHAPE, i
    ws = 1 << 20
    need = _few_size(d)[1]
    for at in (0, need // 2 & ~255, need - 16, 16 - out_b):
        assert call(d, q4=q4, ws=P(ws), n=need, out=P(ws + at)) == SHAPE, at
    if call is _forward:
        assert call(d, q4=q4, out=_at(FAKE[1], 8 * 256 * 2 - 16)) == SHAPE


def test_counts_and_status_must_not_lie_in_the_workspace():
    d, ws = _desc(), 1 << 20
    need = _few_size(d)[1]
    a = [FAKE[i] for i in range(10)]
    call = lambda stats, status: _lib.load().moe_forward_few(ctypes.byref(d), *a, None, FAKE[11], stats, status, P(ws),
                                                             need, None)
    for at in (0, need // 2, need - 4):
        assert call(P(ws + at), None) == SHAPE and call(None, P(ws + at)) == SHAPE
    assert call(P(ws - 4), None) == SHAPE
