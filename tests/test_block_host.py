"""Host side of the operators around the layer: workspaces, BlockLayer's checks,
devices and streams.  No GPU needed: nothing is launched."""
import ctypes

import pytest

import mixture_experts_layer_token_amd as moe
from mixture_experts_layer_token_amd import _lib

P = ctypes.c_void_p
FAKE = [P((i + 1) << 24) for i in range(14)]  # never dereferenced: every call is refused first


def _size(desc, op):
    n = ctypes.c_size_t(0)
    assert _lib.load().moe_workspace_size(ctypes.byref(desc), op, ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("shape,need", [((512, 7168, 256, 128, 1), 16781312), ((640, 5120, 256, 128, 1), None),
                                        ((64, 4096, 8, 14336, 2), None), ((4096, 7168, 256, 2048, 8), None)])
def test_forward_asks_for_no_more_than_it_uses(shape, need):
    """moe_forward takes a workspace of the size that it and the operators older than
    grouped routing ask for, though MOE_OP_FORWARD names one that is enough for all."""
    T, d, E, I, k_max = shape
    desc = moe.make_desc(T, d, E, I, k_max)
    sizes = {op: _size(desc, op) for op in range(8)}
    assert sizes[moe.MOE_OP_FORWARD] == max(sizes.values())
    if need is None:
        need = sizes[moe.MOE_OP_FORWARD]
    # an address off 256 bytes: MOE_ERR_ALIGN once the size is enough, before any launch
    call = lambda n: _lib.load().moe_forward(ctypes.byref(desc), *FAKE[:11], None, None, P((1 << 20) + 16), n, None)
    assert call(need) == 5
    if need < sizes[moe.MOE_OP_FORWARD]:
        assert call(need - 256) == 4
