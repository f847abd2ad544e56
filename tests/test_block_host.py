"""Host side of the operators around the layer: workspaces, BlockLayer's checks,
devices and streams.  No GPU needed: nothing is launched."""
import ctypes

import pytest
import torch

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


class _Devices:
    """Stands in for torch.cuda's current device and streams, and for the steps of a
    BlockLayer: notes the device that is current and the stream of each step."""

    STEPS = ("moe_norm", "moe_route_grouped", "moe_permute", "moe_ffn", "moe_ffn_plan", "moe_ffn_gateup", "moe_ffn_down",
             "moe_adapt", "moe_combine_norm")

    def __init__(self, monkeypatch):
        self.current, self.calls, outer = [], [], self

        class device:
            def __init__(self, d):
                self.d = d

            def __enter__(self):
                outer.current.append(self.d)

            def __exit__(self, *exc):
                outer.current.pop()

        monkeypatch.setattr(torch.cuda, "device", device)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: ("stream", d))
        for name in self.STEPS:
            monkeypatch.setattr(moe, name, lambda *a, _n=name: self.calls.append((_n, a, list(self.current))))


def _block(adapters=0, shared_adapters=0, T=6, d=128, **kw):
    desc = moe.make_desc(T, d, 8, 128, 2, I_shared=128)
    layer = moe.BlockLayer(desc, moe.make_route_rule(), moe.make_norm_desc(T, d), moe.make_norm_desc(T, d), rank=8,
                           adapters=adapters, shared_adapters=shared_adapters, device="cpu")
    z = torch.zeros(1)
    ad = lambda n: (z,) * 5 if n else None
    args = dict(y=z, resid=z, pre_w=z, w_router=z, select_bias=None, k=z, w_gate=z, w_up=z, w_down=z, resid_out=z, x_out=z,
                shared=(z, z, z), adapters=ad(adapters), shared_adapters=ad(shared_adapters))
    return layer, {**args, **kw}


@pytest.mark.parametrize("adapters,shared_adapters", [(0, 0), (3, 0), (0, 2), (3, 2)])
@pytest.mark.parametrize("stream", [None, "own"])
def test_block_layer_runs_all_steps_on_one_device_and_stream(monkeypatch, adapters, shared_adapters, stream):
    layer, args = _block(adapters, shared_adapters)
    dev = _Devices(monkeypatch)
    layer.run(**args, stream=stream)
    here = layer.x.device
    assert [c[0] for c in dev.calls[:3]] == ["moe_norm", "moe_route_grouped", "moe_permute"]
    assert dev.calls[-1][0] == "moe_combine_norm"
    for name, a, current in dev.calls:
        assert a[-1] == (stream or ("stream", here)), name
        assert current == [here], name


def test_block_layer_passes_norm_biases(monkeypatch):
    layer, args = _block()
    dev = _Devices(monkeypatch)
    layer.run(**args, before_post_w="w0", before_post_b="b0", pre_b="b1", behind_post_w="w2", behind_post_b="b2",
              next_w="w3", next_b="b3")
    assert dev.calls[0][1][3:8] == ("w0", "b0", None, args["pre_w"], "b1")
    assert dev.calls[-1][1][8:13] == ("w2", "b2", None, "w3", "b3")


@pytest.mark.parametrize("name", ["w_gate", "w_up", "w_down", "shared"])
def test_block_layer_refuses_weights_elsewhere(monkeypatch, name):
    layer, args = _block()
    dev = _Devices(monkeypatch)
    far = torch.zeros(1, device="meta")
    args[name] = (args["w_up"], far, far) if name == "shared" else far
    with pytest.raises(ValueError, match="on meta, the layer is on cpu"):
        layer.run(**args)
    assert not dev.calls


def test_grouped_routing_of_more_tokens_than_the_screened_grid_holds():
    size = lambda T, router: _size(moe.make_desc(T, 128, 2, 128, 1, router=router), moe.MOE_OP_ROUTE_GROUPED)
    # the tile kernel adds the squared norms to half the bytes of float64 slices
    T = (1 << 28) + 64
    assert size(T, "screened") == size(T, "float64") == T * 2 * 8


@pytest.mark.parametrize("which", ["before", "behind"])
@pytest.mark.parametrize("kw", [dict(T=5), dict(T=7), dict(d=256), dict(dtype=torch.float32)])
def test_block_layer_refuses_norms_of_other_shapes(which, kw):
    """Fewer rows in the norm before the block would leave the rest of its input as it was."""
    shape = dict(T=6, d=128, dtype=torch.bfloat16)
    nd = {"before": moe.make_norm_desc(**shape), "behind": moe.make_norm_desc(**shape)}
    nd[which] = moe.make_norm_desc(**{**shape, **kw})
    with pytest.raises(ValueError, match=which):
        moe.BlockLayer(moe.make_desc(6, 128, 8, 128, 2), moe.make_route_rule(), nd["before"], nd["behind"], device="cpu")
