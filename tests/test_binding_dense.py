"""The binding's own refusals of the norm, the dense products and the pre-norm
layer, without a GPU: tensors that say they are on a device, and a library that
fails the test when a call reaches it."""
import pytest
import torch

from group_limited_routed_moe_b200 import moe


class OnDevice(torch.Tensor):
    index = 0

    def get_device(self):
        return self.index


class OnAnotherDevice(OnDevice):
    index = 1


class NoLibrary:
    """Sizes as the library gives them; a call that would launch is an error."""
    sizes = ("_bytes",)

    def __getattr__(self, name):
        if name.endswith(self.sizes):
            return getattr(moe._lib_for_test, name)

        def reached(*_):
            pytest.fail(f"{name} was reached")
        return reached


@pytest.fixture
def no_library(monkeypatch):
    monkeypatch.setattr(moe, "_lib_for_test", moe.lib, raising=False)
    monkeypatch.setattr(moe, "lib", NoLibrary())
    monkeypatch.setattr(moe, "_current_device", lambda: 0)
    monkeypatch.setattr(moe, "_raw_stream", lambda _: 0)


def dev(shape, dtype=torch.bfloat16, kind=OnDevice):
    return torch.zeros(shape, dtype=dtype).as_subclass(kind)


def bad_memory(nbytes):
    """Memory that is large enough, and yet none that a kernel may take."""
    wide = torch.zeros(2 * nbytes, dtype=torch.uint8)
    return {"host": wide[:nbytes], "other device": wide[:nbytes].as_subclass(OnAnotherDevice),
            "strided": wide.as_subclass(OnDevice)[::2], "not a tensor": bytearray(nbytes)}


BAD = ["host", "other device", "strided", "not a tensor"]


@pytest.mark.parametrize("which", BAD)
def test_layer_normed_workspace(no_library, which):
    T = 4
    x = dev((T, moe.HIDDEN))
    router = dev(moe.lib.moe_router_packed_bytes(), torch.uint8)
    packed = torch.empty(moe.lib.moe_packed_weight_bytes(), dtype=torch.uint8).as_subclass(OnDevice)
    ws = bad_memory(moe.layer_normed_workspace_bytes(T))[which]
    with pytest.raises(ValueError, match="workspace"):
        moe.moe_layer_normed(x, None, None, 1e-6, router, None, packed, out=dev((T, moe.HIDDEN)), workspace=ws)


@pytest.mark.parametrize("which", BAD)
def test_backward_workspaces(no_library, which):
    T, H, I = 4, 64, 72
    x = dev((T, H))
    w, wd = dev((H, I)), dev((I, H))
    ws = bad_memory(moe.lib.moe_add_rmsnorm_backward_workspace_bytes(T, H))[which]
    with pytest.raises(ValueError, match="workspace"):
        moe.moe_add_rmsnorm_backward(x, x, dx=dev((T, H)), dweight=dev((H,), torch.float32), workspace=ws)
    saved = dev((moe._saved_layout(T, I)[1],), torch.uint8)
    ws = bad_memory(moe.lib.moe_gated_ffn_backward_workspace_bytes(T, I))[which]
    with pytest.raises(ValueError, match="workspace"):
        moe.moe_gated_ffn_backward(x, x, w, w, wd, saved, dx=dev((T, H)), dw_gate=dev((H, I)), dw_up=dev((H, I)),
                                   dw_down=dev((I, H)), workspace=ws)


@pytest.mark.parametrize("name", ["a", "a_scale", "b", "b_scale", "bias", "out"])
def test_int8_arguments_that_are_no_tensors(no_library, name):
    args = {"a": dev((4, 64), torch.int8), "a_scale": dev((4,), torch.float32), "b": dev((8, 64), torch.int8),
            "b_scale": dev((8,), torch.float32), "bias": dev((8,), torch.float32), "out": dev((4, 8))}
    args[name] = 0.5
    with pytest.raises(ValueError, match=name):
        moe.moe_int8_matmul(**args)
