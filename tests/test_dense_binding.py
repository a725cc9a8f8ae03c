"""The Python binding of the layer calls without a GPU: what it refuses before it
asks for a device."""
import pytest

import dense_gemm_14_amd as g

SIZES = [(g.bias_act_res_workspace_size, 3, ()), (g.gated_workspace_size, 3, ()), (g.gated_bwd_workspace_size, 3, ()),
         (g.bias_act_bwd_workspace_size, 3, (g.ACT_NONE,)), (g.newton_schulz_workspace_size, 3, ())]


@pytest.mark.parametrize("far", [1 << 31, 1 << 32, (1 << 32) + 8, -(1 << 32) + 8, 1 << 70])
@pytest.mark.parametrize("fn,count,rest", SIZES, ids=[s[0].__name__ for s in SIZES])
def test_sizes_beyond_32_bits_are_refused(fn, count, rest, far):
    # (cut to 32 bits, 2^32 would be an empty product that needs no workspace)
    for i in range(count):
        sizes = [far if j == i else 0 for j in range(count)]
        with pytest.raises(OverflowError):
            fn(*sizes, *rest)


def test_newton_schulz_refuses_numbers_beyond_32_bits():
    ok = dict(batch=1, rows=64, cols=64, G=1 << 40, O=1 << 41, steps=5, workspace=1 << 42, workspace_bytes=1 << 30,
              stream=1 << 43, g_type=g.BF16)
    for name in ("batch", "rows", "cols", "steps", "g_type"):
        with pytest.raises(OverflowError):
            g.newton_schulz(**{**ok, name: 1 << 32})
    with pytest.raises(OverflowError):
        g.bias_act_bwd_workspace_size(8, 8, 8, 1 << 32)
    with pytest.raises(OverflowError):
        g.force_layer_kernel(1 << 32)


def test_a_negative_workspace_size_is_refused():
    # (as an unsigned size it would pass for any need)
    with pytest.raises(ValueError, match="workspace_bytes"):
        g._workspace(1 << 42, -1)

    class Held:
        nbytes = 64

    with pytest.raises(ValueError, match="workspace_bytes"):
        g._workspace(Held(), -1)


def test_tensors_of_another_type_are_refused():
    import torch
    for t in (torch.float32, torch.float16, torch.float64, torch.complex64, torch.float8_e4m3fn):
        with pytest.raises(TypeError, match="A: expected"):
            g._typed_addr(torch.zeros(8, dtype=t), 0, "A")
    # BF16, and integers as its bits, get as far as the device check
    for t in (torch.bfloat16, torch.int16, torch.uint8):
        with pytest.raises(ValueError, match="on the GPU"):
            g._typed_addr(torch.zeros(8, dtype=t), 0, "A")
    with pytest.raises(ValueError, match="on the GPU"):
        g._typed_addr(torch.zeros(8), 0, "G", None, torch.float32)
    with pytest.raises(TypeError, match="float32"):
        g._typed_addr(torch.zeros(8, dtype=torch.bfloat16), 0, "G", None, torch.float32)
    assert g._typed_addr(None, 8, "A") is None and g._typed_addr(64, 8, "A") == 64
