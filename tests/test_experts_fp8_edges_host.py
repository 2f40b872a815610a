"""What the 8-bit experts refuse beyond wrong shapes and pointers, before anything touches a device."""
import ctypes

import pytest
import torch

lm = pytest.importorskip("sigmoid_top_routing_latentmoe_b200")

FAKE = 1 << 20                                           # never dereferenced: checks fail first


def test_caps_of_the_hidden_units():
    """A product of caps that fp32 does not hold, or a cap whose reciprocal it does not hold, is refused: a hidden
    unit could be infinite, which 8 bits are not to hide."""
    def ffn(b1, b2):
        dims = lm.make_dims(8, 64, 128, 24, 4, 0, 256, 0, beta1=b1, beta2=b2)
        return lm._lib.moe_expert_ffn_fp8(ctypes.byref(dims), None, FAKE, FAKE, ctypes.byref(lm.Fp8Experts(*[FAKE] * 6)),
                                          FAKE, FAKE, 1 << 30, None)
    for caps in ((1e20, 1e20), (4.0, 3e38), (float("inf"), 1.0), (1.0, float("inf")), (1e-39, 25.0), (4.0, 1e-40)):
        assert ffn(*caps) == lm.EUNSUPPORTED, caps
    for caps in ((4.0, 25.0), (1e19, 1e18), (1e-37, 3e38), (4.0, 1e30)):    # taken: z is what is missing
        assert ffn(*caps) == lm.EINVAL and b"z is NULL" in lm._lib.lmoe_last_error(), caps


@pytest.mark.parametrize("ws", [torch.zeros(1 << 16, dtype=torch.uint8), FAKE, None], ids=["host", "pointer", "none"])
def test_workspace_has_to_be_on_the_device(ws):
    """A workspace in host memory would be an address that the kernels cannot use."""
    d = lm.make_dims(8, 64, 128, 24, 4, 0, 256, 0)
    for call in (lambda: lm.moe_route_grouped(d, lm.make_route_rule(), None, None, None, None, None, ws),
                 lambda: lm.moe_expert_gemm_fp8(d, None, None, None, torch.zeros(24, 128, 128), None, None, ws),
                 lambda: lm.moe_expert_ffn_fp8(d, *[None] * 10, ws)):
        with pytest.raises(lm.LmoeError, match="ws: expected"):
            call()
