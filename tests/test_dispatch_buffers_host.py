"""The buffers that a dispatch of e4m3 rows writes: scales of another type than
fp32 are refused (the kernel writes four bytes for each).  Host checks only."""
import pytest
import torch

from combine_routing_preprocess_amd import Dispatcher

T, H, E, K = 8, 256, 4, 2


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float64, torch.int32, torch.uint8])
@pytest.mark.parametrize("call", ["permute", "dispatch"])
def test_scales_of_another_type_are_refused(call, dtype):
    d = Dispatcher(T, H, E, K, payload="fp8", device="cpu")
    x, xs = torch.zeros(T, H, dtype=torch.uint8), torch.ones(T, H // 128)
    scales = torch.zeros(d.R, H // 128, dtype=dtype)
    routing = torch.zeros(T, K, dtype=torch.int16)
    with pytest.raises(ValueError, match="out_scales must be float32"):
        if call == "permute":
            d.permute(x, xs, out_scales=scales)
        else:
            d.dispatch(x, routing, x_scales=xs, out_scales=scales)
