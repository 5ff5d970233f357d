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


@pytest.mark.parametrize("rows,out", [(torch.float8_e4m3fn, torch.uint8), (torch.uint8, torch.float8_e4m3fn),
                                      (torch.uint8, torch.uint8), (torch.float8_e4m3fn, torch.float8_e4m3fn)])
def test_codes_go_into_a_buffer_of_either_type(monkeypatch, rows, out):
    """Codes are taken as uint8 or float8_e4m3fn everywhere, so also out of one into the other: layer(rms=), whose norm
    writes float8_e4m3fn, with a caller's uint8 perm.  The library is replaced: no kernel runs."""
    from combine_routing_preprocess_amd import _abi as A
    from combine_routing_preprocess_amd import api

    reached = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: reached.append(name) or 0

    d = Dispatcher(T, H, E, K, payload="fp8", device="cpu")
    x, xs = torch.zeros(T, H, dtype=rows), torch.ones(T, H // 128)
    buf = torch.zeros(d.R, H, dtype=out)
    monkeypatch.setattr(A, "lib", lambda: Library())
    monkeypatch.setattr(api, "_stream", lambda: 0)
    got, _ = d.permute(x, xs, out=buf)
    perm, *_ = d.dispatch(x, torch.zeros(T, K, dtype=torch.int16), x_scales=xs, out=buf)
    assert got is buf and perm is buf and reached == ["moe_permute", "moe_dispatch"]
    with pytest.raises(ValueError, match="out must be"):
        d.permute(x, xs, out=torch.zeros(d.R, H, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="out must be"):
        d.permute(x, xs, out=torch.zeros(d.R, H, dtype=torch.int8))
