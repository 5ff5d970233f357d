"""Every call that takes a scratch tells the library its size in bytes,
whatever the tensor's element type: a bf16 scratch of exactly the needed size
is as good as a byte one."""
import pytest
import torch

from combine_routing_preprocess_amd import Dispatcher
from combine_routing_preprocess_amd import _abi as A
from combine_routing_preprocess_amd import api

E, H, F = 4, 256, 128


class _Recorder:
    """Stands in for the loaded library's entry points: sizes are the real
    ones, calls are noted instead of made."""

    def __init__(self, real):
        self.real, self.calls = real, {}

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.real, name)

        def call(*args):
            self.calls[name] = args
            return A.MOE_OK
        return call


@pytest.mark.parametrize("kind", [torch.uint8, torch.bfloat16, torch.float32])
def test_scratch_size_is_told_in_bytes(monkeypatch, kind):
    d = Dispatcher(64, H, E, 2, device="cpu")
    d.h.state = 1
    rec = _Recorder(A.lib())
    monkeypatch.setattr(A, "lib", lambda: rec)
    monkeypatch.setattr(api, "_stream", lambda: 0)

    def room(n):
        item = torch.empty(0, dtype=kind).element_size()
        return torch.zeros((n + item - 1) // item, dtype=kind)

    bf = torch.bfloat16
    w1, w2 = torch.zeros((E, 2 * F, H), dtype=bf), torch.zeros((E, H, F), dtype=bf)
    perm, out = torch.zeros((d.R, H), dtype=bf), torch.zeros((d.R, H), dtype=bf)
    need = d.mlp_scratch_bytes(F)
    scratch = room(need)
    d.grouped_mlp(perm, w1, w2, scratch=scratch, out=out)
    d.fc1(perm, w1, scratch)
    d.fc2(w2, scratch, out)
    d.fc2_fp8out(w2, scratch)
    for name in ("moe_grouped_swiglu_mlp", "moe_grouped_fc1_swiglu", "moe_grouped_fc2", "moe_grouped_fc2_fp8out"):
        args = rec.calls[name]
        assert args[args.index(scratch.data_ptr()) + 1] == need, name
    q1, s1 = torch.zeros((E, 2 * F, H), dtype=torch.uint8), torch.ones((E, 2 * F // 128, H // 128))
    q2, s2 = torch.zeros((E, H, F), dtype=torch.uint8), torch.ones((E, H // 128, F // 128))
    x, y = torch.zeros((64, H), dtype=bf), torch.zeros((64, H), dtype=bf)
    for need, name, more in ((d.decode_layer_scratch_bytes(F), "decode_layer_fp8",
                              dict(status=torch.zeros(1, dtype=torch.int32))),
                             (d.decode_fused_scratch_bytes(F), "decode_fused_fp8", {})):
        scratch = room(need)
        getattr(d, name)(x, q1, q2, s1, s2, scratch=scratch, expert_out=out, out=y, **more)
        args = rec.calls["moe_" + name]
        assert args[args.index(scratch.data_ptr()) + 1] == need, name
