"""With 4-bit weights, a Dispatcher whose workspace lives on another GPU than
the current one is refused before anything is launched: the kernels run on
the current GPU and read the workspace."""
import pytest
import torch

from combine_routing_preprocess_amd import Dispatcher

E, H, F = 4, 256, 128


class _On(torch.Tensor):
    """Host memory that says it lives on GPU `at`."""
    at = 0

    def get_device(self):
        return self.at


def _on(at, t):
    t = t.as_subclass(_On)
    t.at = at
    return t


@pytest.mark.parametrize("name", ["grouped_mlp", "grouped_mlp_noalloc", "fc1", "fc2"])
@pytest.mark.parametrize("workspace,current", [(0, 1), (1, 0)])
def test_int4_needs_the_workspace_on_the_current_gpu(monkeypatch, name, workspace, current):
    d = Dispatcher(8, H, E, 2, device="cpu")
    d.h.state = 1
    d.device, d._cuda, d.ws = torch.device("cuda", workspace), True, _on(workspace, d.ws)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current, raising=False)

    def no_stream():
        raise AssertionError("the call reached its launch")

    monkeypatch.setattr("combine_routing_preprocess_amd.api._stream", no_stream)
    # tensors on the current GPU and on the Dispatcher's own: the binding takes either
    rows = _on(current, torch.zeros((d.R, H), dtype=torch.bfloat16))
    w1, s1 = _on(current, torch.zeros((E, 2 * F, H // 2), dtype=torch.uint8)), _on(workspace, torch.ones(E, 2 * F, 2))
    w2, s2 = _on(workspace, torch.zeros((E, H, F // 2), dtype=torch.uint8)), _on(current, torch.ones(E, H, 1))
    scratch = _on(current, torch.zeros(d.mlp_scratch_bytes(F, "int4"), dtype=torch.uint8))
    d._fc1_done = (F, "int4", scratch.data_ptr())
    calls = dict(grouped_mlp=lambda: d.grouped_mlp(rows, w1, w2, w1_scales=s1, w2_scales=s2, scratch=scratch, out=rows),
                 grouped_mlp_noalloc=lambda: d.grouped_mlp_noalloc(rows, w1, w2, w1_scales=s1, w2_scales=s2, out=rows),
                 fc1=lambda: d.fc1(rows, w1, scratch, w1_scales=s1),
                 fc2=lambda: d.fc2(w2, scratch, rows, w2_scales=s2))
    with pytest.raises(ValueError, match="current GPU"):
        calls[name]()
