"""layer(rms=...) in all its forms against the same calls one by one, bit for
bit: routing from a router or given, with a residual or without, bf16 payload
and fp8 payload (where the norm writes codes, and rows for a router alone), and
rejected calls that leave the residual as it was."""
import pytest
import torch

from combine_routing_preprocess_amd import Dispatcher, rms_norm
from gpu_util import DEV, log

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
T, H, E, K, F = 96, 256, 8, 2, 128


def _inputs(payload, x_type=BF, res_type=BF, seed=41):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g) * std
    p = dict(x=n(T, H).to(x_type), res=n(T, H).to(res_type), wn=(1 + 0.2 * n(H)).to(BF), wr=n(E, H, std=H ** -0.5),
             probs=torch.rand(T, K, generator=g))
    p["routing"] = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).to(torch.int16)
    if payload == "bf16":
        ws = [n(*s, std=0.05).to(BF) for s in ((E, 2 * F, H), (E, H, F))]
        kw = {}
    else:
        ws = [torch.randint(0, 120, s, generator=g, dtype=torch.uint8) for s in ((E, 2 * F, H), (E, H, F))]
        kw = dict(w1_scales=torch.full((E, 2 * F // 128, H // 128), 1e-3), w2_scales=torch.full((E, H // 128, F // 128), 1e-3))
    return {k: v.to(DEV) for k, v in p.items()}, [w.to(DEV) for w in ws], {k: v.to(DEV) for k, v in kw.items()}


def _parts(payload, p, ws, kw, residual, routed, T_live=None):
    """The layer's output and the new residual stream."""
    fp8 = payload == "fp8"
    n = rms_norm(p["x"], p["wn"], 1e-5, residual=residual, out_dtype=BF, quantize=fp8)
    d = Dispatcher(T, H, E, K, payload=payload, device=DEV)
    routing, probs = (p["routing"], p["probs"]) if not routed else d.gate(n.out.float() @ p["wr"].T, score="sigmoid",
                                                                         normalize=True)
    perm, _, _, _, ps = d.dispatch(n.codes if fp8 else n.out, routing, probs, x_scales=n.scales, T_live=T_live)
    return d.combine(d.grouped_mlp(perm, *ws, perm_scales=ps, **kw)), n.total


def _call(d, p, ws, kw, residual, routed, **more):
    if routed:
        more = dict(router=lambda rows: rows.float() @ p["wr"].T, gate=dict(score="sigmoid", normalize=True), **more)
    return d.layer(p["x"], None if routed else p["routing"], None if routed else p["probs"], *ws, rms=(p["wn"], 1e-5),
                   residual=residual, **kw, **more)


@pytest.mark.parametrize("x_type,res_type", [(BF, BF), (torch.float32, torch.float32), (BF, torch.float32)])
@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("routed", [False, True])
@pytest.mark.parametrize("payload", ["bf16", "fp8"])
def test_layer_is_its_parts(payload, routed, with_residual, x_type, res_type):
    log("layer with rms", payload, routed, with_residual, x_type, res_type)
    p, ws, kw = _inputs(payload, x_type, res_type)
    residual = p["res"] if with_residual else None
    want, total = _parts(payload, p, ws, kw, residual, routed)
    stream = None if residual is None else residual.clone()
    before = p["x"].clone()
    got = _call(Dispatcher(T, H, E, K, payload=payload, device=DEV), p, ws, kw, stream, routed)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and bool(got.isfinite().all()) and float(got.abs().max()) > 0
    assert torch.equal(p["x"], before)
    assert stream is None or torch.equal(stream, total)


@pytest.mark.parametrize("codes", [torch.uint8, torch.float8_e4m3fn])
@pytest.mark.parametrize("with_residual", [False, True])
def test_caller_owned_buffers(codes, with_residual):
    """fp8 payload with every buffer the caller's, perm of either code type, and tokens from T_live on without copies."""
    log("layer with rms, own buffers", codes, with_residual)
    p, ws, kw = _inputs("fp8", seed=7)
    live = torch.tensor([70], dtype=torch.int32, device=DEV)
    residual = p["res"] if with_residual else None
    want, total = _parts("fp8", p, ws, kw, residual, False, live)
    d = Dispatcher(T, H, E, K, payload="fp8", device=DEV)
    bufs = dict(perm=torch.zeros((d.R, H), dtype=codes, device=DEV),
                perm_scales=torch.zeros((d.R, H // 128), device=DEV), scratch=d.alloc_mlp_scratch(F, "fp8"),
                expert_out=torch.zeros((d.R, H), dtype=BF, device=DEV), out=torch.zeros((T, H), dtype=BF, device=DEV))
    stream = None if residual is None else residual.clone()
    got = _call(d, p, ws, kw, stream, False, T_live=live, **bufs)
    torch.cuda.synchronize()
    assert got is bufs["out"] and torch.equal(got, want)
    assert stream is None or torch.equal(stream, total)          # every row, those from T_live on too


@pytest.mark.parametrize("payload", ["bf16", "fp8"])
def test_a_rejected_call_leaves_the_residual(payload):
    p, ws, kw = _inputs(payload)
    want, total = _parts(payload, p, ws, kw, p["res"], False)
    d = Dispatcher(T, H, E, K, payload=payload, device=DEV)
    stream = p["res"].clone()
    for bad in (dict(out=torch.zeros((T, H), device=DEV)), dict(scratch=torch.zeros(8, dtype=torch.uint8, device=DEV)),
                dict(perm=torch.zeros((d.R, H), device=DEV)), dict(expert_out=torch.zeros((3, H), dtype=BF, device=DEV)),
                dict(T_live=torch.zeros(1, device=DEV))):
        with pytest.raises(ValueError):
            _call(d, p, ws, kw, stream, False, **bad)
    with pytest.raises(ValueError, match="routing dtype"):
        _call(d, dict(p, routing=p["routing"].int()), ws, kw, stream, False)
    torch.cuda.synchronize()
    assert torch.equal(stream, p["res"])
    got = _call(d, p, ws, kw, stream, False)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(stream, total)
    # what the router raises comes after the norm: the sum is there, as documented
    def raises(rows):
        raise RuntimeError("no logits")
    again = p["res"].clone()
    with pytest.raises(RuntimeError, match="no logits"):
        d.layer(p["x"], None, None, *ws, rms=(p["wn"], 1e-5), residual=again, router=raises, **kw)
    torch.cuda.synchronize()
    assert torch.equal(again, total)


def test_layer_in_a_graph():
    """The residual adds up over replays as over calls."""
    p, ws, kw = _inputs("fp8", seed=9)
    d = Dispatcher(T, H, E, K, payload="fp8", device=DEV)
    bufs = dict(perm=torch.zeros((d.R, H), dtype=torch.uint8, device=DEV),
                perm_scales=torch.zeros((d.R, H // 128), device=DEV), scratch=d.alloc_mlp_scratch(F, "fp8"),
                expert_out=torch.zeros((d.R, H), dtype=BF, device=DEV), out=torch.zeros((T, H), dtype=BF, device=DEV))
    eager, held = p["res"].clone(), p["res"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        _call(d, p, ws, kw, held, False, **bufs)
    other = Dispatcher(T, H, E, K, payload="fp8", device=DEV)
    for _ in range(3):
        want = _call(other, p, ws, kw, eager, False)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs["out"], want) and torch.equal(held, eager)
