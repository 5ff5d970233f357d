"""layer(rms=, residual=) writes the sum over the residual, so whatever the steps
behind the norm refuse is refused before it runs: a rejected call leaves the
residual as it was, and the corrected one adds x once.  No GPU: the norm is
replaced by a mark that it was reached."""
import pytest
import torch

from combine_routing_preprocess_amd import Dispatcher, MoeError
from combine_routing_preprocess_amd import api

T, H, E, K, F = 8, 256, 4, 2, 128
BF = torch.bfloat16


class _Reached(Exception):
    pass


@pytest.fixture(autouse=True)
def norm_marks(monkeypatch):
    def norm(*args, **kw):
        raise _Reached
    monkeypatch.setattr(api, "rms_norm", norm)


def _args(payload):
    d = Dispatcher(T, H, E, K, payload=payload, device="cpu")
    a = dict(x=torch.zeros(T, H, dtype=BF), routing=torch.zeros(T, K, dtype=torch.int16), probs=torch.zeros(T, K),
             residual=torch.zeros(T, H, dtype=BF), rms=(torch.zeros(H),))
    if payload == "bf16":
        a.update(w1=torch.zeros(E, 2 * F, H, dtype=BF), w2=torch.zeros(E, H, F, dtype=BF))
    else:
        a.update(w1=torch.zeros(E, 2 * F, H, dtype=torch.uint8), w2=torch.zeros(E, H, F, dtype=torch.uint8),
                 w1_scales=torch.zeros(E, 2 * F // 128, H // 128), w2_scales=torch.zeros(E, H // 128, F // 128))
    return d, a


def _off_by(t, n):
    """t's values n bytes further on than an aligned address."""
    room = torch.zeros(t.numel() * t.element_size() + 64, dtype=torch.uint8)
    start = -room.data_ptr() % 16 + n
    return room[start:start + t.numel() * t.element_size()].view(t.dtype).view(t.shape)


def _rows(d, dtype=BF, width=H):
    return torch.zeros(d.R, width, dtype=dtype)


# name -> change of the arguments; a payload in front where it is not for both
BAD = {
    "x of other tokens": lambda d, a: a.update(x=torch.zeros(T + 1, H, dtype=BF),
                                               residual=torch.zeros(T + 1, H, dtype=BF)),
    "routing type": lambda d, a: a.update(routing=a["routing"].int()),
    "routing shape": lambda d, a: a.update(routing=a["routing"][:, :1].contiguous()),
    "routing at an odd address": lambda d, a: a.update(routing=_off_by(a["routing"], 2)),
    "no routing": lambda d, a: a.update(routing=None),
    "probs type": lambda d, a: a.update(probs=a["probs"].double()),
    "T_live type": lambda d, a: a.update(T_live=torch.zeros(1)),
    "w1 shape": lambda d, a: a.update(w1=a["w1"][:3].contiguous()),
    "w1 strides": lambda d, a: a.update(w1=a["w1"].transpose(1, 2).contiguous().transpose(1, 2)),
    "w1 at an odd address": lambda d, a: a.update(w1=_off_by(a["w1"], 8)),
    "w2 width": lambda d, a: a.update(w2=torch.zeros(E, H, 2 * F, dtype=a["w2"].dtype),
                                      **({"w2_scales": torch.zeros(E, H // 128, 2 * F // 128)}
                                         if "w2_scales" in a else {})),
    "w2 at an odd address": lambda d, a: a.update(w2=_off_by(a["w2"], 4)),
    "scratch size": lambda d, a: a.update(scratch=torch.zeros(64, dtype=torch.uint8)),
    "scratch at an odd address": lambda d, a: a.update(scratch=_off_by(torch.zeros(1 << 20, dtype=torch.uint8), 8)),
    "perm shape": lambda d, a: a.update(perm=torch.zeros(3, H, dtype=BF if d.payload == 0 else torch.uint8)),
    "perm type": lambda d, a: a.update(perm=_rows(d, torch.float32)),
    "perm at an odd address": lambda d, a: a.update(perm=_off_by(_rows(d, BF if d.payload == 0 else torch.uint8), 8)),
    "expert_out type": lambda d, a: a.update(expert_out=_rows(d, torch.float32)),
    "expert_out at an odd address": lambda d, a: a.update(expert_out=_off_by(_rows(d), 4)),
    "out shape": lambda d, a: a.update(out=torch.zeros(T - 1, H, dtype=BF)),
    "out type": lambda d, a: a.update(out=torch.zeros(T, H)),
    "out at an odd address": lambda d, a: a.update(out=_off_by(torch.zeros(T, H, dtype=BF), 2)),
    "bf16 with perm_scales": lambda d, a: a.update(perm_scales=_rows(d, torch.float32, H // 128)),
    "bf16 with block scales": lambda d, a: a.update(w1_scales=torch.zeros(E, 2 * F // 128, H // 128)),
    "bf16 with F of no 128": lambda d, a: a.update(w1=torch.zeros(E, 2 * 64, H, dtype=BF),
                                                   w2=torch.zeros(E, H, 64, dtype=BF)),
    "fp8 with perm_scales type": lambda d, a: a.update(perm_scales=_rows(d, torch.float64, H // 128)),
    "fp8 without block scales": lambda d, a: a.update(w2_scales=None),
    "fp8 with bf16 weights": lambda d, a: a.update(w1=torch.zeros(E, 2 * F, H, dtype=BF), w1_scales=None,
                                                   w2=torch.zeros(E, H, F, dtype=BF), w2_scales=None),
}


@pytest.mark.parametrize("name,payload", [(n, p) for n in BAD for p in ("bf16", "fp8")
                                          if n.split()[0] not in {"bf16", "fp8"} - {p}])
def test_refused_before_the_norm(name, payload):
    d, a = _args(payload)
    BAD[name](d, a)
    with pytest.raises((ValueError, MoeError)):
        d.layer(**a)


def test_bf16_weights_of_an_odd_width_refused_before_the_norm():
    d, h = Dispatcher(T, 128, E, K, device="cpu"), 128
    with pytest.raises(ValueError, match="H % 256"):
        d.layer(torch.zeros(T, h, dtype=BF), torch.zeros(T, K, dtype=torch.int16), None,
                torch.zeros(E, 2 * F, h, dtype=BF), torch.zeros(E, h, F, dtype=BF), rms=(None,),
                residual=torch.zeros(T, h, dtype=BF))


_SHARED = torch.zeros(4 * T * K, dtype=torch.uint8)
GATE = {
    "gate score": dict(score="tanh"),
    "gate option": dict(temperature=2.0),
    "gate scale": dict(scale=float("inf")),
    "gate scale in fp32": dict(scale=1e39),
    "gate bias": dict(bias=torch.zeros(E + 1)),
    "gate routing over probs": dict(routing=_SHARED[:2 * T * K].view(torch.int16).view(T, K),
                                    probs=_SHARED.view(torch.float32).view(T, K)),
    "gate routing": dict(routing=torch.zeros(T, K, dtype=torch.int32)),
    "gate routing at an odd address": dict(routing=_off_by(torch.zeros(T, K, dtype=torch.int16), 2)),
    "gate probs": dict(probs=torch.zeros(T, K + 1)),
}


@pytest.mark.parametrize("name", list(GATE))
def test_gate_options_refused_before_the_norm(name):
    d, a = _args("bf16")
    a.update(routing=None, probs=None, router=lambda rows: rows, gate=GATE[name])
    with pytest.raises((ValueError, TypeError)):
        d.layer(**a)


def test_router_refusals_before_the_norm():
    d, a = _args("bf16")
    a.update(routing=None, probs=None, router=lambda rows: rows, T_live=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="T_live"):
        d.layer(**a)


@pytest.mark.parametrize("payload", ["bf16", "fp8"])
def test_accepted_calls_reach_the_norm(payload):
    d, a = _args(payload)
    codes = BF if payload == "bf16" else torch.uint8
    bufs = dict(perm=_rows(d, codes), scratch=d.alloc_mlp_scratch(F, payload), expert_out=_rows(d),
                out=torch.zeros(T, H, dtype=BF), T_live=torch.zeros(1, dtype=torch.int32))
    if payload == "fp8":
        bufs["perm_scales"] = _rows(d, torch.float32, H // 128)
    routed = dict(a, routing=None, probs=None, router=lambda rows: rows,
                  gate=dict(score="sigmoid", normalize=True, scale=2.5, bias=torch.zeros(E)))
    for call in (a, dict(a, **bufs), dict(a, probs=None), routed, dict(routed, gate=None), dict(routed, **bufs)):
        with pytest.raises(_Reached):
            d.layer(**call)
