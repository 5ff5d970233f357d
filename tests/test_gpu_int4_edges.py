"""4-bit expert weights: placements of the scales, live counts, experts that are
mostly empty, empty batches.  Oracle and tolerances are those of
test_gpu_int4; calls that differ in placement alone have to agree bit for
bit."""
import pytest
import torch

from combine_routing_preprocess_amd import Dispatcher
from gpu_util import DEV, log
from test_gpu_int4 import BF, _check, _route, _weights

pytestmark = pytest.mark.gpu


def _shifted(t, floats):
    """The same values at `floats` floats behind a 256-byte boundary."""
    room = torch.empty(t.numel() + 64, dtype=t.dtype, device=DEV)
    assert room.data_ptr() % 256 == 0
    at = room[floats:floats + t.numel()].view(t.shape)
    at.copy_(t)
    return at


@pytest.mark.parametrize("floats", [1, 2, 3])
@pytest.mark.parametrize("T,E,K,H,F", [(2, 16, 4, 1024, 512),        # two sets of wavefronts
                                       (40, 40, 3, 512, 1024),       # many units of few rows
                                       (170, 32, 8, 2048, 1024)])    # wide passes
def test_scales_off_a_16_byte_line(T, E, K, H, F, floats):
    log("int4 scales shifted", T, E, K, H, F, floats)
    d = Dispatcher(T, H, E, K, route_fmt="dense_i32", device=DEV)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(T)).to(BF)
    perm, *_ = d.dispatch(x.to(DEV), _route(T, E, K, 1).to(DEV))
    w = _weights(E, 2 * F, H, 2) + _weights(E, H, F, 3)
    c1, s1, c2, s2 = (t.to(DEV) for t in w)
    out = torch.full((d.R, H), 7.0, dtype=BF, device=DEV)
    d.grouped_mlp(perm, c1, c2, w1_scales=_shifted(s1, floats), w2_scales=_shifted(s2, floats), out=out)
    torch.cuda.synchronize()
    _check(d, perm, w, out, 7.0)
    same = torch.full((d.R, H), 7.0, dtype=BF, device=DEV)
    d.grouped_mlp(perm, c1, c2, w1_scales=s1, w2_scales=s2, out=same)
    torch.cuda.synchronize()
    assert torch.equal(same, out)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_empty_batch_through_the_layer(score):
    """No tokens: the MLP alone and the whole layer with norm and gate return
    empty outputs."""
    E, K, H, F = 4, 2, 256, 128
    d = Dispatcher(0, H, E, K, route_fmt="dense_i32", device=DEV)
    assert d.R == 0
    c1, s1, c2, s2 = (t.to(DEV) for t in _weights(E, 2 * F, H, 2) + _weights(E, H, F, 3))
    x, wr = torch.empty((0, H), dtype=BF, device=DEV), torch.zeros((E, H), device=DEV)
    kw = dict(w1_scales=s1, w2_scales=s2, norm=(torch.ones(H, device=DEV), None),
              router=lambda rows: rows.float() @ wr.T, gate=dict(score=score))
    perm, *_ = d.dispatch(x, torch.empty((0, K), dtype=torch.int32, device=DEV))
    assert tuple(d.grouped_mlp(perm, c1, c2, w1_scales=s1, w2_scales=s2).shape) == (0, H)
    assert tuple(d.layer(x, None, None, c1, c2, **kw).shape) == (0, H)
    torch.cuda.synchronize()
    assert d.tokens_per_expert.cpu().tolist() == [0] * E


@pytest.mark.parametrize("fmt", ["dense_i32", "sparse_bool"])
@pytest.mark.parametrize("live", [0, 1, 4, 16, 64])
def test_live_counts(live, fmt):
    """Tokens past T_live take no part: the live ones' rows are the oracle's,
    all others stay as they were."""
    T, E, K, H, F = 64, 32, 4, 512, 256
    log("int4 live", live, fmt)
    idx = _route(T, E, K, 23)
    routing = idx.to(DEV)
    if fmt == "sparse_bool":
        routing = torch.zeros(T, E, dtype=torch.uint8).scatter_(1, idx.long(), 1).to(DEV)
    w = _weights(E, 2 * F, H, 24) + _weights(E, H, F, 25)
    c1, s1, c2, s2 = (t.to(DEV) for t in w)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(26)).to(BF).to(DEV)
    d = Dispatcher(T, H, E, K, route_fmt=fmt, pad_multiple=2, device=DEV)
    count = torch.tensor([live], dtype=torch.int32, device=DEV)
    perm, *_ = d.dispatch(x, routing, T_live=count, out=torch.zeros((d.R, H), dtype=BF, device=DEV))
    out = torch.full((d.R, H), 7.0, dtype=BF, device=DEV)
    d.grouped_mlp(perm, c1, c2, w1_scales=s1, w2_scales=s2, out=out)
    torch.cuda.synchronize()
    assert int(d.kept.sum()) == live * K
    if live:
        _check(d, perm, w, out, 7.0)
    else:
        assert bool((out == 7.0).all())


@pytest.mark.parametrize("E,H,F", [(300, 128, 128), (1000, 128, 128), (1024, 256, 128)])
@pytest.mark.parametrize("T,K", [(1, 1), (3, 4), (9, 2), (70, 3)])
def test_many_experts_mostly_empty(T, K, E, H, F):
    """Experts beyond the first 256 and gaps of any length between those with
    rows: first, last and random ones."""
    log("int4 mostly empty", T, K, E, H, F)
    idx = _route(T, E, K, 27 + T + E)
    idx[0, 0] = E - 1 if not bool((idx[0] == E - 1).any()) else idx[0, 0]
    if T > 1:
        idx[1, 0] = 0 if not bool((idx[1] == 0).any()) else idx[1, 0]
    w = _weights(E, 2 * F, H, 28) + _weights(E, H, F, 29)
    c1, s1, c2, s2 = (t.to(DEV) for t in w)
    d = Dispatcher(T, H, E, K, route_fmt="dense_i32", device=DEV)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(30)).to(BF)
    perm, *_ = d.dispatch(x.to(DEV), idx.to(DEV))
    out = torch.full((d.R, H), 7.0, dtype=BF, device=DEV)
    d.grouped_mlp(perm, c1, c2, w1_scales=s1, w2_scales=s2, out=out)
    torch.cuda.synchronize()
    assert int(d.kept.sum()) == T * K
    _check(d, perm, w, out, 7.0)
