"""Grouped products whose weights are streamed by the expert MLP's FC2 kernel
(large weights, few rows each), as calls of their own with a width that is not
the handle's and inside the MLP's forward.  Tolerances as in test_gpu_grouped,
references in 64 bits on the GPU.

That a case reaches this kernel is read off the rule itself: its expression in
csrc/grouped.hip is evaluated for the case and the card's CUs."""
import os
import re

import pytest
import torch

from combine_routing_preprocess_amd.build import CSRC

GROUPED = os.path.join(CSRC, "grouped.hip")


def _rule(copies, E, N, M, num_cu):
    """stream_weights(...) of csrc/grouped.hip."""
    body = re.search(r"bool stream_weights\([^)]*\) \{(.*?)\n\}", open(GROUPED).read(), re.S).group(1)
    touched, result = re.fullmatch(r"\s*const long long touched = (.*?);\s*return (.*?);", body, re.S).groups()
    assert touched == "copies(h) < h->desc.E ? copies(h) : h->desc.E"
    text = re.sub(r"(\d)ll\b", r"\1", result).replace("copies(h)", "copies").replace("h->desc.E", "E")
    text = " ".join(text.replace("&&", " and ").split()).replace("/", "//")
    return bool(eval(text, {}, dict(copies=copies, E=E, N=N, M=M, num_cu=num_cu, touched=min(copies, E))))


# rows per expert: single ones and empty experts; every count of blocks of 32; segments of 257 to 320 rows, which take
# units of their own; one expert with all rows
FEW = [1, 0, 5, 2, 0, 1, 3, 300, 0, 0, 17, 1, 1, 0, 2, 4]
BLOCKS = [1, 32, 33, 64, 65, 96, 97, 128, 129, 160, 161, 192, 193, 224, 225, 256]
MIDDLE = [320, 257, 288, 289] * 4
ONE = [0] * 7 + [2000] + [0] * 8
SIZES = [(8192, 4096), (8704, 3200)]      # 256 and 272 blocks of 32 columns: 4 and 2 left over of units of 6


def test_rule_covers_the_cases():
    """On 256 CUs, and not for the neighbours that miss one of its conditions."""
    for counts in (FEW, BLOCKS, MIDDLE, ONE):
        for N, M in SIZES + [(8192, 1664)]:
            assert _rule(sum(counts), 16, N, M, 256)
    assert not _rule(340, 8, 8192, 4096, 256)             # too few units for the CUs
    assert not _rule(340, 16, 8192, 1024, 256)            # too few bytes
    assert not _rule(16 * 321, 16, 8192, 4096, 256)       # too many rows
    assert not _rule(340, 16, 8200, 4096, 256) and not _rule(340, 16, 8192, 4104, 256)


def _case(counts, H=64, **kw):
    from test_gpu_grouped import Case
    return Case(counts, H=H, extra_empty=0, **kw)


def _streamed(c, N, M):
    from gpu_util import DEV
    assert _rule(c.d.T * c.d.K, c.E, N, M, torch.cuda.get_device_properties(DEV).multi_processor_count)


def _check(got, want_tol, what):
    from test_gpu_grouped import _within
    want, tol = want_tol
    _within(got, want.cpu(), tol.cpu(), what)


def _weights(E, n, m):
    from gpu_util import DEV
    g = torch.Generator(device=DEV)
    g.manual_seed(n + m)
    return torch.empty((E, n, m), dtype=torch.bfloat16, device=DEV).normal_(0, m ** -0.5, generator=g)


@pytest.mark.gpu
@pytest.mark.parametrize("N,M", SIZES)
@pytest.mark.parametrize("counts", [FEW, BLOCKS, MIDDLE, ONE], ids=["few", "blocks", "middle", "one"])
def test_product(counts, N, M):
    from gpu_util import DEV, log
    from test_gpu_grouped import BF, _product
    log("streamed product", counts, N, M)
    c = _case(counts, pad=4, seed=3)
    _streamed(c, N, M)
    x, w = c.rows(M).to(DEV), _weights(c.E, N, M)
    out = torch.full((c.R, N), 7.0, dtype=BF, device=DEV)
    c.d.grouped_product(x, w, out=out)
    torch.cuda.synchronize()
    for e, r in enumerate(c.rows_of):
        r = r.to(DEV)
        _check(out[r], _product(x[r].double(), w[e].double().T), ("product", BF, e))
    assert bool((out[~c.live.to(DEV)] == 7.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("out_rows", [1, 9, 600, 1100])
def test_product_of_rows_past_the_end(out_rows):
    """The last row that fits lies inside a segment, whole segments begin behind it."""
    from gpu_util import DEV, log
    from test_gpu_grouped import BF, _product
    log("streamed product, rows past the end", out_rows)
    N, M = SIZES[0]
    c = _case(MIDDLE, out_rows=out_rows, seed=out_rows)
    _streamed(c, N, M)
    assert c.R == out_rows == sum(len(r) for r in c.rows_of)
    x, w = c.rows(M).to(DEV), _weights(c.E, N, M)
    out = torch.full((c.R + 512, N), 7.0, dtype=BF, device=DEV)
    c.d.grouped_product(x, w, out=out[:c.R])
    torch.cuda.synchronize()
    for e, r in enumerate(c.rows_of):
        r = r.to(DEV)
        _check(out[r], _product(x[r].double(), w[e].double().T), ("product", BF, e))
    assert bool((out[c.R:] == 7.0).all())


@pytest.mark.gpu
def test_no_rows_at_all():
    """Every token without an expert: nothing is written."""
    from gpu_util import DEV, log
    from test_gpu_grouped import BF, Case
    log("streamed product without rows")
    N, M = SIZES[0]
    c = Case([0] * 16, extra_empty=40, seed=1)
    _streamed(c, N, M)
    out = torch.full((c.R, N), 7.0, dtype=BF, device=DEV)
    c.d.grouped_product(c.rows(M).to(DEV), _weights(c.E, N, M), out=out)
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [FEW, MIDDLE], ids=["few", "middle"])
def test_mlp_forward(counts):
    """grouped_mlp_keep, whose second product is streamed; repeated in a graph bit for bit."""
    from gpu_util import DEV, log
    from test_gpu_grouped import BF, _keep_reference
    H, F = 8192, 1664
    log("mlp with a streamed product", counts)
    c = _case(counts, H=H, pad=4, seed=5)
    _streamed(c, H, F)
    x, w1, w2 = c.rows(H).to(DEV), _weights(c.E, 2 * F, H), _weights(c.E, H, F)
    y = torch.full((c.R, H), 7.0, dtype=BF, device=DEV)
    _, h = c.d.grouped_mlp_keep(x, w1, w2, out=y)
    torch.cuda.synchronize()
    for e, rows in enumerate(c.rows_of):
        r = c.rows_of[e] = rows.to(DEV)
        hw, dh, yw, dy = _keep_reference(c, x, w1, w2, F, e)
        _check(h[r], (hw, dh), ("h", BF, e))
        _check(y[r], (yw, dy), ("y", BF, e))
    assert bool((y[~c.live.to(DEV)] == 7.0).all())
    live, scratch = c.live.to(DEV), c.d.alloc_mlp_scratch(F)
    held, held_h = torch.zeros_like(y), torch.zeros_like(h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.d.grouped_mlp_keep(x, w1, w2, out=held, h=held_h, scratch=scratch)
    for _ in range(3):
        held.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held[live], y[live])
        c.d.grouped_mlp_keep(x, w1, w2)
        torch.cuda.synchronize()


@pytest.mark.gpu
def test_non_finite_rows():
    """An infinity stays in its row, and what lies behind an expert's rows (NaN here) reaches no sum."""
    from gpu_util import DEV, log
    log("streamed product, non-finite rows")
    N, M = SIZES[0]
    c = _case(FEW, pad=16, seed=9)
    _streamed(c, N, M)
    x = c.rows(M).to(DEV)
    bad = int(c.rows_of[7][200])
    x[bad, 7] = float("inf")
    y = c.d.grouped_product(x, _weights(c.E, N, M))
    torch.cuda.synchronize()
    ok = c.live.clone()
    ok[bad] = False
    assert bool(y[ok.to(DEV)].isfinite().all()) and not bool(y[bad].isfinite().any())
