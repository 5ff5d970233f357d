"""Products grouped by expert at the sizes where they take other kernels than
the small ones: many rows per expert over many tiles, and weights of hundreds of
megabytes.  Tolerances as in test_gpu_grouped, references in 64 bits on the GPU."""
import pytest
import torch

from gpu_util import DEV, log
from test_gpu_grouped import BF, F32, Case, _backward_reference, _keep_reference, _product, _within

pytestmark = pytest.mark.gpu

# rows of each expert: empty ones, whole and partial tiles of 256, blocks of 32
COUNTS = [[300, 0, 128, 257, 96, 513, 31, 224], [96] * 8, [1000, 0, 0, 3, 0, 0, 1, 64]]


def _check(got, want_tol, what):
    want, tol = want_tol
    _within(got, want.cpu(), tol.cpu(), what)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("N,M", [(8328, 72), (8192, 64), (8200, 264)])
@pytest.mark.parametrize("ci", range(len(COUNTS)))
def test_product(ci, N, M, transpose):
    """More than 256 tiles of 256 x 256; the output is the wide dimension in either direction."""
    log("large grouped product", COUNTS[ci], N, M, transpose)
    if transpose:
        N, M = M, N
    c = Case(COUNTS[ci], pad=(1, 4, 16)[ci], seed=ci + N, extra_empty=0)
    x, w = c.rows(N if transpose else M).to(DEV), c.weight(N, M).to(DEV)
    out = torch.full((c.R, M if transpose else N), 7.0, dtype=BF, device=DEV)
    c.d.grouped_product(x, w, transpose=transpose, out=out)
    torch.cuda.synchronize()
    for e, r in enumerate(c.rows_of):
        r = r.to(DEV)
        we = w[e].double()
        _check(out[r], _product(x[r].double(), we if transpose else we.T), ("product", BF, e))
    assert bool((out[~c.live.to(DEV)] == 7.0).all())


@pytest.mark.parametrize("dtype,accumulate", [(BF, False), (BF, True), (F32, False), (F32, True)])
@pytest.mark.parametrize("N,M", [(2840, 2832), (4096, 2048)])
@pytest.mark.parametrize("ci", range(len(COUNTS)))
def test_weight_grad(ci, N, M, dtype, accumulate):
    """More than 1024 tiles of 256 x 256."""
    log("large grouped weight grad", COUNTS[ci], N, M, dtype, accumulate)
    c = Case(COUNTS[ci], pad=(4, 1, 16)[ci], seed=50 + ci + M, extra_empty=0)
    g, x = c.rows(N).to(DEV), c.rows(M).to(DEV)
    before = (torch.randn(c.E, N, M, device=DEV) * 4).to(dtype)
    out = before.clone()
    c.d.grouped_weight_grad(g, x, out=out, accumulate=accumulate)
    torch.cuda.synchronize()
    for e, r in enumerate(c.rows_of):
        r = r.to(DEV)
        want, tol = _product(g[r].double().T, x[r].double())
        if accumulate:
            want = want + before[e].double()
            tol = tol + 2.0 ** -24 * (want.abs() + tol)
        _check(out[e], (want, tol), ("weight grad", dtype, e))


@pytest.mark.parametrize("F", [8200, 8328])
def test_mlp_both_ways(F):
    H, counts = 72, COUNTS[0]
    log("large mlp", counts, H, F)
    c = Case(counts, H=H, pad=4, seed=F, extra_empty=0)
    x, gy, h = c.rows(H).to(DEV), c.rows(H).to(DEV), c.rows(2 * F).to(DEV)
    w1, w2 = c.weight(2 * F, H).to(DEV), c.weight(H, F).to(DEV)
    y, kept = c.d.grouped_mlp_keep(x, w1, w2)
    gx, g1, g2 = c.d.grouped_mlp_backward(gy, x, h, w1, w2)
    torch.cuda.synchronize()
    for e, rows in enumerate(c.rows_of):
        r = rows.to(DEV)
        c.rows_of[e] = r
        hw, dh, yw, dy = _keep_reference(c, x, w1, w2, F, e)
        _check(kept[r], (hw, dh), ("h", BF, e))
        _check(y[r], (yw, dy), ("y", BF, e))
        for name, got, bound in zip(("grad_perm", "grad_w1", "grad_w2"), (gx[r], g1[e], g2[e]),
                                    _backward_reference(gy[r], x[r], h[r], w1[e], w2[e], F)):
            _check(got, bound, (name, BF, e))


@pytest.mark.parametrize("dtype,accumulate", [(BF, False), (BF, True), (F32, False), (F32, True)])
def test_mlp_of_many_experts_with_few_rows(dtype, accumulate):
    """More than two rounds of tiles of 256 features, too few rows for the wide ones."""
    H, F = 72, 3592
    counts = [(i * 37) % 61 if i % 5 else 0 for i in range(63)] + [300]
    log("mlp of many experts", dtype, accumulate)
    c = Case(counts, H=H, pad=4, seed=17, extra_empty=0)
    x, gy, h = c.rows(H).to(DEV), c.rows(H).to(DEV), c.rows(2 * F).to(DEV)
    w1, w2 = c.weight(2 * F, H).to(DEV), c.weight(H, F).to(DEV)
    y, kept = c.d.grouped_mlp_keep(x, w1, w2)
    before = [torch.randn(w.shape, device=DEV).to(dtype) for w in (w1, w2)]
    grads = [b.clone() for b in before]
    gx, _, _ = c.d.grouped_mlp_backward(gy, x, h, w1, w2, grad_w1=grads[0], grad_w2=grads[1], accumulate=accumulate)
    torch.cuda.synchronize()
    for e, rows in enumerate(c.rows_of):
        r = rows.to(DEV)
        c.rows_of[e] = r
        hw, dh, yw, dy = _keep_reference(c, x, w1, w2, F, e)
        _check(kept[r], (hw, dh), ("h", BF, e))
        _check(y[r], (yw, dy), ("y", BF, e))
        rx, *weights = _backward_reference(gy[r], x[r], h[r], w1[e], w2[e], F)
        _check(gx[r], rx, ("grad_perm", BF, e))
        for got, old, (want, tol) in zip(grads, before, weights):
            if accumulate:
                want = want + old[e].double()
                tol = tol + 2.0 ** -24 * (want.abs() + tol)
            _check(got[e], (want, tol), ("weight", dtype, e))


def _within_on_gpu(got, want_tol):
    """_check's bound without its copies to the host, as a tensor."""
    want, tol = want_tol
    tol = tol + (2.0 ** -8 if got.dtype == BF else 2.0 ** -24) * (want.abs() + tol) + 1e-37
    return ((got.double() - want).abs() <= tol).all()


def test_product_of_more_tiles_than_workgroups():
    """Some 80 thousand tiles: a workgroup takes one after the other, of several experts."""
    counts, N, M = [(i * 37) % 21 for i in range(1023)] + [200], 8, 20488
    log("more product tiles than workgroups")
    c = Case(counts, pad=4, seed=23, extra_empty=0)
    x, w = c.rows(N).to(DEV), torch.empty((c.E, N, M), dtype=BF, device=DEV).normal_(0, N ** -0.5)
    out = torch.full((c.R, M), 7.0, dtype=BF, device=DEV)
    c.d.grouped_product(x, w, transpose=True, out=out)
    ok = [_within_on_gpu(out[r.to(DEV)], _product(x[r.to(DEV)].double(), w[e].double()))
          for e, r in enumerate(c.rows_of)]
    torch.cuda.synchronize()
    assert [e for e, good in enumerate(ok) if not bool(good)] == []
    assert bool((out[~c.live.to(DEV)] == 7.0).all())


@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_grad_of_more_tiles_than_workgroups(accumulate):
    """Some 92 thousand tiles, those of experts without rows between the others."""
    counts, N, M = [(i * 37) % 21 for i in range(1023)] + [200], 2312, 1032
    log("more weight tiles than workgroups", accumulate)
    c = Case(counts, pad=4, seed=29, extra_empty=0)
    g, x = c.rows(N).to(DEV), c.rows(M).to(DEV)
    before = torch.empty((c.E, N, M), dtype=BF, device=DEV).normal_(0, 4)
    out = before.clone()
    c.d.grouped_weight_grad(g, x, out=out, accumulate=accumulate)
    ok = []
    for e, r in enumerate(c.rows_of):
        r = r.to(DEV)
        want, tol = _product(g[r].double().T, x[r].double())
        if accumulate:
            want = want + before[e].double()
            tol = tol + 2.0 ** -24 * (want.abs() + tol)
        ok.append(_within_on_gpu(out[e], (want, tol)))
    torch.cuda.synchronize()
    assert [e for e, good in enumerate(ok) if not bool(good)] == []


@pytest.mark.parametrize("counts", [[1, 0, 5, 2, 0, 1, 3, 300], [320] * 8, [0] * 7 + [2000]])
def test_streamed_weights(counts):
    """Half a gigabyte of weights, rows from one to many: the kernel that streams them."""
    N, M = 8192, 4096
    log("streamed grouped product", counts, N, M)
    c = Case(counts, pad=4, seed=3, extra_empty=0)
    x = c.rows(M).to(DEV)
    w = torch.empty((c.E, N, M), dtype=BF, device=DEV).normal_(0, M ** -0.5)
    out = torch.full((c.R, N), 7.0, dtype=BF, device=DEV)
    c.d.grouped_product(x, w, out=out)
    torch.cuda.synchronize()
    for e, r in enumerate(c.rows_of):
        r = r.to(DEV)
        _check(out[r], _product(x[r].double(), w[e].double().T), ("product", BF, e))
    assert bool((out[~c.live.to(DEV)] == 7.0).all())


def test_rows_of_non_finite_values_and_poisoned_neighbours():
    """An infinity stays in its row (product) and expert (weight gradient) in the large kernels too, and what lies behind
    an expert's rows (NaN here) never reaches a sum."""
    c = Case([300, 257, 97, 130, 96, 96, 110, 100], pad=16, seed=9, extra_empty=0)
    x, w, g = c.rows(2832).to(DEV), c.weight(8328, 2832).to(DEV), c.rows(2840).to(DEV)
    bad = int(c.rows_of[1][200])
    x[bad, 7] = float("inf")
    y = c.d.grouped_product(x, w)
    gw = c.d.grouped_weight_grad(g, x)
    torch.cuda.synchronize()
    ok = c.live.clone()
    ok[bad] = False
    assert bool(y[ok.to(DEV)].isfinite().all()) and not bool(y[bad].isfinite().any())
    for e in range(c.E):
        if e != 1:
            assert bool(gw[e].isfinite().all())
    assert bool(gw[1][:, :7].isfinite().all()) and bool(gw[1][:, 8:].isfinite().all())
    assert not bool(gw[1][:, 7].isfinite().any())


def test_large_calls_repeat_in_graphs_and_on_streams():
    counts, H, F = [300, 0, 128, 257, 96, 513, 31, 224], 520, 8200
    c = Case(counts, H=H, pad=4, seed=13, extra_empty=0)
    x, gy = c.rows(H).to(DEV), c.rows(H).to(DEV)
    w1, w2 = c.weight(2 * F, H).to(DEV), c.weight(H, F).to(DEV)
    new = lambda *s: torch.zeros(s, dtype=BF, device=DEV)
    room = lambda: [new(c.R, 2 * F), new(c.R, H), new(c.R, H), new(*w1.shape), new(*w2.shape),
                    c.d.alloc_mlp_scratch(F), c.d.alloc_mlp_backward_scratch(F)]

    def step(b):
        c.d.grouped_mlp_keep(x, w1, w2, h=b[0], scratch=b[5], out=b[1])
        c.d.grouped_mlp_backward(gy, x, b[0], w1, w2, grad_perm=b[2], grad_w1=b[3], grad_w2=b[4], scratch=b[6])

    want, other, held = room(), room(), room()
    step(want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st, b in zip(streams, (other, held)):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            step(b)
    torch.cuda.synchronize()
    for k in range(5):
        assert torch.equal(other[k], want[k]) and torch.equal(held[k], want[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(held)
    for _ in range(3):
        for k in range(5):
            held[k].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k in range(5):
            assert torch.equal(held[k], want[k]), k
        step(other)
        torch.cuda.synchronize()
