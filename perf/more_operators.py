"""Cases of the expert products and the norm of a training or serving step: products grouped by
expert over the dispatched rows in both directions, the weights' gradients, the SwiGLU MLP that keeps
its pre-activations and its backward pass, and the RMS norm with the residual's addition and 8-bit rows.

``run`` computes a case in elementary torch operations where ``own`` is false and with the
framework's calls where it is true; ``exact`` gives the same outputs from the definitions in 64
bits.  The sizes are those of the repository's workloads (8192 tokens x 7168, 256 experts top-8,
FFN 2048, decode batches, 32 experts as one of eight devices holds them) and odd ones.
"""
import torch

own = False

DEV = "cuda"
GROUP = 128          # columns that share a scale of the 8-bit rows
E4M3_MAX = 448.0
_T = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


# ---- the cases --------------------------------------------------------------------------------
def _routed(op, T, E, K, pad, empty, skew, **more):
    """T tokens over E experts, K each; segments padded to ``pad`` rows, ``empty`` unused slots."""
    return dict(op=op, T=T, E=E, K=K, pad=pad, empty=empty, skew=skew, **more)


def _rms(T, H, x, res, y, w, grad_total=False, backward=False):
    """y: "bf16" or "f32" rows, "fp8" codes with scales, "both" bf16 rows and codes."""
    return dict(op="rms_backward" if backward else "rms", T=T, H=H, x=x, res=res, y=y, w=w, grad_total=grad_total)


def listed():
    return [
        # a decode batch through one projection of its experts: the weights are streamed for a row or two
        dict(_routed("product", 16, 256, 8, 1, 0, 0.0, N=4096, M=7168), name="product_decode"),
        # the training / prefill batch: FC1's pre-activations of the flagship layer
        dict(_routed("product", 8192, 256, 8, 16, 0, 0.0, N=4096, M=7168), name="product_batch"),
        # gradient to the rows, sizes of no round number, uneven and empty experts
        dict(_routed("product_t", 3001, 60, 4, 1, 200, 0.7, N=2056, M=1416), name="product_input_grad_odd"),
        # gradient of the flagship layer's second weight: a short sum for each of many elements
        dict(_routed("weight_grad", 8192, 256, 8, 16, 0, 0.0, N=7168, M=2048, out="bf16", add=False),
             name="weight_grad_batch"),
        # gradients added up in fp32 over micro-batches, odd sizes, uneven experts
        dict(_routed("weight_grad", 1501, 24, 4, 1, 60, 0.7, N=1048, M=904, out="f32", add=True),
             name="weight_grad_odd"),
        # the experts that one of eight devices holds, a training batch: forward with what backward needs
        dict(_routed("mlp_keep", 4096, 32, 8, 16, 0, 0.3, H=7168, F=2048), name="mlp_keep_batch"),
        # its backward pass: gradients of the rows and of both weights
        dict(_routed("mlp_backward", 4096, 32, 8, 16, 0, 0.3, H=7168, F=2048), name="mlp_backward_batch"),
        # a small layer of odd sizes
        dict(_routed("mlp_backward", 701, 12, 3, 4, 40, 0.7, H=1160, F=712), name="mlp_backward_odd"),
        # one decoded token: rows for the router and codes for an fp8 dispatch in one call, latency
        dict(_rms(1, 7168, "bf16", "bf16", "both", "bf16"), name="rms_token"),
        # the flagship batch into 8-bit rows
        dict(_rms(8192, 7168, "bf16", "bf16", "fp8", "f32"), name="rms_batch"),
        # its backward pass, with the gradient that arrives along the residual stream
        dict(_rms(8192, 7168, "bf16", "bf16", "bf16", "f32", True, True), name="rms_backward_batch"),
        # an fp32 residual stream, widths and batches of no round size
        dict(_rms(3001, 1537, "f32", "f32", "bf16", "bf16", True, True), name="rms_backward_odd"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["product", "product_t", "weight_grad", "mlp_keep", "mlp_backward", "rms", "rms_backward"])
    if op.startswith("rms"):
        T, H = _spread(rng, 1, 8192), _spread(rng, 64, 7168)
        x = rng.choice(["bf16", "f32"])
        y = rng.choice(["bf16", "f32"] if op == "rms_backward" else ["bf16", "f32", "fp8", "both"])
        if y in ("fp8", "both"):
            H = max(1, H // GROUP) * GROUP
        res = rng.choice(["", "bf16", "f32"]) if op == "rms" else rng.choice(["bf16", "f32"])
        return _rms(T, H, x, res, y, rng.choice(["bf16", "f32"]), op == "rms_backward" and rng.choice([True, False]),
                    op == "rms_backward")
    T, E = _spread(rng, 1, 4096), _spread(rng, 4, 64)
    K = rng.randint(1, min(E, 8))
    empty = rng.choice([0, rng.randint(0, 100)])
    wide, narrow = 8 * _spread(rng, 8, 512), 8 * _spread(rng, 8, 256)
    more = dict(H=wide, F=narrow) if op.startswith("mlp") else dict(N=narrow, M=wide) if rng.random() < 0.5 else \
        dict(N=wide, M=narrow)
    if op == "weight_grad":
        more.update(out=rng.choice(["bf16", "f32"]), add=rng.choice([True, False]))
    return _routed(op, T, E, K, rng.choice([1, 4, 16]), empty, rng.choice([0.0, 0.5]), **more)


# ---- inputs -----------------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, std=1.0, mean=0.0, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(mean, std, generator=g)


def _prepare_routed(case, g):
    T, E, K, pad = case["T"], case["E"], case["K"], case["pad"]
    # experts of uneven popularity: the K largest of noise plus the expert's own offset
    noise = -torch.log(-torch.log(torch.rand((T, E), generator=g, device=DEV).clamp(1e-6, 1 - 1e-6)))
    idx = (noise + case["skew"] * torch.randn(E, generator=g, device=DEV)).topk(K, dim=1).indices.contiguous()
    if case["empty"]:
        flat = idx.view(-1)
        flat[torch.randperm(T * K, generator=g, device=DEV)[:min(case["empty"], T * K // 2)]] = -1
    # the dispatched rows: expert after expert, tokens in order, segments padded
    flat = idx.view(-1)
    kept = int((flat >= 0).sum())
    expert = torch.where(flat < 0, E, flat).sort(stable=True).values[:kept]
    counts = torch.bincount(expert, minlength=E)
    padded = (counts + pad - 1) // pad * pad
    place = torch.arange(kept, device=DEV) - (counts.cumsum(0) - counts)[expert]
    s = dict(expert=expert, place=place, row=(padded.cumsum(0) - padded)[expert] + place, most=int(counts.max()))
    R, op = T * K + E * (pad - 1), case["op"]

    def rows(width):
        return _normal(g, (R, width), dtype=torch.bfloat16)

    def weights(n, m):
        return _normal(g, (E, n, m), 1.0 / m ** 0.5, dtype=torch.bfloat16)

    def room(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16, device=DEV)

    if op in ("product", "product_t"):
        N, M = case["N"], case["M"]
        s.update(rows=rows(M if op == "product" else N), w=weights(N, M), out=room(R, N if op == "product" else M))
    elif op == "weight_grad":
        N, M = case["N"], case["M"]
        s.update(grad=rows(N), rows=rows(M), add=case["add"])
        s["out"] = torch.zeros((E, N, M), dtype=_T[case["out"]], device=DEV)
        if case["add"]:   # what earlier micro-batches left
            s["out"].normal_(0.0, 3.0, generator=g)
    else:
        H, F = case["H"], case["F"]
        s.update(rows=rows(H), w1=weights(2 * F, H), w2=weights(H, F), F=F)
        if op == "mlp_keep":
            s.update(out=room(R, H), h=room(R, 2 * F))
        else:
            s.update(grad=rows(H), h=rows(2 * F), out=room(R, H), g1=torch.empty_like(s["w1"]),
                     g2=torch.empty_like(s["w2"]))
    if own:
        from combine_routing_preprocess_amd import Dispatcher
        d = s["dispatcher"] = Dispatcher(T, s["rows"].shape[1], E, K, route_fmt="dense_i32", pad_multiple=pad, device=DEV)
        d.preprocess(idx.to(torch.int32))
        if op == "mlp_keep":
            s["scratch"] = d.alloc_mlp_scratch(case["F"])
        elif op == "mlp_backward":
            s["scratch"] = d.alloc_mlp_backward_scratch(case["F"])
    return s


def _prepare_rms(case, g):
    T, H, xt, wt = case["T"], case["H"], _T[case["x"]], _T[case["w"]]
    s = dict(weight=_normal(g, (H,), 0.2, 1.0, wt), eps=1e-6)
    # rows of a residual stream: each of its own size
    size = torch.exp(0.5 * torch.randn((T, 1), generator=g, device=DEV))
    if case["op"] == "rms":
        s["x"] = (torch.randn((T, H), generator=g, device=DEV) * 0.5 * size).to(xt)
        s["residual"] = (torch.randn((T, H), generator=g, device=DEV) * size).to(_T[case["res"]]) if case["res"] else None
        quantize, rows = case["y"] in ("fp8", "both"), case["y"] != "fp8"
        s.update(quantize=quantize, y_type=_T.get(case["y"], torch.bfloat16) if rows else None)
        s["out"] = dict(rstd=torch.empty(T, device=DEV))
        if rows:
            s["out"]["out"] = torch.empty((T, H), dtype=s["y_type"], device=DEV)
        if quantize:
            s["out"]["codes"] = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=DEV)
            s["out"]["scales"] = torch.empty((T, H // GROUP), device=DEV)
        if case["res"]:
            s["out"]["total"] = torch.empty((T, H), dtype=_T[case["res"]], device=DEV)
    else:
        tt = _T[case["res"]]
        s["total"] = (torch.randn((T, H), generator=g, device=DEV) * size).to(tt)
        s["rstd"] = (s["total"].double().square().mean(1) + s["eps"]).rsqrt().float()
        s["grad"] = _normal(g, (T, H), dtype=_T[case["y"]])
        s["grad_total"] = _normal(g, (T, H), 0.5, dtype=tt) if case["grad_total"] else None
        s["out"] = dict(out=torch.empty((T, H), dtype=tt, device=DEV), grad_weight=torch.empty(H, device=DEV))
        if own:
            from combine_routing_preprocess_amd import rms_norm_backward_scratch_bytes
            s["out"]["scratch"] = torch.empty(rms_norm_backward_scratch_bytes(T, H), dtype=torch.uint8, device=DEV)
    return s


def prepare(case, seed):
    g = _generator(seed)
    s = _prepare_rms(case, g) if case["op"].startswith("rms") else _prepare_routed(case, g)
    s["op"] = case["op"]
    return s


# ---- the plain forms --------------------------------------------------------------------------
def _by_expert(s):
    """The touched experts, and for each row which of them it belongs to."""
    return torch.unique_consecutive(s["expert"], return_inverse=True)


def _padded(s, t, which, touched):
    """fp32 [touched experts, most rows, width] of the kept rows of t."""
    p = torch.zeros((touched, s["most"], t.shape[1]), device=DEV)
    p[which, s["place"]] = t[s["row"]].float()
    return p


def _plain_product(s, transpose):
    e, which = _by_expert(s)
    x, w = _padded(s, s["rows"], which, e.numel()), s["w"][e].float()
    y = torch.bmm(x, w if transpose else w.transpose(1, 2))
    s["out"][s["row"]] = y[which, s["place"]].to(torch.bfloat16)
    return s["out"]


def _plain_weight_grad(s):
    e, which = _by_expert(s)
    g, x = (_padded(s, s[k], which, e.numel()) for k in ("grad", "rows"))
    y = torch.bmm(g.transpose(1, 2), x)
    if s["add"]:
        s["out"][e] = (s["out"][e].float() + y).to(s["out"].dtype)
        return s["out"]
    s["out"].zero_()
    s["out"][e] = y.to(s["out"].dtype)
    return s["out"]


def _plain_mlp_keep(s):
    F = s["F"]
    e, which = _by_expert(s)
    h = torch.bmm(_padded(s, s["rows"], which, e.numel()), s["w1"][e].float().transpose(1, 2))
    gate, up = h[..., :F], h[..., F:]
    y = torch.bmm(gate / (1.0 + torch.exp(-gate)) * up, s["w2"][e].float().transpose(1, 2))
    s["out"][s["row"]] = y[which, s["place"]].to(torch.bfloat16)
    s["h"][s["row"]] = h[which, s["place"]].to(torch.bfloat16)
    return s["out"], s["h"]


def _plain_mlp_backward(s):
    F = s["F"]
    e, which = _by_expert(s)
    x, gy, h = (_padded(s, s[k], which, e.numel()) for k in ("rows", "grad", "h"))
    gate, up = h[..., :F], h[..., F:]
    sig = 1.0 / (1.0 + torch.exp(-gate))
    da = torch.bmm(gy, s["w2"][e].float())
    dh = torch.cat((da * up * sig * (1.0 + gate * (1.0 - sig)), da * gate * sig), dim=2)
    gx = torch.bmm(dh, s["w1"][e].float())
    s["out"][s["row"]] = gx[which, s["place"]].to(torch.bfloat16)
    s["g1"].zero_()
    s["g2"].zero_()
    s["g1"][e] = torch.bmm(dh.transpose(1, 2), x).to(torch.bfloat16)
    s["g2"][e] = torch.bmm(gy.transpose(1, 2), gate * sig * up).to(torch.bfloat16)
    return s["out"], s["g1"], s["g2"]


def _plain_rms(s):
    t = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
    rstd = 1.0 / torch.sqrt((t * t).mean(dim=1, keepdim=True) + s["eps"])
    y = t * rstd * s["weight"].float()
    codes = scales = None
    if s["quantize"]:
        blocks = y.unflatten(1, (-1, GROUP))
        top = blocks.abs().amax(dim=2)
        scales = torch.where(top > 0, top / E4M3_MAX, 1.0)
        codes = (blocks / scales.unsqueeze(2)).clamp(-E4M3_MAX, E4M3_MAX).flatten(1).to(torch.float8_e4m3fn)
    return (None if s["y_type"] is None else y.to(s["y_type"]), codes, scales,
            None if s["residual"] is None else t.to(s["residual"].dtype), rstd[:, 0])


def _plain_rms_backward(s):
    rstd, gy = s["rstd"][:, None], s["grad"].float()
    xh = s["total"].float() * rstd
    q = gy * s["weight"].float()
    g = rstd * (q - xh * (q * xh).mean(dim=1, keepdim=True))
    if s["grad_total"] is not None:
        g = g + s["grad_total"].float()
    return g.to(s["total"].dtype), (gy * xh).sum(dim=0)


# ---- one pass ---------------------------------------------------------------------------------
def run(state):
    s = state
    op = s["op"]
    if op in ("product", "product_t"):
        if own:
            return s["dispatcher"].grouped_product(s["rows"], s["w"], transpose=op == "product_t", out=s["out"])
        return _plain_product(s, op == "product_t")
    if op == "weight_grad":
        if own:
            return s["dispatcher"].grouped_weight_grad(s["grad"], s["rows"], out=s["out"], accumulate=s["add"])
        return _plain_weight_grad(s)
    if op == "mlp_keep":
        if own:
            return s["dispatcher"].grouped_mlp_keep(s["rows"], s["w1"], s["w2"], h=s["h"], scratch=s["scratch"],
                                                    out=s["out"])
        return _plain_mlp_keep(s)
    if op == "mlp_backward":
        if own:
            return s["dispatcher"].grouped_mlp_backward(s["grad"], s["rows"], s["h"], s["w1"], s["w2"],
                                                        grad_perm=s["out"], grad_w1=s["g1"], grad_w2=s["g2"],
                                                        scratch=s["scratch"])
        return _plain_mlp_backward(s)
    if op == "rms":
        if own:
            from combine_routing_preprocess_amd import rms_norm
            return rms_norm(s["x"], s["weight"], s["eps"], residual=s["residual"], quantize=s["quantize"],
                            want_rows=s["y_type"] is not None, **s["out"])
        return _plain_rms(s)
    if own:
        from combine_routing_preprocess_amd import rms_norm_backward
        return rms_norm_backward(s["grad"], s["total"], s["rstd"], s["weight"], grad_total=s["grad_total"], **s["out"])
    return _plain_rms_backward(s)


def work(case):
    T, op = case["T"], case["op"]
    if op == "rms":
        H, sx, sr = case["H"], _SIZE[case["x"]], _SIZE.get(case["res"], 0)
        out = {"bf16": 2, "f32": 4, "fp8": 1 + 4 / GROUP, "both": 3 + 4 / GROUP}[case["y"]]
        return {"bytes": int(T * H * (sx + 2 * sr + out)) + H * _SIZE[case["w"]] + 4 * T, "flops": 6 * T * H}
    if op == "rms_backward":
        H, st = case["H"], _SIZE[case["res"]]
        rows = T * H * (st * (3 if case["grad_total"] else 2) + _SIZE[case["y"]])
        return {"bytes": rows + H * (_SIZE[case["w"]] + 4) + 4 * T, "flops": 9 * T * H}
    E = case["E"]
    copies = T * case["K"] - min(case["empty"], T * case["K"] // 2)
    touched = E * (1.0 - (1.0 - 1.0 / E) ** copies)
    if op.startswith("mlp"):
        H, F = case["H"], case["F"]
        weights = int(touched * 6 * F * H)
        if op == "mlp_keep":
            return {"bytes": weights + copies * (2 * H + 2 * F) * 2, "flops": 6 * copies * F * H}
        return {"bytes": weights + 6 * E * F * H + copies * (3 * H + 2 * F) * 2, "flops": 12 * copies * F * H}
    N, M = case["N"], case["M"]
    flops = 2 * copies * N * M
    if op == "weight_grad":
        size = _SIZE[case["out"]]
        return {"bytes": int((2 * touched if case["add"] else E) * N * M * size) + copies * (N + M) * 2, "flops": flops}
    return {"bytes": int(touched * N * M * 2) + copies * (N + M) * 2, "flops": flops}


# ---- the definitions in 64 bits ---------------------------------------------------------------
def _each_expert(s):
    ids, counts = torch.unique_consecutive(s["expert"], return_counts=True)
    at = 0
    for e, n in zip(ids.tolist(), counts.tolist()):
        yield e, s["row"][at:at + n]
        at += n


def _exact_routed(s, case):
    op, f64 = case["op"], torch.float64
    if op in ("product", "product_t"):
        y = torch.zeros(s["out"].shape, dtype=f64, device=DEV)
        for e, r in _each_expert(s):
            w = s["w"][e].to(f64)
            y[r] = s["rows"][r].to(f64) @ (w.T if op == "product" else w)
        return y
    if op == "weight_grad":
        y = s["out"].to(f64) if s["add"] else torch.zeros(s["out"].shape, dtype=f64, device=DEV)
        for e, r in _each_expert(s):
            y[e] += s["grad"][r].to(f64).T @ s["rows"][r].to(f64)
        return y
    F = case["F"]
    y = torch.zeros(s["out"].shape, dtype=f64, device=DEV)
    if op == "mlp_keep":
        h = torch.zeros(s["h"].shape, dtype=f64, device=DEV)
        for e, r in _each_expert(s):
            h[r] = s["rows"][r].to(f64) @ s["w1"][e].to(f64).T
            a = torch.special.expit(h[r, :F]) * h[r, :F] * h[r, F:]
            y[r] = a @ s["w2"][e].to(f64).T
        return y, h
    g1 = torch.zeros(s["g1"].shape, dtype=f64, device=DEV)
    g2 = torch.zeros(s["g2"].shape, dtype=f64, device=DEV)
    for e, r in _each_expert(s):
        gy = s["grad"][r].to(f64)
        with torch.enable_grad():
            h = s["h"][r].to(f64).requires_grad_(True)
            a = torch.special.expit(h[:, :F]) * h[:, :F] * h[:, F:]
            dh, = torch.autograd.grad((a @ s["w2"][e].to(f64).T * gy).sum(), h)
        y[r] = dh @ s["w1"][e].to(f64)
        g1[e] = dh.T @ s["rows"][r].to(f64)
        g2[e] = gy.T @ a.detach()
    return y, g1, g2


def _exact_rms(s):
    t = s["x"].to(torch.float64)
    if s["residual"] is not None:
        t = t + s["residual"].to(torch.float64)
    rstd = torch.rsqrt(torch.linalg.vector_norm(t, dim=1) ** 2 / t.shape[1] + s["eps"])
    y = torch.einsum("th,t,h->th", t, rstd, s["weight"].to(torch.float64))
    codes = scales = None
    if s["quantize"]:
        scales = torch.linalg.vector_norm(y.view(len(y), -1, GROUP), ord=float("inf"), dim=2) / E4M3_MAX
        scales[scales == 0] = 1.0
        codes = y / scales.repeat_interleave(GROUP, dim=1)     # before their rounding to 8 bits
    return None if s["y_type"] is None else y, codes, scales, None if s["residual"] is None else t, rstd


def _exact_rms_backward(s):
    t, gy = s["total"].to(torch.float64), s["grad"].to(torch.float64)
    r = s["rstd"].to(torch.float64).unsqueeze(1)
    q = gy * s["weight"].to(torch.float64)
    g = r * q - t * (r ** 3 * (q * t).sum(1, keepdim=True) / t.shape[1])
    if s["grad_total"] is not None:
        g += s["grad_total"].to(torch.float64)
    return g, torch.einsum("th,th,t->h", gy, t, r[:, 0])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rms":
        return _exact_rms(s)
    if case["op"] == "rms_backward":
        return _exact_rms_backward(s)
    return _exact_routed(s, case)
