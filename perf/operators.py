"""The operators around the expert layer, as measured cases: the norm in front
of it, the balance loss on its routing, and the gradient of its router.

    norm            RMS norm with the residual's addition, 16/32-bit and e4m3 outputs
    norm_backward   its gradient (input and weight)
    balance         balance loss, per-expert counts, and the loss's gradient in the logits
    route_backward  gradient of the routing weights and logits in the router's
                    weights, its bias and the activations

`own` selects the library's kernels; otherwise `run` computes the plain form
with elementary torch operations.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -126


def listed():
    return [
        # one decoded token of the DeepSeek-V2-Lite-shaped layer: latency
        dict(name="norm one token", op="norm", T=1, H=2048, dtype="bf16", residual=True, group=0),
        # an odd width and a ragged batch in fp32, no residual yet (first layer)
        dict(name="norm odd width fp32", op="norm", T=129, H=1413, dtype="f32", residual=False,
             group=0),
        # the 8192-token prefill layer, rows also sent on in 8 bits
        dict(name="norm prefill and 8 bits", op="norm", T=8192, H=4096, dtype="bf16",
             residual=True, group=128),
        # a short training batch of the DeepSeek-V2-Lite-shaped layer
        dict(name="norm gradient 300 tokens", op="norm_backward", T=300, H=2048, dtype="f16",
             residual=True),
        # the prefill layer's batch as a training batch
        dict(name="norm gradient 8192 tokens", op="norm_backward", T=8192, H=4096, dtype="bf16",
             residual=True),
        # the largest small batch of the layer, 64 experts top-6: latency
        dict(name="balance 64 tokens", op="balance", T=64, E=64, k=6, mode="softmax", seqs=1,
             mask=False),
        # the prefill layer's routing, one sequence
        dict(name="balance 8192 tokens", op="balance", T=8192, E=256, k=8, mode="softmax", seqs=1,
             mask=False),
        # a packed training batch of ragged, partly padded sequences, the
        # sigmoid-routed layer's 256 experts top-10
        dict(name="balance packed sequences", op="balance", T=131072, E=256, k=10, mode="sigmoid",
             seqs=37, mask=True),
        # a short batch of the DeepSeek-V2-Lite-shaped router
        dict(name="router gradient 129 tokens", op="route_backward", T=129, H=2048, E=64, k=6,
             mode="softmax"),
        # few experts, sigmoid routing
        dict(name="router gradient 32 experts", op="route_backward", T=2048, H=4096, E=32, k=8,
             mode="sigmoid"),
        # the prefill layer's router and batch
        dict(name="router gradient 8192 tokens", op="route_backward", T=8192, H=4096, E=256, k=8,
             mode="softmax"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "balance", "balance", "route_backward"])
    if op in ("norm", "norm_backward"):
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        H = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            H = (H + 7) // 8 * 8
        T = _log(rng, 1, min(8192, 8192 * 4096 * 2 // (BYTES[dtype] * H)))
        case = dict(op=op, T=T, H=H, dtype=dtype, residual=rng.random() < 0.7)
        if op == "norm":
            case["group"] = rng.choice([0, 0, 32, 64, 128, H])
        return case
    E = rng.choice([8, 16, 32, 60, 64, 100, 128, 160, 255, 256])
    k = rng.randint(1, min(10, E))
    mode = rng.choice(["softmax", "sigmoid"])
    if op == "balance":
        T = _log(rng, 1, 131072)
        return dict(op=op, T=T, E=E, k=k, mode=mode, seqs=rng.choice([1, 1, _log(rng, 2, 64)]),
                    mask=rng.random() < 0.5)
    return dict(op=op, T=_log(rng, 1, 8192), H=128 * _log(rng, 2, 32), E=E, k=k, mode=mode)


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _routing(case, g):
    """Logits of unit scale with a few favoured experts, and the selected ids."""
    T, E, k = case["T"], case["E"], case["k"]
    skew = torch.randn(E, device="cuda", generator=g) * 0.7
    logits = torch.randn(T, E, device="cuda", generator=g) + skew
    idx = torch.topk(logits, k, dim=1).indices.to(torch.int32).contiguous()
    return logits, idx


def _layer(case, hidden, W=None, bias=None):
    """The layer handle that a user's program keeps (router only: no expert is bound)."""
    from quantized_routed_expert_04_b200 import binding
    layer = binding.StrataMoE(hidden, 128, case["E"], case["k"], 0, case["E"])
    if case["mode"] == "sigmoid":
        layer.set_routing(binding.ROUTE_SIGMOID, None, 2.5)
    if W is not None:
        layer.set_router(W, bias)
    return layer


def prepare(case, seed):
    g = _gen(seed)
    op, T = case["op"], case["T"]
    st = dict(case)
    if op in ("norm", "norm_backward"):
        H, dt = case["H"], DTYPES[case["dtype"]]
        # a few wide channels, as residual streams have them
        chan = torch.exp(torch.randn(H, device="cuda", generator=g) * 0.5)
        st["x"] = (torch.randn(T, H, device="cuda", generator=g) * chan).to(dt)
        st["weight"] = 1 + 0.2 * torch.randn(H, device="cuda", generator=g)
        second = None
        if case["residual"]:
            second = (torch.randn(T, H, device="cuda", generator=g) * chan * 2).to(dt)
        if op == "norm":
            st["residual"] = second
            st["residual_out"] = torch.empty_like(st["x"]) if case["residual"] else None
            st["out"] = torch.empty_like(st["x"])
            st["out_q8"] = st["scales"] = None
            if case["group"]:
                st["out_q8"] = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda")
                st["scales"] = torch.empty(T, -(-H // case["group"]), device="cuda")
        else:
            st["dout"] = torch.randn(T, H, device="cuda", generator=g).to(dt)
            st["dsum"] = second
            st["dx"] = torch.empty_like(st["x"])
            st["dweight"] = torch.empty(H, device="cuda")
            if own:
                from quantized_routed_expert_04_b200 import binding
                st["workspace"] = torch.empty(binding.strata_rmsnorm_backward_workspace(T, H),
                                              dtype=torch.uint8, device="cuda")
        return st
    E = case["E"]
    st["logits"], st["idx"] = _routing(case, g)
    if op == "balance":
        n = case["seqs"]
        st["coef"] = 0.01
        st["seq_off"] = st["mask"] = None
        if n > 1:
            # ragged sequences, empty ones among them, and rows behind the last
            cuts = torch.rand(n + 1, device="cuda", generator=g).sort().values
            cuts = ((cuts - cuts[0]) * T * 0.98 / max(1e-3, float(cuts[-1] - cuts[0])))
            st["seq_off"] = cuts.to(torch.int32).clamp_(0, T)
        if case["mask"]:
            st["mask"] = (torch.rand(T, device="cuda", generator=g) < 0.9).to(torch.uint8)
        st["grad"] = torch.rand(1, device="cuda", generator=g) + 0.5
        st["counts"] = torch.empty(n, E, dtype=torch.int32, device="cuda")
        st["tokens"] = torch.empty(n, dtype=torch.int32, device="cuda")
        st["loss"] = torch.empty(1, device="cuda")
        st["dlogits"] = torch.empty(T, E, device="cuda")
        if own:
            st["layer"] = layer = _layer(case, 128)
            st["workspace"] = torch.empty(layer.balance_workspace(T, n), dtype=torch.uint8,
                                          device="cuda")
        return st
    H = case["H"]
    st["x"] = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
    st["W"] = torch.randn(E, H, device="cuda", generator=g) / math.sqrt(H)
    st["dw"] = torch.randn(T, case["k"], device="cuda", generator=g) * 0.1
    st["dlogits"] = torch.randn(T, E, device="cuda", generator=g) * 1e-3
    st["dW"] = torch.empty(E, H, device="cuda")
    st["db"] = torch.empty(E, device="cuda")
    st["dx"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    if own:
        st["layer"] = layer = _layer(case, H, st["W"])
        st["workspace"] = torch.empty(layer.route_backward_workspace(T), dtype=torch.uint8,
                                      device="cuda")
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    return _RUN[st["op"]](st)


def _run_norm(st):
    if own:
        from quantized_routed_expert_04_b200 import binding
        binding.strata_rmsnorm(st["x"], st["residual"], st["weight"], EPS, st["residual_out"],
                               st["out"], st["out_q8"], st["scales"], st["group"])
        return [st["residual_out"], st["out"], st["out_q8"], st["scales"]]
    dt, G = st["x"].dtype, st["group"]
    s = st["x"].float()
    if st["residual"] is not None:
        s = s + st["residual"].float()
    y = s * torch.rsqrt((s * s).mean(1, keepdim=True) + EPS) * st["weight"]
    q = scales = None
    if G:
        T, H = y.shape
        n = -(-H // G)
        yg = torch.nn.functional.pad(y, (0, n * G - H)).view(T, n, G)
        scales = (yg.abs().amax(2) / E4M3_MAX).clamp(min=MIN_SCALE)
        q = (yg / scales[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        q = q.view(T, n * G)[:, :H]
    return [s.to(dt) if st["residual"] is not None else None, y.to(dt), q, scales]


def _run_norm_backward(st):
    if own:
        from quantized_routed_expert_04_b200 import binding
        binding.strata_rmsnorm_backward(st["x"], st["weight"], EPS, st["dout"], st["dsum"],
                                        st["dx"], st["dweight"], st["workspace"])
        return [st["dx"], st["dweight"]]
    h, dy = st["x"].float(), st["dout"].float()
    i = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    n = h * i
    gy = dy * st["weight"]
    dx = i * (gy - n * (gy * n).mean(1, keepdim=True))
    if st["dsum"] is not None:
        dx = dx + st["dsum"].float()
    return [dx.to(st["x"].dtype), (dy * n).sum(0)]


def _segments(st):
    """Per token: its sequence (n_seq: none) and whether it counts."""
    T, n = st["T"], st["seqs"]
    t = torch.arange(T, dtype=torch.int32, device="cuda")
    if st["seq_off"] is None:
        seg, live = torch.zeros_like(t), torch.ones(T, device="cuda")
    else:
        seg = (t[:, None] >= st["seq_off"][None, 1:]).sum(1).to(torch.int32)
        live = ((seg < n) & (t >= st["seq_off"][0])).float()
    if st["mask"] is not None:
        live = live * (st["mask"] != 0)
    return seg.clamp(max=n - 1).long(), live


def _run_balance(st):
    if own:
        layer = st["layer"]
        layer.balance(st["logits"], st["idx"], st["coef"], st["counts"], st["tokens"], st["loss"],
                      st["workspace"], st["seq_off"], st["mask"])
        layer.balance_backward(st["logits"], st["coef"], st["counts"], st["tokens"], st["dlogits"],
                               st["grad"], st["seq_off"], st["mask"])
        return [st["loss"], st["counts"], st["tokens"], st["dlogits"]]
    T, E, k, n = st["T"], st["E"], st["k"], st["seqs"]
    logits, (seg, live) = st["logits"], _segments(st)
    if st["mode"] == "softmax":
        ex = torch.exp(logits - logits.amax(1, keepdim=True))
        p = ex / ex.sum(1, keepdim=True)
    else:
        s = 1 / (1 + torch.exp(-logits))
        total = s.sum(1, keepdim=True)
        p = s / total
    member = (seg[None, :] == torch.arange(n, device="cuda")[:, None]) * live   # [n][T]
    tokens = member.sum(1)
    safe = tokens.clamp(min=1)
    P = (member @ p) / safe[:, None]
    slot = (seg[:, None] * E + st["idx"].long()).reshape(-1)
    hit = live.to(torch.int32)[:, None].expand(T, k).reshape(-1)
    counts = torch.zeros(n * E, dtype=torch.int32, device="cuda").index_add_(0, slot, hit)
    counts = counts.view(n, E)
    f = counts.float() * (E / k) / safe[:, None]
    loss = (f * P).sum().reshape(1) * (st["coef"] / n)
    ft = f[seg]
    u = (st["grad"] * (st["coef"] / n) / safe)[seg] * live
    centred = ft - (ft * p).sum(1, keepdim=True)
    slope = p if st["mode"] == "softmax" else s * (1 - s) / total
    return [loss, counts, tokens.to(torch.int32), u[:, None] * slope * centred]


def _run_route_backward(st):
    if own:
        st["layer"].route_backward(st["x"], st["logits"], st["idx"], st["dw"], st["dlogits"],
                                   st["dW"], st["db"], st["dx"], st["workspace"])
        return [st["dW"], st["db"], st["dx"]]
    sel = st["idx"].long()
    l = st["logits"].gather(1, sel)
    if st["mode"] == "softmax":
        ex = torch.exp(l - l.amax(1, keepdim=True))
        w = ex / ex.sum(1, keepdim=True)
        d = w * (st["dw"] - (w * st["dw"]).sum(1, keepdim=True))
    else:
        s = 1 / (1 + torch.exp(-l))
        total = s.sum(1, keepdim=True)
        d = 2.5 * s * (1 - s) / total * (st["dw"] - (s / total * st["dw"]).sum(1, keepdim=True))
    dl = st["dlogits"].scatter_add(1, sel, d)
    return [dl.t() @ st["x"].float(), dl.sum(0), (dl @ st["W"]).to(torch.bfloat16)]


_RUN = {"norm": _run_norm, "norm_backward": _run_norm_backward, "balance": _run_balance,
        "route_backward": _run_route_backward}


# ---------------------------------------------------------------- work
def work(case):
    """Bytes of every input read once and every output written once, and the
    operations of the formulas."""
    op, T = case["op"], case["T"]
    if op in ("norm", "norm_backward"):
        H, b = case["H"], BYTES[case["dtype"]]
        n = T * H
        if op == "norm":
            moved = n * b * (4 if case["residual"] else 2) + 4 * H
            if case["group"]:
                moved += n + 4 * T * -(-H // case["group"])
            return {"bytes": moved, "flops": 6 * n}
        return {"bytes": n * b * (4 if case["residual"] else 3) + 8 * H, "flops": 12 * n}
    E, k = case["E"], case["k"]
    if op == "balance":
        # logits and ids in; the gradient out.  The loss couples every token,
        # so a backward of its own reads the logits again
        return {"bytes": T * (12 * E + 4 * k) + case["seqs"] * 4 * E, "flops": 16 * T * E}
    H = case["H"]
    return {"bytes": 4 * T * H + 8 * E * H + T * (8 * E + 8 * k) + 4 * E,
            "flops": 4 * T * E * H + 10 * T * k}


# ---------------------------------------------------------------- 64-bit definitions
def exact(case, seed):
    st = prepare(case, seed)
    return _EXACT[case["op"]](st)


def _exact_norm(st):
    x = st["x"].double()
    if st["residual"] is not None:
        x = x + st["residual"].double()
    length = torch.sqrt(x.pow(2).sum(1) / x.shape[1] + EPS)
    y = x / length[:, None] * st["weight"].double()
    q = scales = None
    if st["group"]:
        G, parts, sc = st["group"], [], []
        for c in range(0, x.shape[1], G):
            part = y[:, c:c + G]
            step = torch.clamp(part.abs().max(1).values / E4M3_MAX, min=MIN_SCALE)
            parts.append(part / step[:, None])
            sc.append(step)
        q, scales = torch.cat(parts, 1), torch.stack(sc, 1)
    return [x if st["residual"] is not None else None, y, q, scales]


def _exact_norm_backward(st):
    x = st["x"].double().requires_grad_(True)
    g = st["weight"].double().requires_grad_(True)
    y = x / torch.sqrt(x.pow(2).sum(1, keepdim=True) / x.shape[1] + EPS) * g
    total = (y * st["dout"].double()).sum()
    if st["dsum"] is not None:
        total = total + (x * st["dsum"].double()).sum()
    return list(torch.autograd.grad(total, (x, g)))


def _exact_balance(st):
    T, E, k, n = st["T"], st["E"], st["k"], st["seqs"]
    logits = st["logits"].double().requires_grad_(True)
    off = [0, T] if st["seq_off"] is None else st["seq_off"].tolist()
    keep = torch.ones(T, dtype=torch.bool, device="cuda") if st["mask"] is None \
        else st["mask"] != 0
    loss = torch.zeros((), dtype=torch.float64, device="cuda")
    counts = torch.zeros(n, E, dtype=torch.int64, device="cuda")
    tokens = torch.zeros(n, dtype=torch.int64, device="cuda")
    for b in range(n):
        use = keep[off[b]:off[b + 1]]
        l = logits[off[b]:off[b + 1]][use]
        if l.shape[0] == 0:
            continue
        if st["mode"] == "softmax":
            p = torch.softmax(l, 1)
        else:
            p = torch.sigmoid(l)
            p = p / p.sum(1, keepdim=True)
        ids = st["idx"][off[b]:off[b + 1]][use].long().reshape(-1)
        counts[b] = torch.bincount(ids, minlength=E)
        tokens[b] = l.shape[0]
        share = counts[b].double() * E / (k * l.shape[0])
        loss = loss + (share * p.mean(0)).sum()
    loss = loss * st["coef"] / n
    d = torch.zeros_like(logits)
    if loss.requires_grad:
        d = torch.autograd.grad(loss, logits, st["grad"].double()[0])[0]
    return [loss.detach().reshape(1), counts, tokens, d]


def _exact_route_backward(st):
    l = st["logits"].double().requires_grad_(True)
    W = st["W"].double().requires_grad_(True)
    x = st["x"].double().requires_grad_(True)
    b = torch.zeros(st["E"], dtype=torch.float64, device="cuda", requires_grad=True)
    sel = torch.gather(l, 1, st["idx"].long())
    if st["mode"] == "softmax":
        w = torch.softmax(sel, 1)
    else:
        w = torch.sigmoid(sel)
        w = 2.5 * w / w.sum(1, keepdim=True)
    dl, = torch.autograd.grad((w * st["dw"].double()).sum(), l)
    dl = dl + st["dlogits"].double()
    out = torch.nn.functional.linear(x, W, b)
    dW, db, dx = torch.autograd.grad(out, (W, b, x), dl)
    return [dW, db, dx]


_EXACT = {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "balance": _exact_balance,
          "route_backward": _exact_route_backward}
