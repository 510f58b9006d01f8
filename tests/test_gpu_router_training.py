"""Balance loss, counts and the router's gradient against 64-bit formulas.

Tolerances (u = 2^-24, fp32).  A probability comes from one exponential (2
units in the last place), a sum of at most 256 terms taken 8 and then a tree of
5, and two products: within 32 u.  Sums over tokens run over at most 32 rows of
a warp, 8 warps, then double: the loss, a sum of positive terms, is within
128 u.  dlogits = u_b slope (f - sum f p) is a difference: 128 u times
u_b slope (f + sum f p).
dW: dl carries 32 u of the sum of its terms' magnitudes; its products with x
are exact to u (dl as a sum of three bf16 numbers keeps 24 bits); the tensor
core adds 16 of them at a time and may cut the running sum at 2^-23, three
times per 16 tokens: (3 T / 8 + 64) u of sum |dl| |x|.
dx: dl and W rounded once to f16, half a step each: 2^-11 relative, so 2^-10
(1 + 2^-10) of sum |dl| |W|; below f16's normal range half a step is absolute:
2^-25 of the row's power of two for dl, 2^-25 / 2^8 for W.  Then half a bf16
step, 2^-8.
"""
import math

import pytest

torch = pytest.importorskip("torch")

from quantized_routed_expert_04_b200 import binding  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BAD = binding.Status.INVALID_ARG
SCALE = 2.5


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def make_layer(E, k, mode="softmax", H=128, W=None, bias=None):
    layer = binding.StrataMoE(H, 128, E, k, 0, E)
    if mode == "sigmoid":
        layer.set_routing(binding.ROUTE_SIGMOID, None, SCALE)
    if W is not None:
        layer.set_router(W, bias)
    return layer


def routing(T, E, k, seed, scale=1.5):
    g = gen(seed)
    logits = torch.randn(T, E, device="cuda", generator=g) * scale
    idx = torch.topk(logits, k, dim=1).indices.int().contiguous() if T else \
        torch.empty(0, k, dtype=torch.int32, device="cuda")
    return logits, idx


def probs(logits, mode):
    """(p, slope) in 64 bits; a row of -inf has no probabilities."""
    l = logits.double()
    if mode == "softmax":
        m = l.amax(1, keepdim=True)
        p = torch.where(m == -math.inf, torch.zeros_like(l), torch.softmax(l, 1))
        return p, p
    s = torch.sigmoid(l)
    S = s.sum(1, keepdim=True)
    return (s / S).nan_to_num(), (s * torch.sigmoid(-l) / S).nan_to_num()


def exact_balance(logits, idx, mode, k, coef, dloss, off, mask):
    T, E = logits.shape
    n_seq = len(off) - 1
    p, slope = probs(logits, mode)
    keep = torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask != 0
    counts = torch.zeros(n_seq, E, dtype=torch.int64, device="cuda")
    tokens = torch.zeros(n_seq, dtype=torch.int64, device="cuda")
    d = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(d)
    loss = 0.0
    for b in range(n_seq):
        rows = torch.arange(off[b], off[b + 1], device="cuda")
        rows = rows[keep[rows]]
        n = rows.numel()
        tokens[b] = n
        if n == 0:
            continue
        counts[b] = torch.bincount(idx[rows].long().reshape(-1), minlength=E)
        f = counts[b].double() * E / (k * n)
        loss += float((f * p[rows].sum(0) / n).sum())
        u = dloss * coef / (n_seq * n)
        dot = (p[rows] * f).sum(1, keepdim=True)
        d[rows] = u * slope[rows] * (f - dot)
        mag[rows] = abs(u) * slope[rows] * (f + dot)
    return loss * coef / n_seq, counts, tokens, d, mag


def run_balance(layer, logits, idx, coef, dloss=None, off=None, mask=None, fill=True, stream=None):
    T, E = logits.shape
    n_seq = 1 if off is None else len(off) - 1
    seq = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    counts = torch.full((n_seq, E), -7, dtype=torch.int32, device="cuda")
    tokens = torch.full((n_seq,), -7, dtype=torch.int32, device="cuda")
    loss = torch.full((1,), 7.0, device="cuda")
    ws = torch.empty(layer.balance_workspace(T, n_seq), dtype=torch.uint8, device="cuda")
    if fill:
        ws.fill_(0xFF)   # NaN and -1: nothing may be read before it is written
    d = torch.full((T, E), 7.0, device="cuda")
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    layer.balance(logits, idx, coef, counts, tokens, loss, ws, seq, mask, stream=stream)
    g = None if dloss is None else torch.full((1,), dloss, device="cuda")
    layer.balance_backward(logits, coef, counts, tokens, d, g, seq, mask, stream=stream)
    torch.cuda.synchronize()
    return loss, counts, tokens, d


def check_balance(layer, logits, idx, mode, k, coef=0.01, dloss=None, off=None, mask=None):
    T = logits.shape[0]
    loss, counts, tokens, d = run_balance(layer, logits, idx, coef, dloss, off, mask)
    assert int(layer.status()[0]) == 0
    el, ec, et, ed, mag = exact_balance(logits, idx, mode, k, coef, 1.0 if dloss is None else dloss,
                                        [0, T] if off is None else off, mask)
    assert torch.equal(counts.long(), ec) and torch.equal(tokens.long(), et)
    assert abs(float(loss) - el) <= abs(el) * 128 * U, (float(loss), el)
    err = (d.double() - ed).abs()
    assert not bool(d.isnan().any())
    assert bool((err <= mag * 128 * U + 2.0 ** -140).all()), float((err / mag.clamp(min=1e-300)).max() / U)
    return loss, counts, tokens, d


@pytest.mark.parametrize("mode", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 8, 8), (7, 16, 3), (64, 64, 6),
                                   (65, 60, 6), (129, 32, 8), (200, 100, 4), (33, 256, 32),
                                   (17, 255, 10), (300, 129, 2), (5000, 256, 8), (20011, 24, 4)])
def test_balance_one_sequence(T, E, k, mode):
    layer = make_layer(E, k, mode)
    logits, idx = routing(T, E, k, 1)
    check_balance(layer, logits, idx, mode, k)
    g = gen(2)
    mask = (torch.rand(T, device="cuda", generator=g) < 0.7).to(torch.uint8) * 3
    check_balance(layer, logits, idx, mode, k, coef=1.5, dloss=-2.0, mask=mask)
    layer.close()


@pytest.mark.parametrize("mode", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,off", [
    (10, 8, 2, [0, 0, 3, 3, 4, 10, 10]),         # empty sequences at both ends and between
    (300, 64, 6, [5, 100, 101, 290]),            # tokens in front of the first, behind the last
    (9, 16, 1, [0, 1, 2, 3, 4, 5, 6, 7, 8, 9]),  # one token each
    (700, 256, 8, [0, 16, 32, 33, 600, 700]),    # cuts at and beside the blocks' cuts
    (40, 32, 4, [40, 40, 40]),                   # nothing but empty sequences
    (9000, 60, 3, [0, 8999, 9000]),
])
def test_balance_sequences(T, E, k, off, mode):
    layer = make_layer(E, k, mode)
    logits, idx = routing(T, E, k, 3)
    check_balance(layer, logits, idx, mode, k, off=off)
    mask = (torch.rand(T, device="cuda", generator=gen(4)) < 0.5).to(torch.uint8)
    check_balance(layer, logits, idx, mode, k, off=off, mask=mask, dloss=0.25)
    layer.close()


def test_balance_many_sequences():
    T, E, k = 12000, 64, 6
    layer = make_layer(E, k)
    logits, idx = routing(T, E, k, 5)
    off = [0] + sorted(torch.randint(0, T, (900,), generator=torch.Generator().manual_seed(6)).tolist()) + [T]
    check_balance(layer, logits, idx, "softmax", k, off=off)
    layer.close()


@pytest.mark.parametrize("mode", ["softmax", "sigmoid"])
def test_balance_masked_places_may_hold_anything(mode):
    T, E, k = 90, 64, 6
    layer = make_layer(E, k, mode)
    logits, idx = routing(T, E, k, 7)
    mask = torch.ones(T, dtype=torch.uint8, device="cuda")
    mask[10:40] = 0
    want = check_balance(layer, logits, idx, mode, k, mask=mask)
    logits[10:20] = float("nan")
    logits[20:30] = float("inf")
    logits[30:40] = -float("inf")
    idx[10:40] = 1 << 30
    got = run_balance(layer, logits, idx, 0.01, mask=mask)
    assert int(layer.status()[0]) == 0
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    mask.zero_()   # nothing counts at all
    loss, counts, tokens, d = run_balance(layer, logits, idx, 0.01, mask=mask)
    assert float(loss) == 0 and not counts.any() and not tokens.any() and not d.any()
    layer.close()


@pytest.mark.parametrize("mode", ["softmax", "sigmoid"])
def test_balance_extreme_logits(mode):
    # experts ruled out by -inf or the lowest number, a row of nothing but
    # -inf, rows of the lowest number alone, wide spreads
    T, E, k = 40, 16, 2
    layer = make_layer(E, k, mode)
    logits, idx = routing(T, E, k, 8)
    low = torch.finfo(torch.float32).min
    logits[:10, 4:] = -math.inf
    logits[10:20, 4:] = low
    logits[20] = -math.inf
    logits[21] = low
    logits[22] = 3e38
    logits[23] *= 40
    check_balance(layer, logits, idx, mode, k)
    logits[5, 1] = math.nan        # a counting NaN is not hidden
    loss, _, _, d = run_balance(layer, logits, idx, 0.01)
    assert bool(loss.isnan()) and bool(d[5].isnan().any()) and not bool(d[6].isnan().any())
    layer.close()


def test_balance_same_expert_twice_and_bad_ids():
    T, E, k = 50, 8, 4
    layer = make_layer(E, k)
    logits, idx = routing(T, E, k, 9)
    idx[:, 1] = idx[:, 0]
    check_balance(layer, logits, idx, "softmax", k)
    good = idx.clone()
    idx[3, 2], idx[7, 0] = -1, E
    _, counts, tokens, _ = run_balance(layer, logits, idx, 0.01)
    st, bits = layer.status()
    assert st == binding.Status.DEVICE_STATUS and bits == 2
    want = torch.bincount(good.reshape(-1).long(), minlength=E)
    want[good[3, 2].long()] -= 1
    want[good[7, 0].long()] -= 1
    assert torch.equal(counts[0].long(), want) and int(tokens[0]) == T
    assert int(layer.status()[0]) == 0
    layer.close()


def test_balance_bad_offsets_are_reported():
    T, E, k = 100, 8, 2
    layer = make_layer(E, k)
    logits, idx = routing(T, E, k, 10)
    for off in ([0, 50, 40, 100], [-5, 100], [0, 101], [0, 1 << 30, 3]):
        run_balance(layer, logits, idx, 0.01, off=off)   # spans are clamped: nothing out of bounds
        st, bits = layer.status()
        assert st == binding.Status.DEVICE_STATUS and bits == 8, off
    check_balance(layer, logits, idx, "softmax", k, off=[0, 100])
    layer.close()


def test_balance_unaligned_rows():
    T, E, k = 77, 64, 6
    layer = make_layer(E, k)
    logits, idx = routing(T, E, k, 11)
    buf = torch.empty(T * E + 3, device="cuda")
    shifted = buf[3:].view(T, E)
    shifted.copy_(logits)
    # (its experts sit in other lanes, so sums round differently)
    check_balance(layer, shifted, idx, "softmax", k)
    layer.close()


def test_balance_no_tokens():
    layer = make_layer(8, 2)
    logits, idx = routing(0, 8, 2, 12)
    for off in (None, [0, 0, 0]):
        loss, counts, tokens, d = run_balance(layer, logits, idx, 0.01, off=off)
        assert float(loss) == 0 and not counts.any() and not tokens.any() and d.numel() == 0
    layer.close()


def test_balance_refusals():
    T, E, k = 16, 8, 2
    layer = make_layer(E, k)
    L = binding.load_library()
    logits, idx = routing(T, E, k, 13)
    c = torch.zeros(E, dtype=torch.int32, device="cuda")
    t = torch.zeros(1, dtype=torch.int32, device="cuda")
    f = torch.zeros(1, device="cuda")
    need = layer.balance_workspace(T)
    ws = torch.zeros(need + 16, dtype=torch.uint8, device="cuda")
    ok = dict(h=layer.h, logits=logits.data_ptr(), idx=idx.data_ptr(), T=T, off=None, n=1, mask=None,
              coef=0.1, counts=c.data_ptr(), tokens=t.data_ptr(), loss=f.data_ptr(),
              ws=ws.data_ptr(), nws=need)

    def call(**kw):
        a = {**ok, **kw}
        return L.strata_moe_balance(a["h"], a["logits"], a["idx"], a["T"], a["off"], a["n"],
                                    a["mask"], a["coef"], a["counts"], a["tokens"], a["loss"],
                                    a["ws"], a["nws"], None)

    assert call() == 0
    for kw in (dict(h=None), dict(logits=None), dict(idx=None), dict(T=-1), dict(T=(1 << 28) + 1),
               dict(n=0), dict(n=2), dict(counts=None), dict(tokens=None), dict(loss=None),
               dict(ws=None), dict(nws=need - 1), dict(ws=ws.data_ptr() + 8), dict(coef=math.nan),
               dict(coef=math.inf), dict(logits=logits.data_ptr() + 2),
               dict(idx=idx.data_ptr() + 1)):
        assert call(**kw) == int(BAD), kw
    d = torch.zeros(T, E, device="cuda")
    for kw in (dict(counts=c[:7]), dict(tokens=c), dict(dlogits=d[:, :7]), dict(mask=c),
               dict(logits=logits.cpu()), dict(dlogits=logits)):
        a = {**dict(logits=logits, coef=0.1, counts=c, tokens=t, dlogits=d), **kw}
        with pytest.raises(binding.StrataError):
            layer.balance_backward(**a)
    assert layer.balance_workspace(-1) == 0 and layer.balance_workspace(4, 0) == 0
    torch.cuda.synchronize()
    layer.close()


# ---------------------------------------------------------------- the router's gradient
def exact_dl(logits, idx, dw, dlogits, mode):
    """(dl, the sum of its terms' magnitudes) in 64 bits."""
    T, E = (dlogits if dlogits is not None else logits).shape
    dl = torch.zeros(T, E, dtype=torch.float64, device="cuda") if dlogits is None else \
        dlogits.double()
    mag = dl.abs()
    if dw is not None:
        sel = idx.long()
        l, g = logits.double().gather(1, sel), dw.double()
        if mode == "softmax":
            w = torch.softmax(l, 1)
            slope = w
        else:
            s = torch.sigmoid(l)
            w = s / s.sum(1, keepdim=True)
            slope = SCALE * w * torch.sigmoid(-l)
        dl = dl.scatter_add(1, sel, slope * (g - (w * g).sum(1, keepdim=True)))
        mag = mag.scatter_add(1, sel, slope * (g.abs() + (w * g.abs()).sum(1, keepdim=True)))
    return dl, mag


def run_route_backward(layer, x, logits, idx, dw, dlogits, want=("dW", "db", "dx"), stream=None):
    T, H, E = x.shape[0], layer.hidden, layer.n_experts
    out = dict(dW=torch.full((E, H), 7.0, device="cuda"), db=torch.full((E,), 7.0, device="cuda"),
               dx=torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda"))
    out = {n: t for n, t in out.items() if n in want}
    ws = torch.empty(layer.route_backward_workspace(T), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    layer.route_backward(x, logits, idx, dw, dlogits, out.get("dW"), out.get("db"), out.get("dx"),
                         ws, stream=stream)
    torch.cuda.synchronize()
    return out


def dx_rounding(dl, W):
    """The bound on what rounding dl and W to f16 changes in dl W."""
    a, w = dl.abs(), W.double().abs()
    return (a @ w) * 2.0 ** -10 * (1 + 2.0 ** -9) + \
        (a.amax(1, keepdim=True) * w.sum(0)) * 2.0 ** -25 + a.sum(1, keepdim=True) * 2.0 ** -33


def check_route_backward(layer, x, W, logits, idx, dw, dlogits, mode, **kw):
    T = x.shape[0]
    out = run_route_backward(layer, x, logits, idx, dw, dlogits, **kw)
    st = layer.status()
    assert int(st[0]) == 0, st
    dl, mag = exact_dl(logits, idx, dw, dlogits, mode)
    if "dW" in out:
        want = dl.t() @ x.double()
        tol = (dl.abs().t() @ x.double().abs()) * (3 * T / 8 + 64) * U + \
            (mag.t() @ x.double().abs()) * 32 * U
        err = (out["dW"].double() - want).abs()
        assert bool((err <= tol + 1e-38).all()), float((err / (tol + 1e-38)).max())
        # and, unlike the worst case above, close as a whole
        assert float(err.norm()) <= 2e-6 * float(want.norm()) + 1e-30
    if "db" in out:
        tol = dl.abs().sum(0) * (T / 8 + 64) * U + mag.sum(0) * 32 * U
        err = (out["db"].double() - dl.sum(0)).abs()
        assert bool((err <= tol + 1e-38).all()), float((err / (tol + 1e-38)).max())
    if "dx" in out:
        want = dl @ W.double()
        tol = dx_rounding(dl, W) + (mag @ W.double().abs()) * 32 * U + want.abs() * 2.0 ** -8
        err = (out["dx"].double() - want).abs()
        assert bool((err <= tol + 1e-38).all()), float((err / (tol + 1e-38)).max())
    return out


def router(E, H, seed):
    return torch.randn(E, H, device="cuda", generator=gen(seed)) / math.sqrt(H)


def acts(T, H, seed):
    return torch.randn(T, H, device="cuda", generator=gen(seed)).bfloat16()


SHAPES = [(1, 128, 1, 1), (1, 256, 8, 2), (2, 128, 64, 6), (31, 384, 60, 6), (33, 256, 100, 5),
          (64, 512, 16, 1), (129, 2048, 64, 6), (127, 256, 255, 10), (128, 128, 256, 8),
          (257, 640, 256, 32), (1000, 1152, 160, 4), (2048, 4096, 32, 8), (4099, 512, 129, 3),
          # few tokens (one launch) and just beyond, 16 and 32 h a block
          (40, 512, 255, 8), (41, 512, 256, 8), (19, 4096, 256, 10), (25, 4096, 256, 10),
          (160, 2048, 64, 6), (161, 2048, 64, 6), (1280, 256, 7, 2), (1281, 256, 8, 1)]


@pytest.mark.parametrize("mode", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,H,E,k", SHAPES)
def test_route_backward(T, H, E, k, mode):
    W, x = router(E, H, 21), acts(T, H, 22)
    layer = make_layer(E, k, mode, H, W)
    logits, idx = routing(T, E, k, 23)
    dw = torch.randn(T, k, device="cuda", generator=gen(24))
    dlg = torch.randn(T, E, device="cuda", generator=gen(25)) * 0.05
    full = check_route_backward(layer, x, W, logits, idx, dw, dlg, mode)
    again = run_route_backward(layer, x, logits, idx, dw, dlg)
    for n in full:
        assert torch.equal(full[n], again[n]), n
    check_route_backward(layer, x, W, logits, idx, dw, None, mode)
    check_route_backward(layer, x, W, None, None, None, dlg, mode)
    for n in full:   # each output alone is the same
        assert torch.equal(run_route_backward(layer, x, logits, idx, dw, dlg, (n,))[n], full[n]), n
    layer.close()


# beside the borders between the forms: one launch or three; of the three, a run
# for each tile of h, several, or runs that cut tiles anywhere
@pytest.mark.parametrize("T,H,E,k", [
    (60, 256, 256, 8), (61, 256, 256, 8), (77, 1024, 128, 6), (78, 1024, 128, 6), (394, 256, 8, 3),
    (395, 256, 8, 3), (485, 128, 3, 1), (486, 128, 3, 1), (59, 4096, 64, 6), (60, 4096, 64, 6),
    (22, 7168, 64, 4), (23, 7168, 64, 4), (1, 16384, 16, 2), (65, 16384, 250, 4), (3, 18944, 40, 2),
    (600, 19200, 70, 3), (511, 2048, 256, 8), (1023, 4096, 128, 8), (2049, 640, 200, 8),
    (64, 384, 256, 1), (8190, 896, 50, 2)])
def test_route_backward_beside_the_forms_borders(T, H, E, k):
    W, x = router(E, H, 171), acts(T, H, 172)
    layer = make_layer(E, k, "softmax", H, W)
    logits, idx = routing(T, E, k, 173)
    dw = torch.randn(T, k, device="cuda", generator=gen(174))
    dlg = torch.randn(T, E, device="cuda", generator=gen(175)) * 0.05
    full = check_route_backward(layer, x, W, logits, idx, dw, dlg, "softmax")
    for n in full:
        assert torch.equal(run_route_backward(layer, x, logits, idx, dw, dlg, (n,))[n], full[n]), n
    layer.close()


def test_route_backward_ranges_of_values():
    # gradients of every size (1e-12 .. 1e3 in one batch) keep their relative accuracy
    T, H, E, k = 200, 256, 64, 4
    W, x = router(E, H, 26), acts(T, H, 27)
    layer = make_layer(E, k, H=H, W=W)
    dlg = torch.randn(T, E, device="cuda", generator=gen(28)) * \
        10 ** (torch.rand(1, E, device="cuda", generator=gen(29)) * 15 - 12)
    check_route_backward(layer, x, W, None, None, None, dlg.contiguous(), "softmax")
    layer.close()


def test_route_backward_sizes_of_router_weights():
    # weights down to where f16 steps are absolute, and up to the limit
    T, H, E = 130, 256, 32
    x = acts(T, H, 42)
    dlg = torch.randn(T, E, device="cuda", generator=gen(43))
    for scale in (1e-6, 1e-3, 30.0):
        W = router(E, H, 44) * scale
        layer = make_layer(E, 2, H=H, W=W)
        check_route_backward(layer, x, W, None, None, None, dlg, "softmax")
        layer.close()
    W = router(E, H, 44)
    W[3, 7] = 256.0
    layer = make_layer(E, 2, H=H, W=W)
    run_route_backward(layer, x, None, None, None, dlg)
    st, bits = layer.status()
    assert st == binding.Status.RANGE and bits == 16
    out = run_route_backward(layer, x, None, None, None, dlg, ("dW", "db"))   # W is not read
    assert int(layer.status()[0]) == 0 and not bool(out["dW"].isnan().any())
    layer.close()


def test_route_backward_same_expert_twice_extreme_logits():
    T, H, E, k = 40, 128, 8, 3
    W, x = router(E, H, 31), acts(T, H, 32)
    for mode in ("softmax", "sigmoid"):
        layer = make_layer(E, k, mode, H, W)
        logits, idx = routing(T, E, k, 33)
        idx[:, 2] = idx[:, 0]
        dw = torch.randn(T, k, device="cuda", generator=gen(34))
        check_route_backward(layer, x, W, logits, idx, dw, None, mode)
        # selected logits at -inf (fewer experts left than top_k), and all of them
        logits[5].scatter_(0, idx[5, 1:2].long(), -math.inf)
        check_route_backward(layer, x, W, logits, idx, dw, None, mode)
        logits[6] = -math.inf
        out = run_route_backward(layer, x, logits, idx, dw, None)
        assert all(not bool(t.isnan().any()) for t in out.values())
        assert not out["dx"][6].any()
        layer.close()


def test_route_backward_bad_ids():
    T, H, E, k = 20, 128, 8, 2
    W, x = router(E, H, 35), acts(T, H, 36)
    layer = make_layer(E, k, H=H, W=W)
    logits, idx = routing(T, E, k, 37)
    dw = torch.randn(T, k, device="cuda", generator=gen(38))
    zeroed = dw.clone()
    zeroed[4] = 0
    want = run_route_backward(layer, x, logits, idx, zeroed, None)
    idx[4, 1] = E
    got = run_route_backward(layer, x, logits, idx, dw, None)
    st, bits = layer.status()
    assert st == binding.Status.DEVICE_STATUS and bits == 2
    for n in want:
        assert torch.equal(want[n], got[n])
    layer.close()


def test_route_backward_no_tokens_and_refusals():
    T, H, E, k = 8, 128, 8, 2
    W, x = router(E, H, 39), acts(T, H, 40)
    layer = make_layer(E, k, H=H, W=W)
    empty = torch.empty(0, H, dtype=torch.bfloat16, device="cuda")
    out = run_route_backward(layer, empty, None, None, None, None)
    assert not out["dW"].any() and not out["db"].any()
    L = binding.load_library()
    logits, idx = routing(T, E, k, 41)
    dw = torch.zeros(T, k, device="cuda")
    dlg = torch.zeros(T, E, device="cuda")
    dW, db, dx = torch.zeros(E, H, device="cuda"), torch.zeros(E, device="cuda"), torch.zeros_like(x)
    need = layer.route_backward_workspace(T)
    ws = torch.zeros(need + 256, dtype=torch.uint8, device="cuda")
    ok = dict(h=layer.h, x=x.data_ptr(), T=T, logits=logits.data_ptr(), idx=idx.data_ptr(),
              dw=dw.data_ptr(), dlg=dlg.data_ptr(), dW=dW.data_ptr(), db=db.data_ptr(),
              dx=dx.data_ptr(), ws=ws.data_ptr(), n=need)

    def call(**kw):
        a = {**ok, **kw}
        return L.strata_moe_route_backward(a["h"], a["x"], a["T"], a["logits"], a["idx"], a["dw"],
                                           a["dlg"], a["dW"], a["db"], a["dx"], a["ws"], a["n"],
                                           None)

    assert call() == 0
    for kw in (dict(h=None), dict(x=None), dict(T=-1), dict(T=(1 << 28) + 1), dict(logits=None),
               dict(idx=None), dict(dw=None, dlg=None), dict(dW=None, db=None, dx=None),
               dict(ws=None), dict(n=need - 1), dict(ws=ws.data_ptr() + 16),
               dict(x=x.data_ptr() + 2), dict(dx=dx.data_ptr() + 2), dict(dW=dW.data_ptr() + 4)):
        assert call(**kw) == int(BAD), kw
    with pytest.raises(binding.StrataError):   # another 16-bit type
        layer.route_backward(x.half(), logits, idx, dw, dlg, dW, db, dx, ws)
    with pytest.raises(binding.StrataError):   # not on the device
        layer.route_backward(x.cpu(), logits, idx, dw, dlg, dW, db, dx, ws)
    bare = make_layer(E, k, H=H)   # no router set: dx cannot be had, the others can
    assert call(h=bare.h) == int(BAD)
    assert call(h=bare.h, dx=None) == 0
    torch.cuda.synchronize()
    bare.close()
    layer.close()


@pytest.mark.parametrize("mode", ["softmax", "sigmoid"])
def test_gradients_against_differences(mode):
    # f(W, x) = sum dw w(W x) + balance loss, routed experts and counts held;
    # central differences in 64 bits, step 1e-4: off by about 1e-8
    T, H, E, k, coef = 12, 128, 8, 3, 0.5
    W, x = router(E, H, 51), acts(T, H, 52)
    layer = make_layer(E, k, mode, H, W)
    logits = torch.empty(T, E, device="cuda")
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    layer.route(x, logits, idx, w)
    dw = torch.randn(T, k, device="cuda", generator=gen(53))
    _, counts, tokens, dlg = run_balance(layer, logits, idx, coef)
    out = run_route_backward(layer, x, logits, idx, dw, dlg)
    f = counts[0].double() * E / (k * T)

    def value(Wd, xd):
        l = xd @ Wd.t()
        p, _ = probs(l, mode)
        s = l.gather(1, idx.long())
        if mode == "softmax":
            ww = torch.softmax(s, 1)
        else:
            ww = torch.sigmoid(s)
            ww = SCALE * ww / ww.sum(1, keepdim=True)
        return float((ww * dw.double()).sum() + coef * (f * p.mean(0)).sum())

    d = 1e-4
    for e, c in ((0, 0), (3, 77), (7, 127)):
        step = torch.zeros(E, H, dtype=torch.float64, device="cuda")
        step[e, c] = d
        num = (value(W.double() + step, x.double()) - value(W.double() - step, x.double())) / (2 * d)
        assert abs(num - float(out["dW"][e, c])) < 2e-5
    dl, _ = exact_dl(logits, idx, dw, dlg, mode)
    room = dx_rounding(dl, W)
    for t, c in ((0, 5), (11, 100)):
        step = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        step[t, c] = d
        num = (value(W.double(), x.double() + step) - value(W.double(), x.double() - step)) / (2 * d)
        assert abs(num - float(out["dx"][t, c])) < 2e-5 + abs(num) * 2.0 ** -8 + float(room[t, c])
    layer.close()


def test_streams_and_graphs():
    T, H, E, k = 300, 512, 64, 6
    W = router(E, H, 61)
    layer = make_layer(E, k, "softmax", H, W)
    off, coef = [0, 100, 300], 0.1
    seq = torch.tensor(off, dtype=torch.int32, device="cuda")

    def inputs(seed):
        logits, idx = routing(T, E, k, seed)
        return (acts(T, H, seed + 1), logits, idx,
                torch.randn(T, k, device="cuda", generator=gen(seed + 2)))

    def eager(x, logits, idx, dw, stream=None):
        loss, counts, tokens, d = run_balance(layer, logits, idx, coef, off=off, stream=stream)
        out = run_route_backward(layer, x, logits, idx, dw, d, stream=stream)
        return [loss, counts, tokens, d, out["dW"], out["db"], out["dx"]]

    side = torch.cuda.Stream()
    first = inputs(70)
    for a, b in zip(eager(*first), eager(*first, stream=side)):
        assert torch.equal(a, b)
    graphs = []
    for seed in (80, 90):
        src = inputs(seed)
        x, logits, idx, dw = src
        out = [torch.empty(1, device="cuda"), torch.empty(2, E, dtype=torch.int32, device="cuda"),
               torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty(T, E, device="cuda"),
               torch.empty(E, H, device="cuda"), torch.empty(E, device="cuda"),
               torch.empty(T, H, dtype=torch.bfloat16, device="cuda")]
        ws1 = torch.empty(layer.balance_workspace(T, 2), dtype=torch.uint8, device="cuda")
        ws2 = torch.empty(layer.route_backward_workspace(T), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.balance(logits, idx, coef, out[1], out[2], out[0], ws1, seq)
            layer.balance_backward(logits, coef, out[1], out[2], out[3], None, seq)
            layer.route_backward(x, logits, idx, dw, out[3], out[4], out[5], out[6], ws2)
        graphs.append((g, src, out, (ws1, ws2), torch.cuda.Stream()))
    for r in range(3):
        for i, (g, src, out, _, _) in enumerate(graphs):
            for dst, new in zip(src, inputs(100 + 10 * (2 * r + i))):
                dst.copy_(new)
        torch.cuda.synchronize()
        for g, _, _, _, s in graphs:   # at once, on two streams
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for g, src, out, _, _ in graphs:
            for a, b in zip(eager(*src), out):
                assert torch.equal(a, b)
    layer.close()


@pytest.mark.parametrize("T,H,E,k", [(2700, 256, 40, 4), (1500, 2048, 120, 6), (2300, 1024, 250, 8)])
def test_route_backward_calls_in_a_row_share_a_workspace(T, H, E, k):
    # in stream order and without a wait between them, every call writes over what
    # the one before it read
    W = router(E, H, 121)
    layer = make_layer(E, k, "softmax", H, W)
    cases, want = [], []
    for seed in (122, 132, 142):
        logits, idx = routing(T, E, k, seed)
        cases.append((acts(T, H, seed + 1), logits, idx,
                      torch.randn(T, k, device="cuda", generator=gen(seed + 2)),
                      torch.randn(T, E, device="cuda", generator=gen(seed + 3)) * 10.0 ** (seed - 132)))
        want.append(run_route_backward(layer, *cases[-1]))
    ws = torch.empty(layer.route_backward_workspace(T), dtype=torch.uint8, device="cuda")
    got = []
    for i in range(24):
        out = (torch.empty(E, H, device="cuda"), torch.empty(E, device="cuda"),
               torch.empty(T, H, dtype=torch.bfloat16, device="cuda"))
        layer.route_backward(*cases[i % 3], *out, ws)
        got.append(out)
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        for n, t in zip(("dW", "db", "dx"), out):
            assert torch.equal(t, want[i % 3][n]), (i, n)
    assert int(layer.status()[0]) == 0
    layer.close()


# rows of fewer experts than one 16-byte access, past the few tokens of one launch
@pytest.mark.parametrize("T,H,E,k", [(10300, 128, 1, 1), (2600, 256, 3, 2), (1300, 384, 5, 5),
                                     (1290, 512, 7, 1)])
def test_route_backward_few_experts(T, H, E, k):
    W, x = router(E, H, 151), acts(T, H, 152)
    layer = make_layer(E, k, "sigmoid", H, W)
    logits, idx = routing(T, E, k, 153)
    dw = torch.randn(T, k, device="cuda", generator=gen(154))
    dlg = torch.randn(T, E, device="cuda", generator=gen(155)) * 0.05
    check_route_backward(layer, x, W, logits, idx, dw, dlg, "sigmoid")
    layer.close()


def test_offsets_past_32_bits():
    # more than 2^31 logits (2^33 bytes); what is checked in detail lies behind them
    T, H, E, k, n, coef = 2 ** 23 + 1003, 128, 256, 2, 1000, 0.5
    W = router(E, H, 161)
    layer = make_layer(E, k, "softmax", H, W)
    logits = torch.randn(T, E, device="cuda", generator=gen(162))
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    idx = torch.stack((t % 251, (t + 3) % 256), 1).contiguous()
    counts, tokens = (torch.empty(m, dtype=torch.int32, device="cuda") for m in (E, 1))
    loss, d = torch.empty(1, device="cuda"), torch.empty(T, E, device="cuda")
    ws = torch.empty(layer.balance_workspace(T), dtype=torch.uint8, device="cuda")
    layer.balance(logits, idx, coef, counts, tokens, loss, ws)
    layer.balance_backward(logits, coef, counts, tokens, d)
    assert int(tokens) == T
    assert torch.equal(counts.long(), torch.bincount(idx.view(-1).long(), minlength=E))
    f = counts.double() * E / (k * T)
    P = sum(torch.softmax(c.double(), 1).sum(0) for c in logits.split(2 ** 18)) / T
    # (a warp's own share: up to 1800 rows one by one)
    want = float(coef * (f * P).sum())
    assert abs(float(loss) - want) <= (1800 + 128) * U * want
    p = torch.softmax(logits[-n:].double(), 1)
    dot = (p * f).sum(1, keepdim=True)
    err = (d[-n:].double() - coef / T * p * (f - dot)).abs()
    assert bool((err <= coef / T * p * (f + dot) * 128 * U + 2.0 ** -140).all())

    # the router: only the last n tokens have gradients, so dW and db are sums
    # over those n, and dx is zero in front of them
    d[:-n] = 0
    d[-n:] = torch.randn(n, E, device="cuda", generator=gen(163)) * 0.1
    dw = torch.zeros(T, k, device="cuda")
    dw[-n:] = torch.randn(n, k, device="cuda", generator=gen(164))
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[-n:] = acts(n, H, 165)
    out = run_route_backward(layer, x, logits, idx, dw, d)
    assert int(layer.status()[0]) == 0
    dl, mag = exact_dl(logits[-n:], idx[-n:], dw[-n:], d[-n:], "softmax")
    xd = x[-n:].double()
    for got, want, tol in (
            (out["dW"], dl.t() @ xd, (dl.abs().t() @ xd.abs()) * (3 * n / 8 + 64) * U + (mag.t() @ xd.abs()) * 32 * U),
            (out["db"], dl.sum(0), dl.abs().sum(0) * (n / 8 + 64) * U + mag.sum(0) * 32 * U),
            (out["dx"][-n:], dl @ W.double(), dx_rounding(dl, W) + (mag @ W.double().abs()) * 32 * U +
             (dl @ W.double()).abs() * 2.0 ** -8)):
        assert bool(((got.double() - want).abs() <= tol + 1e-38).all())
    assert not bool(out["dx"][:-n].any())
    layer.close()


@pytest.mark.parametrize("mode", ["softmax", "sigmoid"])
def test_one_training_step_of_a_router(mode):
    """norm -> route -> balance -> their gradients, chained as a training loop
    chains them, against one 64-bit autograd graph."""
    T, H, E, k, coef = 96, 256, 16, 4, 0.3
    W, bias = router(E, H, 111) * 2, torch.randn(E, device="cuda", generator=gen(112)) * 0.1
    layer = make_layer(E, k, mode, H, W, bias)
    a, r = acts(T, H, 113), acts(T, H, 114)
    gain = 1 + 0.2 * torch.randn(H, device="cuda", generator=gen(115))
    dw = torch.randn(T, k, device="cuda", generator=gen(116))
    s, x = torch.empty_like(a), torch.empty_like(a)
    binding.strata_rmsnorm(a, r, gain, 1e-6, s, x)
    logits = torch.empty(T, E, device="cuda")
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    layer.route(x, logits, idx, w)
    loss, counts, tokens, dlg = run_balance(layer, logits, idx, coef)
    out = run_route_backward(layer, x, logits, idx, dw, dlg)
    ds, dgain = torch.empty_like(s), torch.empty(H, device="cuda")
    ws = torch.empty(binding.strata_rmsnorm_backward_workspace(T, H), dtype=torch.uint8, device="cuda")
    binding.strata_rmsnorm_backward(s, gain, 1e-6, out["dx"], None, ds, dgain, ws)
    assert int(layer.status()[0]) == 0

    leaf = [t.double().requires_grad_(True) for t in (s, gain, W, bias)]
    sd, gd, Wd, bd = leaf
    xn = sd / (sd.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * gd
    xr = xn + (x.double() - xn).detach()          # the rounded activations that the router saw
    l = xr @ Wd.t() + bd
    if mode == "softmax":
        p, wt = torch.softmax(l, 1), torch.softmax(l.gather(1, idx.long()), 1)
    else:
        sg = torch.sigmoid(l)
        p = sg / sg.sum(1, keepdim=True)
        wt = sg.gather(1, idx.long())
        wt = SCALE * wt / wt.sum(1, keepdim=True)
    f = counts[0].double() * E / (k * T)
    bal = coef * (f * p.mean(0)).sum()
    assert abs(float(bal.detach()) - float(loss)) < 1e-5 * float(loss)
    grads = torch.autograd.grad((wt * dw.double()).sum() + bal, leaf)
    # dx was rounded to bf16 (2^-8) on its way into the norm's gradient, ds and
    # x again: as a whole within 2^-7
    for got, want, tol in zip((ds, dgain, out["dW"], out["db"]), grads, (2.0 ** -7, 2.0 ** -7, 1e-5, 1e-5)):
        assert float((got.double() - want).norm()) <= tol * float(want.norm())
    layer.close()


# Consecutive tokens of a warp scatter to the same experts from other lanes, and the
# last one's places become those of db's sums: without dx nothing else orders them.
@pytest.mark.parametrize("T,E,k", [(2700, 64, 8), (2500, 128, 12), (1300, 256, 32), (9000, 8, 8)])
@pytest.mark.parametrize("want", [("db",), ("dW", "db")])
def test_route_backward_tokens_in_a_row_select_the_same_experts(T, E, k, want):
    H = 256
    x = acts(T, H, 181)
    layer = make_layer(E, k, H=H)
    logits, _ = routing(T, E, k, 182)
    turn = torch.arange(T, device="cuda")[:, None] + torch.arange(k, device="cuda")
    idx = (turn % k).int().contiguous()
    dw = torch.randn(T, k, device="cuda", generator=gen(183))
    for i in range(3):
        check_route_backward(layer, x, None, logits, idx, dw, None, "softmax", want=want)
        idx = (E - 1 - idx).contiguous()
    layer.close()


# Decreasing offsets: nothing counts, whatever an earlier call left in the workspace
@pytest.mark.parametrize("T,off", [(100, [0, 50, 40, 100]), (100, [0, 1 << 30, 3]), (700, [0, 300, 290, 310, 700]),
                                   (700, [0, 200, 320, 100, 150, 700]), (5000, [4000, 3000, 5000]),
                                   (300, [300, 0]), (9000, list(range(2000, 0, -1)) + [9000])])
def test_balance_decreasing_offsets_count_nothing(T, off):
    E, k = 64, 4
    layer = make_layer(E, k)
    logits, idx = routing(T, E, k, 191)
    n = len(off) - 1
    seq = torch.tensor(off, dtype=torch.int32, device="cuda")
    ws = torch.empty(layer.balance_workspace(T, n), dtype=torch.uint8, device="cuda")
    ordered = torch.tensor(sorted(min(o, T) for o in off), dtype=torch.int32, device="cuda")
    for before in (None, ordered):
        counts = torch.full((n, E), -7, dtype=torch.int32, device="cuda")
        tokens, loss = torch.full((n,), -7, dtype=torch.int32, device="cuda"), torch.full((1,), 7.0, device="cuda")
        d = torch.full((T, E), 7.0, device="cuda")
        if before is None:
            ws.fill_(0xFF)
        else:
            layer.balance(logits, idx, 0.5, counts, tokens, loss, ws, before)
            assert int(layer.status()[0]) == 0
        layer.balance(logits, idx, 0.5, counts, tokens, loss, ws, seq)
        st, bits = layer.status()
        assert st == binding.Status.DEVICE_STATUS and bits == 8
        layer.balance_backward(logits, 0.5, counts, tokens, d, None, seq)
        assert float(loss) == 0 and not counts.any() and not tokens.any() and not d.any()
    layer.close()


# Offsets that only leave the tokens are clamped
def test_balance_offsets_outside_are_clamped():
    T, E, k = 700, 64, 4
    layer = make_layer(E, k)
    logits, idx = routing(T, E, k, 192)
    for off, inside in (([-9, 100, 400, 700], [0, 100, 400, 700]), ([0, 333, 1 << 30], [0, 333, 700]),
                        ([-5, -2, 20, 800, 900], [0, 0, 20, 700, 700])):
        want = run_balance(layer, logits, idx, 0.5, off=inside)
        assert int(layer.status()[0]) == 0
        got = run_balance(layer, logits, idx, 0.5, off=off)
        st, bits = layer.status()
        assert st == binding.Status.DEVICE_STATUS and bits == 8
        for a, b in zip(want, got):
            assert torch.equal(a, b)
    layer.close()


# A gradient that is not finite shows wherever it reaches, and nowhere else: zeros in
# x and W do not hide it
@pytest.mark.parametrize("T,E", [(20, 64), (300, 40), (300, 100), (700, 256)])   # one launch, three
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_route_backward_of_a_gradient_that_is_not_finite(T, E, value):
    H, t, e = 256, 17, 5
    W, x = router(E, H, 201), acts(T, H, 202)
    W[:, ::3] = 0
    x[:, ::3] = 0
    layer = make_layer(E, 2, H=H, W=W)
    d = torch.randn(T, E, device="cuda", generator=gen(203))
    d[t, e] = value
    out = run_route_backward(layer, x, None, None, None, d)
    assert int(layer.status()[0]) == 0
    lost = {n: ~v.isfinite() for n, v in out.items()}
    assert bool(lost["dx"][t].all()) and int(lost["dx"].sum()) == H
    assert bool(lost["dW"][e].all()) and int(lost["dW"].sum()) == H
    assert bool(lost["db"][e]) and int(lost["db"].sum()) == 1
    layer.close()
