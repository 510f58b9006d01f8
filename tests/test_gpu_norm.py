"""RMS norm with residual and 8-bit output, and its gradient, against the
formulas in 64 bits.

Tolerances.  An output rounded to a type with step eps is off by at most
eps / 2 relative (f16 below its normal range: 2^-25 absolute).  Before that,
everything is fp32 (u = 2^-24): the sum has relative error u; the sum of H <=
16384 squares is taken in chains of at most 16 and a tree of 10, so the
reciprocal length is within 32 u, and y within 40 u relative -- 64 u is used.
dx = i gy - h i^3 mean(gy h) + ds is a difference: its error is 64 u times the
sum of the magnitudes of its terms (with mean |gy h|).  dweight sums T terms in
chains of at most T / 296 + 1 rows, 37 and 8 partial sums.
"""
import pytest

torch = pytest.importorskip("torch")

from quantized_routed_expert_04_b200 import binding  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}
EPS = 1e-6


def rows(T, H, dt, seed, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(T, H, device="cuda", generator=g) * scale).to(DT[dt])


def weight(H, seed=9):
    g = torch.Generator("cuda").manual_seed(seed)
    return 1 + 0.3 * torch.randn(H, device="cuda", generator=g)


def exact(x, r, w):
    s = x.double() + (0 if r is None else r.double())
    return s, s / (s.pow(2).mean(1, keepdim=True) + EPS).sqrt() * w.double()


def close(got, want, tol, what):
    bad = ((got.double() - want).abs() > tol) | (got.double().isnan() != want.isnan())
    assert not bool(bad.any()), "%s: %d of %d beyond the bound, worst ratio %.3g" % (
        what, int(bad.sum()), bad.numel(),
        float(((got.double() - want).abs() / tol.clamp(min=1e-300)).nan_to_num().max()))


def check_q8(q, sc, y, group):
    T, H = y.shape
    n = -(-H // group)
    pad = torch.nn.functional.pad(y, (0, n * group - H)).view(T, n, group)
    want = (pad.abs().amax(2) / 448).clamp(min=2.0 ** -126)
    close(sc, want, want * 65 * U, "scales")
    v = (pad / sc.double()[:, :, None]).view(T, n * group)[:, :H]
    # half a step: 2^-4 relative, 2^-10 below the normal range (steps of 2^-9)
    close(q.view(torch.float8_e4m3fn).float(), v, (v.abs() * (2.0 ** -4 + 66 * U)).clamp(min=2.0 ** -10 + 2.0 ** -20),
          "e4m3")


def run_forward(x, r, w, group=0, **kw):
    T, H = x.shape
    ro = torch.empty_like(x) if r is not None else None
    out = torch.empty_like(x)
    q = sc = None
    if group:
        q = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda")
        sc = torch.empty(T, -(-H // group), device="cuda")
    binding.strata_rmsnorm(x, r, w, EPS, ro, out, q, sc, group, **kw)
    return ro, out, q, sc


SHAPES = [(1, 1), (1, 7), (3, 8), (5, 100), (4, 256), (9, 257), (2, 512), (7, 1000), (3, 1024),
          (1, 2048), (5, 2047), (33, 4096), (2, 4104), (3, 8192), (2, 11000), (2, 16383),
          (2, 16384)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_forward(T, H, dt, residual):
    x, w = rows(T, H, dt, 1), weight(H)
    r = rows(T, H, dt, 2, 3.0) if residual else None
    s, y = exact(x, r, w)
    for group in (0, 32, 64, 128, H):
        ro, out, q, sc = run_forward(x, r, w, group)
        close(out, y, y.abs() * (HALF[dt] + 64 * U) + TINY[dt], "out")
        if residual:
            close(ro, s, s.abs() * (HALF[dt] + U) + TINY[dt], "sum")
        if group:
            check_q8(q, sc, y, group)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_forward_strides_offsets_and_in_place(dt):
    T, H = 6, 640
    w = weight(H)
    for off, ld in ((0, 648), (1, 641), (8, 1280), (3, 700)):
        big, big2 = rows(T, ld + 16, dt, 3), rows(T, ld + 16, dt, 4)
        x, r = big[:, off:off + H], big2[:, off:off + H]
        s, y = exact(x, r, w)
        keep, keep2 = big.clone(), big2.clone()
        # the sum over the residual, y over x, both in place
        binding.strata_rmsnorm(x, r, w, EPS, r, x)
        close(x, y, y.abs() * (HALF[dt] + 64 * U), "out")
        close(r, s, s.abs() * (HALF[dt] + U), "sum")
        for a, b in ((big, keep), (big2, keep2)):   # nothing outside the rows
            assert torch.equal(a[:, :off], b[:, :off]) and torch.equal(a[:, off + H:], b[:, off + H:])


def test_forward_sees_the_unrounded_sum():
    # residual 256, x 0.5: bf16 keeps 256, the norm sees 256.5
    x = torch.full((1, 64), 0.5, dtype=torch.bfloat16, device="cuda")
    x[0, 0] = 0.0
    r = torch.full((1, 64), 256.0, dtype=torch.bfloat16, device="cuda")
    ro = torch.empty_like(x)
    out32 = torch.empty(1, 64, device="cuda")
    binding.strata_rmsnorm(x, r, torch.ones(64, device="cuda"), 0.0, ro, torch.empty_like(x))
    assert bool((ro == 256).all())
    q = torch.empty(1, 64, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(1, 1, device="cuda")
    binding.strata_rmsnorm(x, r, torch.ones(64, device="cuda"), 0.0, None, None, q, sc, 64)
    s = x.double() + r.double()
    y = s / s.pow(2).mean().sqrt()
    assert abs(float(sc[0, 0]) * 448 - float(y.max())) < 1e-6
    assert out32.numel() == 64


@pytest.mark.parametrize("H,group", [(256, 32), (250, 32), (640, 128), (640, 640)])
def test_special_values(H, group):
    x = rows(5, H, "f32", 5)
    x[1] = 0                       # zero row: y = 0, scale 2^-126
    x[2, 3] = float("nan")         # the row's length is NaN: all of it is
    x[3, 4] = float("inf")         # inf / inf: NaN there, 0 elsewhere
    x[4] *= 1e-30                  # far below eps
    w = torch.ones(H, device="cuda")
    _, out, q, sc = run_forward(x, None, w, group)
    f = q.float()
    assert bool((out[1] == 0).all()) and bool((f[1] == 0).all())
    assert bool((sc[1] == 2.0 ** -126).all())
    assert bool(out[2].isnan().all()) and bool(f[2].isnan().all()) and bool(sc[2].isnan().all())
    assert bool(out[3, 4].isnan()) and int(out[3].isnan().sum()) == 1
    g = min(group, H)
    assert bool(f[3, :g].isnan().all())       # its group's scale is NaN
    if g < H:
        assert bool((f[3, g:] == 0).all())
    assert not bool(out[4].isnan().any()) and float(out[4].abs().max()) < 1e-25
    assert not bool(out[0].isnan().any())


def test_huge_row_offsets():
    # in place, over more than 2^31 elements (and 2^32 bytes)
    H, T = 8192, 262145 + 8
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[-1] = rows(1, H, "bf16", 6)[0]
    x[262144] = rows(1, H, "bf16", 7)[0]
    last, mid, w = x[-1:].clone(), x[262144:262145].clone(), weight(H)
    binding.strata_rmsnorm(x, None, w, EPS, None, x)
    for got, src in ((x[-1:], last), (x[262144:262145], mid)):
        _, y = exact(src, None, w)
        close(got, y, y.abs() * (HALF["bf16"] + 64 * U), "out")
    assert bool((x[-2] == 0).all())


# ---------------------------------------------------------------- gradient
def run_backward(h, w, dy, ds, want_dw=True, **kw):
    dx = torch.empty_like(h)
    dw = torch.empty(h.shape[1], device="cuda") if want_dw else None
    ws = torch.empty(binding.strata_rmsnorm_backward_workspace(*h.shape), dtype=torch.uint8,
                     device="cuda") if want_dw else None
    binding.strata_rmsnorm_backward(h, w, EPS, dy, ds, dx, dw, ws, **kw)
    return dx, dw


def exact_backward(h, w, dy, ds):
    """(dx, its error scale, dweight, its sum of magnitudes) in 64 bits."""
    h, w, dy = h.double(), w.double(), dy.double()
    i = 1 / (h.pow(2).mean(1, keepdim=True) + EPS).sqrt()
    gy = dy * w
    dx = i * gy - h * i ** 3 * (gy * h).mean(1, keepdim=True)
    mag = i * gy.abs() + h.abs() * i ** 3 * (gy * h).abs().mean(1, keepdim=True)
    if ds is not None:
        dx, mag = dx + ds.double(), mag + ds.double().abs()
    return dx, mag, (dy * h * i).sum(0), (dy * h * i).abs().sum(0)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 9), (2, 64), (3, 513), (300, 512), (1, 1024),
                                 (65, 1000), (700, 2048), (5, 4096), (299, 4097), (4, 8192),
                                 (3, 9000), (600, 16384), (2, 16383)])
@pytest.mark.parametrize("direct", [False, True])
def test_backward(T, H, dt, direct):
    h, dy, w = rows(T, H, dt, 11, 2.0), rows(T, H, dt, 12), weight(H)
    ds = rows(T, H, dt, 13) if direct else None
    dx, dw = run_backward(h, w, dy, ds)
    ex, mag, ew, magw = exact_backward(h, w, dy, ds)
    close(dx, ex, ex.abs() * HALF[dt] + mag * 64 * U + TINY[dt], "dx")
    chain = T / 296 + 1 + 37 + 8 + 40
    close(dw, ew, magw * chain * U + 1e-37, "dweight")
    again = run_backward(h, w, dy, ds)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    only, none = run_backward(h, w, dy, ds, want_dw=False)
    assert torch.equal(only, dx) and none is None


def test_backward_against_differences():
    # (f(h + d) - f(h - d)) / 2 of f = sum(dy * norm(h)) in 64 bits; the
    # central difference is off by d^2 / 6 f''' ~ 1e-9 here
    h, dy, w = rows(2, 24, "f32", 14), rows(2, 24, "f32", 15), weight(24)
    dx, dw = run_backward(h, w, dy, None)
    d = 1e-4

    def f(hh, ww):
        return float((exact(hh, None, ww)[1] * dy.double()).sum())

    for c in (0, 7, 23):
        for r in (0, 1):
            e = torch.zeros(2, 24, device="cuda", dtype=torch.float64)
            e[r, c] = d
            num = (f(h.double() + e, w) - f(h.double() - e, w)) / (2 * d)
            assert abs(num - float(dx[r, c])) < 1e-5
        e = torch.zeros(24, device="cuda", dtype=torch.float64)
        e[c] = d
        num = (f(h, w.double() + e) - f(h, w.double() - e)) / (2 * d)
        assert abs(num - float(dw[c])) < 1e-5


def test_backward_in_place_and_strides():
    T, H = 9, 1280
    w = weight(H)
    big = [rows(T, 1400, "bf16", 20 + i) for i in range(3)]
    h, dy, ds = (b[:, 5:5 + H] for b in big)
    want, _ = run_backward(h.contiguous(), w, dy.contiguous(), ds.contiguous())
    for target in (ds, dy, h):
        src = [t.clone() for t in (h, dy, ds)]
        dw = torch.empty(H, device="cuda")
        ws = torch.empty(binding.strata_rmsnorm_backward_workspace(T, H), dtype=torch.uint8,
                         device="cuda")
        binding.strata_rmsnorm_backward(h, w, EPS, dy, ds, target, dw, ws)
        # the unaligned rows take another mapping of elements to threads, so
        # the row sums differ in their last bits
        assert float((target.double() - want.double()).abs().max()) <= 2.0 ** -6
        for t, s in zip((h, dy, ds), src):
            t.copy_(s)


def test_no_rows_zeroes_the_weight_gradient():
    H = 100
    h = torch.empty(0, H, device="cuda")
    dw = torch.full((H,), 7.0, device="cuda")
    ws = torch.empty(binding.strata_rmsnorm_backward_workspace(0, H), dtype=torch.uint8,
                     device="cuda")
    binding.strata_rmsnorm_backward(h, torch.ones(H, device="cuda"), EPS, h, None, h, dw, ws)
    assert bool((dw == 0).all())
    binding.strata_rmsnorm(h, None, torch.ones(H, device="cuda"), EPS, None, h)


def test_streams_and_graphs():
    T, H = 130, 2048
    w = weight(H)
    x, r, dy = rows(T, H, "bf16", 31), rows(T, H, "bf16", 32), rows(T, H, "bf16", 33)
    want = run_forward(x, r, w, 128)
    bwant = run_backward(want[0], w, dy, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run_forward(x, r, w, 128, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # two graphs, a workspace each, replayed at once on two streams with new
    # inputs in the same buffers
    graphs = []
    for seed in (41, 42):
        bufs = dict(x=x.clone(), r=r.clone(), ro=torch.empty_like(x), out=torch.empty_like(x),
                    dx=torch.empty_like(x), dw=torch.empty(H, device="cuda"),
                    ws=torch.empty(binding.strata_rmsnorm_backward_workspace(T, H),
                                   dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            binding.strata_rmsnorm(bufs["x"], bufs["r"], w, EPS, bufs["ro"], bufs["out"])
            binding.strata_rmsnorm_backward(bufs["ro"], w, EPS, dy, None, bufs["dx"], bufs["dw"],
                                            bufs["ws"])
        graphs.append((g, bufs, torch.cuda.Stream()))
    for round_ in range(3):
        for i, (g, b, s) in enumerate(graphs):
            b["x"].copy_(rows(T, H, "bf16", 50 + 2 * round_ + i))
        torch.cuda.synchronize()
        for g, b, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for g, b, s in graphs:
            ro, out, _, _ = run_forward(b["x"], b["r"], w)
            dx, dw = run_backward(ro, w, dy, None)
            assert torch.equal(ro, b["ro"]) and torch.equal(out, b["out"])
            assert torch.equal(dx, b["dx"]) and torch.equal(dw, b["dw"])
    assert bwant[0].shape == (T, H)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_one_row_is_the_same_in_any_stride(dt):
    H = 4096
    w = weight(H)

    def row(seed, ld):
        return rows(1, H, dt, seed).as_strided((1, H), (ld, 1))

    got = []
    for ld in (H, H + 1, 3):
        x, r, dy, ds = (row(s, ld) for s in (1, 2, 3, 4))
        ro, out = (torch.empty(1, H, dtype=DT[dt], device="cuda").as_strided((1, H), (ld, 1)) for _ in range(2))
        binding.strata_rmsnorm(x, r, w, EPS, ro, out)
        dx, dg = torch.empty(1, H, dtype=DT[dt], device="cuda"), torch.empty(H, device="cuda")
        ws = torch.empty(binding.strata_rmsnorm_backward_workspace(1, H), dtype=torch.uint8, device="cuda")
        binding.strata_rmsnorm_backward(ro, w, EPS, dy, ds, dx, dg, ws)
        got.append((ro, out, dx, dg))
    for a, b in zip(got[0], got[1]):
        assert torch.equal(a, b)
    for a, b in zip(got[0], got[2]):
        assert torch.equal(a, b)
