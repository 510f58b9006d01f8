"""The layer with its norm in front, and on 8-bit activations: the same bits as
the separate calls, and the oracle's result within the layer's tolerance."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from harness import GpuLayer, assert_within_tolerance, oracle_reference  # noqa: E402
from quantized_routed_expert_04_b200 import binding, synth  # noqa: E402

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def gl():
    layer = GpuLayer(synth.CONFIGS["tiny"])
    yield layer
    layer.close()


def inputs(T, H, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    r = (torch.randn(T, H, device="cuda", generator=g) * 2).bfloat16()
    return x, r, 1 + 0.2 * torch.randn(H, device="cuda", generator=g)


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("T", [1, 4, 64, 65, 130])
@pytest.mark.parametrize("residual", [False, True])
def test_forward_norm(gl, T, residual):
    H = gl.cfg.hidden
    x, r, w = inputs(T, H, T)
    r = r if residual else None
    s1, n1, o1 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    binding.strata_rmsnorm(x, r, w, EPS, s1, n1)
    gl.layer.forward(n1, o1)
    s2, n2, o2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    gl.layer.forward_norm(x, r, w, EPS, s2, n2, o2)
    assert int(gl.layer.status()[0]) == 0
    for a, b in ((s1, s2), (n1, n2), (o1, o2)):
        assert torch.equal(a, b)
    ref, _, _ = oracle_reference(gl.cfg, gl.blobs, gl.W, gl.b, bits(n2))
    assert_within_tolerance(bits(o2), ref)
    # the sum over the residual, as a chain of layers keeps it
    if residual:
        keep = r.clone()
        gl.layer.forward_norm(x, r, w, EPS, r, n2, o2)
        assert torch.equal(r, s1) and torch.equal(o2, o1)
        r.copy_(keep)


@pytest.mark.parametrize("T", [1, 64, 65])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
def test_forward_q8(gl, T, group):
    H = gl.cfg.hidden
    x, r, w = inputs(T, H, 7 + T)
    q = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(T, -(-H // group), device="cuda")
    binding.strata_rmsnorm(x, r, w, EPS, None, None, q, sc, group)
    want_x = (q.float() * sc.repeat_interleave(group, 1)[:, :H]).bfloat16()
    want = torch.empty_like(x)
    gl.layer.forward(want_x, want)
    xb, out = torch.empty_like(x), torch.empty_like(x)
    gl.layer.forward_q8(q, sc, group, xb, out)
    assert int(gl.layer.status()[0]) == 0
    assert torch.equal(xb, want_x) and torch.equal(out, want)


def test_captured(gl):
    T, H = 8, gl.cfg.hidden
    x, r, w = inputs(T, H, 31)
    s, n, o = (torch.empty_like(x) for _ in range(3))
    gl.layer.reserve(T)
    gl.layer.forward_norm(x, r, w, EPS, s, n, o)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gl.layer.forward_norm(x, r, w, EPS, s, n, o)
    x2, _, _ = inputs(T, H, 32)
    x.copy_(x2)
    g.replay()
    got = [t.clone() for t in (s, n, o)]
    gl.layer.forward_norm(x, r, w, EPS, s, n, o)
    torch.cuda.synchronize()
    for a, b in zip(got, (s, n, o)):
        assert torch.equal(a, b)
    assert int(gl.layer.status()[0]) == 0


def test_refusals(gl):
    lib = binding.load_library()
    T, H = 4, gl.cfg.hidden
    x, r, w = inputs(T, H, 41)
    o = torch.empty_like(x)
    n = torch.empty_like(x)
    bad = int(binding.Status.INVALID_ARG)

    def fn(h=gl.layer.h, x=x.data_ptr(), r=r.data_ptr(), w=w.data_ptr(), eps=EPS, T=T, s=None,
           n=n.data_ptr(), o=o.data_ptr()):
        return lib.strata_moe_forward_norm(h, x, r, w, eps, T, s, n, o, None)

    for kw in (dict(h=None), dict(x=None), dict(w=None), dict(eps=-1.0), dict(T=-1), dict(n=None),
               dict(o=None), dict(o=n.data_ptr()), dict(n=n.data_ptr() + 2),
               dict(s=o.data_ptr())):
        assert fn(**kw) == bad, kw
    assert fn(T=0) == 0
    q = torch.zeros(T, H, dtype=torch.uint8, device="cuda")
    sc = torch.ones(T, 8, device="cuda")

    def fq(h=gl.layer.h, q=q.data_ptr(), sc=sc.data_ptr(), group=32, T=T, x=n.data_ptr(),
           o=o.data_ptr()):
        return lib.strata_moe_forward_q8(h, q, sc, group, T, x, o, None)

    for kw in (dict(h=None), dict(q=None), dict(q=q.data_ptr() + 8), dict(sc=None), dict(group=0),
               dict(group=96), dict(T=-1), dict(x=None), dict(o=None), dict(x=o.data_ptr())):
        assert fq(**kw) == bad, kw
    assert fq(T=0) == 0
    with pytest.raises(binding.StrataError):
        gl.layer.forward_norm(x, r[:3], w, EPS, None, n, o)
    with pytest.raises(binding.StrataError):
        gl.layer.forward_q8(q, sc[:3], 32, n, o)


def test_types_are_checked(gl):
    # 16-bit operands of another type than the layer's
    T, H = 4, gl.cfg.hidden
    x, r, w = inputs(T, H, 42)
    s, n, o = (torch.empty_like(x) for _ in range(3))
    args = [x, r, w, EPS, s, n, o]
    for i in (0, 1, 4, 5, 6):
        bad = list(args)
        bad[i] = bad[i].half()
        with pytest.raises(binding.StrataError):
            gl.layer.forward_norm(*bad)
    q = torch.zeros(T, H, dtype=torch.uint8, device="cuda")
    sc = torch.ones(T, H // 32, device="cuda")
    for a, b in ((n.half(), o), (n, o.half())):
        with pytest.raises(binding.StrataError):
            gl.layer.forward_q8(q, sc, 32, a, b)
