"""Argument checks of the norm calls (no GPU: every call here is refused, or
has nothing to do, before anything is enqueued)."""
import pytest

from quantized_routed_expert_04_b200 import binding, build

BAD, UNSUP, OK = (int(binding.Status.INVALID_ARG), int(binding.Status.UNSUPPORTED),
                  int(binding.Status.OK))
P = 1 << 20   # aligned addresses that are never read
Q = 1 << 21


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def fwd(lib, dtype=0, x=P, ldx=256, r=P, ldr=256, w=P, eps=1e-6, T=4, H=256, ro=P, ldro=256, out=Q,
        ldo=256, q8=None, sc=None, group=0):
    return lib.strata_rmsnorm(dtype, x, ldx, r, ldr, w, eps, T, H, ro, ldro, out, ldo, q8, sc,
                              group, None)


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(dtype=-1), dict(x=None), dict(w=None), dict(out=None), dict(T=-1),
    dict(H=0), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(ldx=255),
    dict(ldr=255), dict(ldro=0), dict(ldo=-256), dict(x=P + 1), dict(r=P + 1), dict(ro=P + 1),
    dict(out=P + 1), dict(w=P + 2), dict(ro=Q, out=Q), dict(q8=P, sc=None, group=32), dict(q8=None, sc=P),
    dict(q8=P, sc=P, group=0), dict(q8=P, sc=P, group=96), dict(q8=P, sc=P, group=-32),
    dict(q8=P, sc=P + 2, group=32), dict(dtype=2, x=P + 2),
])
def test_forward_refuses(lib, kw):
    assert fwd(lib, **kw) == BAD


def test_forward_limits_and_nothing_to_do(lib):
    assert fwd(lib, H=16385, ldx=16385, ldr=16385, ldro=16385, ldo=16385) == UNSUP
    assert fwd(lib, T=0) == OK
    assert fwd(lib, T=0, x=None, r=None, ro=None, out=None) == OK


def bwd(lib, dtype=0, h=P, ldh=256, w=P, eps=1e-6, dy=P, ldd=256, ds=P, lds=256, T=4, H=256, dx=P,
        ldx=256, dw=P, ws=P, n=1 << 30):
    return lib.strata_rmsnorm_backward(dtype, h, ldh, w, eps, dy, ldd, ds, lds, T, H, dx, ldx, dw,
                                       ws, n, None)


@pytest.mark.parametrize("kw", [
    dict(dtype=5), dict(h=None), dict(w=None), dict(dy=None), dict(dx=None), dict(T=-2),
    dict(H=-1), dict(eps=-1.0), dict(ldh=100), dict(ldd=100), dict(lds=100), dict(ldx=100),
    dict(dw=P + 1), dict(ws=None), dict(ws=P + 8), dict(n=0), dict(dy=P + 1), dict(ds=P + 1),
])
def test_backward_refuses(lib, kw):
    assert bwd(lib, **kw) == BAD


def test_backward_limits(lib):
    assert bwd(lib, H=20000, ldh=20000, ldd=20000, lds=20000, ldx=20000) == UNSUP
    assert bwd(lib, T=0, dw=None, ws=None, n=0) == OK
    need = binding.strata_rmsnorm_backward_workspace(4, 256)
    assert need > 0 and bwd(lib, n=need - 1) == BAD
    assert binding.strata_rmsnorm_backward_workspace(4, 20000) == 0
    assert binding.strata_rmsnorm_backward_workspace(-1, 256) == 0


def test_binding_refuses_operands_that_do_not_go_together():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64)

    def refused(*a, **k):
        with pytest.raises(binding.StrataError) as e:
            binding.strata_rmsnorm(*a, **k)
        assert e.value.status == binding.Status.INVALID_ARG

    refused(x, None, w, 1e-6, out=torch.empty_like(x))                      # not on the GPU
    refused(x, x.float(), w, 1e-6, out=torch.empty_like(x))                 # another type
    refused(x, x[:3], w, 1e-6, out=torch.empty_like(x))                     # another shape
    refused(x, None, w[:63], 1e-6, out=torch.empty_like(x))                 # short weight
    refused(x, None, w.half(), 1e-6, out=torch.empty_like(x))               # weight not fp32
    refused(x.t().contiguous().t(), None, w, 1e-6, out=torch.empty_like(x))  # column stride
    refused(x[0], None, w, 1e-6, out=x[0])                                  # not rows
    refused(x, None, w, 1e-6, out_q8=torch.empty(4, 64, dtype=torch.uint8), group=32)   # no scales
    refused(x, None, w, 1e-6, out_q8=torch.empty(4, 64, dtype=torch.uint8),
            scales=torch.empty(4, 3), group=32)                             # wrong scales
