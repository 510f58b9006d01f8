"""What the binding refuses of the tensors of a norm or training call, on the CPU:
with the library's side and the device check put aside, a call that goes together
gets through, and one with a single operand changed is refused."""
import pytest

torch = pytest.importorskip("torch")

from quantized_routed_expert_04_b200 import binding  # noqa: E402

T, H, E, K, G = 8, 256, 16, 4, 64
BF16, F16, F32, I32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.uint8


@pytest.fixture
def reached(monkeypatch):
    """The names of the library calls that were reached."""
    calls = []
    for name in ("rmsnorm", "rmsnorm_backward", "balance", "balance_backward", "route_backward"):
        packed = getattr(binding, "_packed_" + name)
        monkeypatch.setattr(packed, "call", lambda words, n=name: calls.append(n) or 0)
    for name in ("forward_norm", "forward_q8"):
        monkeypatch.setattr(binding, "strata_moe_" + name, lambda *a, n=name: calls.append(n))
    monkeypatch.setattr(binding, "_stream_on", lambda stream, dev, where: 0)
    return calls


class Layer(binding.StrataMoE):
    """A layer without a handle."""

    def __init__(self):
        self.h, self.hidden, self.n_experts, self.top_k = 0, H, E, K

    def close(self):
        pass


layer = Layer


def t(dtype, *shape):
    return torch.zeros(*shape, dtype=dtype)


def norm(**kw):
    binding.strata_rmsnorm(kw["x"], kw["residual"], kw["weight"], 1e-6, kw["residual_out"], kw["out"],
                           kw["out_q8"], kw["scales"], G)


def norm_backward(**kw):
    binding.strata_rmsnorm_backward(kw["h"], kw["weight"], 1e-6, kw["dout"], kw["dsum"], kw["dx"],
                                    kw["dweight"], kw["workspace"])


def forward_norm(**kw):
    layer().forward_norm(kw["x"], kw["residual"], kw["weight"], 1e-6, kw["residual_out"], kw["normed"],
                         kw["out"])


def forward_q8(**kw):
    layer().forward_q8(kw["x_q8"], kw["scales"], G, kw["x"], kw["out"])


def balance(**kw):
    layer().balance(kw["logits"], kw["idx"], 0.1, kw["counts"], kw["tokens"], kw["loss"], kw["workspace"],
                    kw["seq_off"], kw["mask"])


def balance_backward(**kw):
    layer().balance_backward(kw["logits"], 0.1, kw["counts"], kw["tokens"], kw["dlogits"], kw["dloss"],
                             kw["seq_off"], kw["mask"])


def route_backward(**kw):
    layer().route_backward(kw["x"], kw["logits"], kw["idx"], kw["dw"], kw["dlogits"], kw["dW"], kw["db"],
                           kw["dx"], kw["workspace"])


def rows():
    return t(BF16, T, H)


CALLS = {
    norm: lambda: dict(x=rows(), residual=rows(), weight=t(F32, H), residual_out=rows(), out=rows(),
                       out_q8=t(torch.float8_e4m3fn, T, H), scales=t(F32, T, H // G)),
    norm_backward: lambda: dict(h=rows(), weight=t(F32, H), dout=rows(), dsum=rows(), dx=rows(),
                                dweight=t(F32, H), workspace=t(U8, 4096)),
    forward_norm: lambda: dict(x=rows(), residual=rows(), weight=t(F32, H), residual_out=rows(),
                               normed=rows(), out=rows()),
    forward_q8: lambda: dict(x_q8=t(torch.float8_e4m3fn, T, H), scales=t(F32, T, H // G), x=rows(), out=rows()),
    balance: lambda: dict(logits=t(F32, T, E), idx=t(I32, T, K), counts=t(I32, 2, E), tokens=t(I32, 2),
                          loss=t(F32, 1), workspace=t(U8, 4096), seq_off=t(I32, 3), mask=t(U8, T)),
    balance_backward: lambda: dict(logits=t(F32, T, E), counts=t(I32, 2, E), tokens=t(I32, 2),
                                   dlogits=t(F32, T, E), dloss=t(F32, 1), seq_off=t(I32, 3), mask=t(U8, T)),
    route_backward: lambda: dict(x=rows(), logits=t(F32, T, E), idx=t(I32, T, K), dw=t(F32, T, K),
                                 dlogits=t(F32, T, E), dW=t(F32, E, H), db=t(F32, E), dx=rows(),
                                 workspace=t(U8, 4096)),
}
# another type of the same size: what a check of bytes alone lets through
OTHER = {BF16: F16, F32: I32, I32: F32, U8: torch.float8_e5m2, torch.float8_e4m3fn: torch.float8_e5m2}


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
def test_operands(call, reached):
    call(**CALLS[call]())
    assert reached == [call.__name__.replace("norm", "rmsnorm") if call in (norm, norm_backward)
                       else call.__name__]
    for name, good in CALLS[call]().items():
        changes = dict(type=good.view(OTHER[good.dtype]), size=torch.cat((good, good[:1])))
        if name in ("x", "h") and call in (norm, norm_backward):
            del changes["size"]      # (its rows are what the others go by)
            changes["type"] = good.half()
        if name == "workspace":      # any type; the library checks its size
            changes = dict()
        if good.dim() == 2:
            changes["order"] = good.t().contiguous().t()
        elif name != "loss" and name != "dloss":
            changes["order"] = torch.cat((good, good))[::2]
        for what, bad in changes.items():
            del reached[:]
            with pytest.raises(binding.StrataError) as e:
                call(**{**CALLS[call](), name: bad})
            assert e.value.status == binding.Status.INVALID_ARG and not reached, (name, what)


def test_operands_of_more_than_one_type(reached):
    for call, name, good in ((norm, "out_q8", t(U8, T, H)), (forward_q8, "x_q8", t(U8, T, H)),
                             (balance, "mask", t(torch.bool, T)), (balance, "mask", t(torch.int8, T)), (balance_backward, "mask", t(torch.bool, T))):
        call(**{**CALLS[call](), name: good})
    for dt in (F16, F32):
        a = {n: v.to(dt) if v.dtype is BF16 else v for n, v in CALLS[norm]().items()}
        norm(**a)
        norm_backward(**{n: v.to(dt) if v.dtype is BF16 else v for n, v in CALLS[norm_backward]().items()})
    assert len(reached) == 9


def test_a_closed_layer_is_refused():
    # (a null handle goes to the library, which refuses it before anything else)
    from quantized_routed_expert_04_b200 import build
    build.build()
    closed = Layer()
    closed.h = None
    a, b, r = CALLS[balance](), CALLS[balance_backward](), CALLS[route_backward]()
    with pytest.MonkeyPatch.context() as m:
        m.setattr(binding, "_stream_on", lambda stream, dev, where: 0)
        for call in (lambda: closed.balance(a["logits"], a["idx"], 0.1, a["counts"], a["tokens"], a["loss"],
                                            a["workspace"], a["seq_off"], a["mask"]),
                     lambda: closed.balance_backward(b["logits"], 0.1, b["counts"], b["tokens"], b["dlogits"],
                                                     b["dloss"], b["seq_off"], b["mask"]),
                     lambda: closed.route_backward(*(r[n] for n in ("x", "logits", "idx", "dw", "dlogits", "dW",
                                                                    "db", "dx", "workspace")))):
            with pytest.raises(binding.StrataError) as e:
                call()
            assert e.value.status == binding.Status.INVALID_ARG
