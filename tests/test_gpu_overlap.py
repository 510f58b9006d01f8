"""Training and layer calls whose outputs share part of an operand's memory are
refused (an operand as a whole in the place of another is in the other files)."""
import pytest

torch = pytest.importorskip("torch")

from harness import GpuLayer  # noqa: E402
from quantized_routed_expert_04_b200 import binding, synth  # noqa: E402

pytestmark = pytest.mark.gpu


def refused(call, *a, **kw):
    with pytest.raises(binding.StrataError) as e:
        call(*a, **kw)
    assert e.value.status == binding.Status.INVALID_ARG


def views(total, *offsets, n, like):
    """Contiguous views of n elements at the offsets of one buffer, shaped as `like`."""
    buf = torch.zeros(total, dtype=like.dtype, device="cuda")
    return [buf[o:o + n].view_as(like) for o in offsets]


@pytest.mark.parametrize("T,E", [(4, 8), (300, 64)])
def test_training_calls(T, E):
    H, k = 256, 2
    layer = binding.StrataMoE(H, 128, E, k, 0, E)
    W = torch.randn(E, H, device="cuda")
    layer.set_router(W, None)
    d, dW = torch.randn(T, E, device="cuda"), torch.empty(E, H, device="cuda")
    ws = torch.empty(layer.route_backward_workspace(T), dtype=torch.uint8, device="cuda")
    like, n = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), T * H
    for off, ok in ((0, False), (H, False), (n - 8, False), (n, True)):
        for swap in (False, True):
            x, dx = views(2 * n, *((off, 0) if swap else (0, off)), n=n, like=like)
            args = (x, None, None, None, d, dW, None, dx, ws)
            layer.route_backward(*args) if ok else refused(layer.route_backward, *args)
    counts = torch.zeros(1, E, dtype=torch.int32, device="cuda")
    tokens = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = T * E
    for off, ok in ((0, False), (E, False), (n - 4, False), (n, True)):
        logits, dlogits = views(2 * n, 0, off, n=n, like=d)
        args = (logits, 0.1, counts, tokens, dlogits)
        layer.balance_backward(*args) if ok else refused(layer.balance_backward, *args)
    torch.cuda.synchronize()
    assert int(layer.status()[0]) == 0
    layer.close()


def test_layer_calls():
    gl = GpuLayer(synth.CONFIGS["tiny"])
    T, H, n = 4, gl.cfg.hidden, 4 * gl.cfg.hidden
    like = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    x, gain = torch.randn(T, H, device="cuda").bfloat16(), torch.ones(H, device="cuda")
    q, scales = torch.zeros(T, H, dtype=torch.uint8, device="cuda"), torch.ones(T, 1, device="cuda")
    for off, ok in ((0, False), (H, False), (n - 8, False), (n, True)):
        a, b = views(2 * n, 0, off, n=n, like=like)
        other = torch.empty_like(like)
        for args in ((x, None, gain, 1e-6, None, a, b), (x, None, gain, 1e-6, a, other, b),
                     (x, None, gain, 1e-6, a, b, other)):
            gl.layer.forward_norm(*args) if ok else refused(gl.layer.forward_norm, *args)
        args = (q, scales, H, a, b)
        gl.layer.forward_q8(*args) if ok else refused(gl.layer.forward_q8, *args)
    raw = torch.zeros(3 * n, dtype=torch.uint8, device="cuda")
    for off, ok in ((0, False), (n, False), (2 * n - 16, False), (2 * n, True)):
        rows = raw[:2 * n].view(torch.bfloat16).view(T, H)
        args = (raw[off:off + n].view(T, H), scales, H, rows, torch.empty_like(like))
        gl.layer.forward_q8(*args) if ok else refused(gl.layer.forward_q8, *args)
    torch.cuda.synchronize()
    assert int(gl.layer.status()[0]) == 0
    gl.close()
