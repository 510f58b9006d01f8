"""Calls of two host threads whose launches of one kernel need different amounts
of shared memory: neither may lower the kernel's limit under the other.  All work
goes to one stream; each thread has its own buffers and its own handle."""
import threading

import pytest

torch = pytest.importorskip("torch")

from quantized_routed_expert_04_b200 import binding  # noqa: E402

pytestmark = pytest.mark.gpu

CALLS = 3000


def both(*calls):
    """Each call over and over in a thread of its own; what they raised."""
    stream = torch.cuda.current_stream().cuda_stream
    raised, start = [], threading.Barrier(len(calls))

    def run(call):
        start.wait()
        try:
            for _ in range(CALLS):
                call(stream)
        except Exception as e:   # noqa: BLE001 (the thread's, for the test to show)
            raised.append(e)

    threads = [threading.Thread(target=run, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not raised, raised


def test_norm_gradient_of_two_widths():
    L = binding.load_library()

    def call(H, T=4):
        h, dy, ds = (torch.randn(T, H, device="cuda").bfloat16() for _ in range(3))
        dx, w, dg = torch.empty_like(h), torch.ones(H, device="cuda"), torch.empty(H, device="cuda")
        ws = torch.empty(binding.strata_rmsnorm_backward_workspace(T, H), dtype=torch.uint8, device="cuda")

        def run(stream):   # (the C call: the interpreter is not held during it)
            st = L.strata_rmsnorm_backward(binding.DTYPE_BF16, h.data_ptr(), H, w.data_ptr(), 1e-6,
                                           dy.data_ptr(), H, ds.data_ptr(), H, T, H, dx.data_ptr(), H,
                                           dg.data_ptr(), ws.data_ptr(), ws.nbytes, stream)
            if st:
                raise binding.StrataError(st, "strata_rmsnorm_backward %d" % H)
        return run

    both(call(2304), call(4096))


# one launch on the fp32 units; three launches, where dx's kernel goes by the experts
@pytest.mark.parametrize("shapes", [[(8, 16), (40, 64)], [(300, 60), (260, 256)], [(300, 60), (260, 100)]])
def test_router_gradient_of_two_sizes(shapes):
    L = binding.load_library()
    H, layers = 256, []

    def call(T, E):
        layer = binding.StrataMoE(H, 128, E, 1, 0, E)
        layers.append(layer)
        W = torch.randn(E, H, device="cuda")
        layer.set_router(W, None)
        x, d = torch.randn(T, H, device="cuda").bfloat16(), torch.randn(T, E, device="cuda")
        dW, db, dx = torch.empty_like(W), torch.empty(E, device="cuda"), torch.empty_like(x)
        ws = torch.empty(layer.route_backward_workspace(T), dtype=torch.uint8, device="cuda")

        def run(stream):
            st = L.strata_moe_route_backward(layer.h, x.data_ptr(), T, None, None, None, d.data_ptr(),
                                             dW.data_ptr(), db.data_ptr(), dx.data_ptr(), ws.data_ptr(),
                                             ws.nbytes, stream)
            if st:
                raise binding.StrataError(st, "strata_moe_route_backward %d x %d" % (T, E))
        run.keep = W
        return run

    both(*(call(*s) for s in shapes))
    for layer in layers:
        assert int(layer.status()[0]) == 0
        layer.close()


def test_decode_of_two_batches():
    from harness import GpuLayer
    from quantized_routed_expert_04_b200 import synth
    L = binding.load_library()
    layers = [GpuLayer(synth.CONFIGS["tiny"]) for _ in range(2)]

    def call(gl, T):
        x = torch.randn(T, gl.cfg.hidden, device="cuda").bfloat16()
        out = torch.empty_like(x)
        gl.layer.reserve(T)

        def run(stream):
            st = L.strata_moe_forward(gl.layer.h, x.data_ptr(), T, out.data_ptr(), stream)
            if st:
                raise binding.StrataError(st, "strata_moe_forward %d" % T)
        return run

    both(call(layers[0], 9), call(layers[1], 64))
    for gl in layers:
        assert int(gl.layer.status()[0]) == 0
        gl.close()
