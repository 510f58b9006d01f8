"""Norm calls whose outputs share memory with other operands other than row by row
in the same place are refused.  The addresses are made up and no call may reach a
GPU, so the file is left out where there is one; a call that is not refused ends
with a CUDA error here."""
import random

import pytest

torch = pytest.importorskip("torch")

from quantized_routed_expert_04_b200 import binding, build  # noqa: E402

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where no GPU is")

BAD = int(binding.Status.INVALID_ARG)
FAR = 1 << 30


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def forward(lib, T, H, x, ldx, r, ldr, ro, ldro, out, ldo):
    return lib.strata_rmsnorm(2, x, ldx, r, ldr, FAR * 9, 1e-6, T, H, ro, ldro, out, ldo, None, None, 0,
                              None) == BAD


def backward(lib, T, H, h, ldh, dy, ldd, ds, lds, dx, ldx):
    return lib.strata_rmsnorm_backward(2, h, ldh, FAR * 9, 1e-6, dy, ldd, ds, lds, T, H, dx, ldx, None,
                                       None, 0, None) == BAD


def test_whole_rows_shifted_or_in_another_stride(lib):
    T, H, a, b, c = 4, 8, FAR, 2 * FAR, 3 * FAR
    assert not forward(lib, T, H, a, H, b, H, b, H, a, H)            # the sum over the residual, y over x
    assert forward(lib, T, H, a, H, b, H, c, H, a + 4 * H, H)        # y one row behind x
    assert forward(lib, T, H, a, 2 * H, b, H, c, H, a, H)            # y over x in another stride
    assert forward(lib, T, H, a, H, b, H, a - 4, H, c, H)            # the sum one element before x
    assert forward(lib, T, H, a, H, b, H, c, H, c + 4 * H, H)        # y over the sum's rows
    assert forward(lib, T, H, a, H, None, 0, b, H, b, H)             # ... in their place
    assert not forward(lib, T, H, a, 2 * H, b, H, c, H, a + 4 * H, 2 * H)   # between x's rows
    assert not forward(lib, T, H, a, H, b, H, c, H, a + 4 * H * T, H)       # right behind x
    assert not forward(lib, 1, H, a, H, None, 0, None, 0, a, 99)     # one row: strides do not matter
    d = 4 * FAR
    assert not backward(lib, T, H, a, H, b, H, c, H, c, H)
    assert backward(lib, T, H, a, H, b, H, c, H, c + 4, H)
    assert backward(lib, T, H, a, H, b, H, None, 0, a, H + 4)
    assert backward(lib, T, H, a, H, b, H, None, 0, b - 4 * H, H)
    assert not backward(lib, T, H, a, H, b, H, c, H, d, H)


def test_against_sets_of_elements(lib):
    rng = random.Random(5)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        T, H = rng.randint(1, 7), rng.randint(1, 6)
        ld = [rng.randint(H, 3 * H) for _ in range(2)]
        if rng.random() < 0.5:
            ld[1] = ld[0]
        at = rng.randint(-2 * T * H, 2 * T * H)
        x = {i * ld[0] + j for i in range(T) for j in range(H)}
        out = {at + i * ld[1] + j for i in range(T) for j in range(H)}
        same = at == 0 and (T == 1 or ld[0] == ld[1])
        want = bool(x & out) and not same
        seen[want] += 1
        assert forward(lib, T, H, FAR, ld[0], None, 0, None, 0, FAR + 4 * at, ld[1]) == want, (T, H, ld, at)
        assert backward(lib, T, H, 2 * FAR, H, FAR, ld[0], None, 0, FAR + 4 * at, ld[1]) == want
    assert min(seen.values()) > 500
