"""qg_combine with Y and C at one address, on the CPU: taken only where they have one type and pitch (no call here reaches a device)."""
import pytest
import torch

import quantized_gemm_bf16_amd as qg

FAKE = 1 << 20


def combine(cd, yd, t, c=FAKE, y=FAKE, beta=1.0):
    return qg.Gemm().combine_raw(FAKE, qg.layout("bf16", 8, 64), FAKE, FAKE, qg.layout("f32", t, 2), y, yd, beta=beta, C=c, Cd=cd)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are no device's")
@pytest.mark.parametrize("t", [1, 4])
def test_in_place(t):
    d = lambda dtype, ld=64: qg.layout(dtype, t, 64, ld=ld)  # noqa: E731
    bad, goes = qg.ERR_INVALID_ARG, qg.ERR_HIP
    for a, b in (("bf16", "f32"), ("f32", "bf16"), ("bf16", "f16"), ("f16", "f32")):
        assert combine(d(a), d(b), t) == bad, (a, b)
        assert combine(d(a), d(b), t, c=FAKE + (1 << 20)) == goes
        assert combine(d(a), d(b), t, beta=0.0) == goes  # C is not read
    for dtype in ("bf16", "f16", "f32"):
        assert combine(d(dtype), d(dtype), t) == goes
        assert combine(d(dtype, 72), d(dtype), t) == (bad if t > 1 else goes)
        assert combine(d(dtype), d(dtype, 72), t) == (bad if t > 1 else goes)
    assert combine(qg.layout("bf16", 0, 64), qg.layout("f32", 0, 64), 0, c=None, y=None) == qg.OK
