"""Grouped products whose bounded waits run out: the call reports the time-out,
the kernel leaves nothing behind, and the next call is right."""
import time

import pytest

import dense_fp32_matrix_strict_gb300 as sg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("transw", [True, False])
@pytest.mark.parametrize("sizes", [[20], [20, 0, 12]], ids=str)
def test_a_wait_that_runs_out_is_reported(sizes, transw):
    # The longest wait of the kernel is the epilogue's for a whole sum. A limit
    # of a microsecond ends it after about 70 (the barrier's own suspension);
    # these sums, one tile each for all pairs of SMs, take 200.
    import torch
    N, K = 256 * 76, 32768
    x = torch.randn(sum(sizes), K, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(len(sizes), *((N, K) if transw else (K, N)), device="cuda", dtype=torch.bfloat16)
    off = torch.tensor([sum(sizes[:i]) for i in range(len(sizes) + 1)], dtype=torch.int32, device="cuda")
    want, y = (torch.empty(sum(sizes), N, device="cuda", dtype=torch.bfloat16) for _ in range(2))

    def call(out):
        sg.sgemm_grouped_tensors(1.0, x, w, off, 0.0, out, transw=transw)

    call(want)
    sg.check_status()
    assert sg.sgemm_set_wait_timeout_ns(1000) == sg.SGEMM_OK
    try:
        start = time.monotonic()
        call(y)
        rc, bits = sg.sgemm_check_status(torch.cuda.current_stream().cuda_stream)
        assert time.monotonic() - start < 5.0
        assert rc == sg.SGEMM_ERR_DEVICE_TIMEOUT and bits & 7
    finally:
        assert sg.sgemm_set_wait_timeout_ns(2_000_000_000) == sg.SGEMM_OK
    for _ in range(2):
        y.fill_(float("nan"))
        call(y)
        sg.check_status()
        assert torch.equal(y, want)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("kind", ["nk", "kn", "wgrad"])
@pytest.mark.parametrize("sizes,a,b", [([70, 0, 300], 200, 96), ([40, 20], 130, 4100), ([1500], 72, 64)], ids=str)
def test_float_blocks_see_their_copies_land(sizes, a, b, kind, shift):
    # Blocks wait for their last copies at the end, with a limit of their own
    # where the caller's is shorter: no status bit, and the same results.
    import torch
    rows = sum(sizes)
    off = torch.tensor([sum(sizes[:i]) for i in range(len(sizes) + 1)], dtype=torch.int32, device="cuda")

    def operand(*shape):
        n = 1
        for v in shape:
            n *= v
        return torch.randn(n + shift, device="cuda")[shift:].view(shape)

    if kind == "wgrad":
        p, q = operand(rows, a), operand(rows, b)
        outs = [torch.empty(len(sizes), a, b, device="cuda") for _ in range(2)]

        def call(out):
            sg.sgemm_grouped_wgrad_tensors(1.0, p, q, off, 0.0, out)
    else:
        x, w = operand(rows, b), operand(len(sizes), *((a, b) if kind == "nk" else (b, a)))
        outs = [torch.empty(rows, a, device="cuda") for _ in range(2)]

        def call(out):
            sg.sgemm_grouped_tensors(1.0, x, w, off, 0.0, out, transw=kind == "nk")

    call(outs[0])
    sg.check_status()
    assert sg.sgemm_set_wait_timeout_ns(1_000_000) == sg.SGEMM_OK
    try:
        call(outs[1])
        sg.check_status()
    finally:
        assert sg.sgemm_set_wait_timeout_ns(2_000_000_000) == sg.SGEMM_OK
    assert torch.equal(outs[0], outs[1])
