"""Products grouped by expert against a loop over the groups in 64 bits."""
import numpy as np
import pytest

import dense_fp32_matrix_strict_gb300 as sg

pytestmark = pytest.mark.gpu

TYPES = ["float32", "bfloat16"]


def _torch():
    import torch
    return torch


def placed(x, extra=0, shift=0):
    """x on the GPU with rows `extra` elements further apart, starting `shift` elements
    into its buffer, NaN around it; returns (view, buffer)."""
    torch = _torch()
    rows, cols = x.shape[-2:]
    lead = x.shape[0] if x.dim() == 3 else 1
    ld = cols + extra
    buf = torch.full((lead * rows * ld + shift + 64,), float("nan"), dtype=x.dtype, device="cuda")
    view = buf[shift:shift + lead * rows * ld].view(lead, rows, ld)[:, :, :cols]
    view.copy_(x.reshape(lead, rows, cols))
    return (view if x.dim() == 3 else view[0]), buf


def offsets_of(sizes, before=0):
    torch = _torch()
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]) + before, dtype=torch.int32).cuda()


def tolerance(ref, size, depth, dtype):
    torch = _torch()
    # 4 K 2^-24 sum|terms| covers FP32 sums in any order (and the tensor cores'
    # truncating ones); a bfloat16 result adds its own rounding.
    tol = 4.0 * max(depth, 8) * 2.0 ** -24 * size + 1e-30
    return tol + 2.0 ** -8 * ref.abs() if dtype == torch.bfloat16 else tol


def forward(sizes, N, K, dtype, transw, alpha=1.0, beta=0.0, extra=0, shift=0, before=0, after=0, seed=0):
    torch = _torch()
    g = torch.Generator().manual_seed(seed + N * 3 + K)
    E, rows = len(sizes), sum(sizes) + before + after
    x = torch.randn(rows, K, generator=g).to(dtype)
    w = (torch.randn(E, N, K, generator=g) if transw else torch.randn(E, K, N, generator=g)).to(dtype)
    y0 = torch.randn(rows, N, generator=g).to(dtype) if beta else torch.full((rows, N), float("nan")).to(dtype)
    dx, _ = placed(x, extra, shift)
    dw, _ = placed(w, extra, shift)
    dy, buf = placed(y0, extra, shift)
    sg.sgemm_grouped_tensors(alpha, dx, dw, offsets_of(sizes, before), beta, dy, transw=transw)
    sg.check_status()
    xd, wd, yd = x.cuda().double(), w.cuda().double(), y0.cuda().double()
    at = before
    for e, n in enumerate(sizes):
        if n:
            m = wd[e].t() if transw else wd[e]
            ref = alpha * (xd[at:at + n] @ m)
            size = abs(alpha) * (xd[at:at + n].abs() @ m.abs())
            if beta:
                ref = ref + beta * yd[at:at + n]
                size = size + abs(beta) * yd[at:at + n].abs()
            err = (dy[at:at + n].double() - ref).abs()
            assert bool((err <= tolerance(ref, size, K, dtype)).all()), (e, float((err / size).max()))
        at += n
    # Rows of no group, and what lies around the matrix, are untouched.
    outside = torch.ones_like(buf, dtype=torch.bool)
    ld = N + extra
    inner = outside[shift:shift + rows * ld].view(rows, ld)
    inner[:, :N] = False
    assert torch.isnan(buf[outside]).all()
    for part in (slice(0, before), slice(rows - after, rows)):
        same = dy[part].cpu()
        assert torch.equal(same.nan_to_num(7.0), y0[part].nan_to_num(7.0))


SIZES = [
    ([5], 8, 8), ([1], 1, 1), ([0, 0, 3], 16, 64), ([64, 0, 65, 1], 70, 33), ([128, 127, 129], 128, 96),
    ([300, 0, 0, 17, 256, 1, 1, 90], 264, 200), ([1] * 40, 512, 256), ([7, 33, 16, 15, 31], 1000, 130),
    ([257, 513], 520, 1032),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("transw", [False, True])
@pytest.mark.parametrize("sizes,N,K", SIZES, ids=lambda v: str(v)[:24])
def test_forward(sizes, N, K, transw, dtype):
    forward(sizes, N, K, getattr(_torch(), dtype), transw)


@pytest.mark.parametrize("transw", [False, True])
@pytest.mark.parametrize("sizes,N,K", [([10, 9, 11, 0, 10], 130, 300), ([8, 8, 8], 512, 2048), ([20, 1, 9], 37, 4100),
                                       ([30, 0, 0, 3], 129, 9000)], ids=lambda v: str(v)[:24])
def test_forward_of_few_rows(sizes, N, K, transw):
    # Around the mean rows up to which W is streamed, sums in parts and in slabs.
    forward(sizes, N, K, _torch().float32, transw)
    forward(sizes, N, K, _torch().float32, transw, alpha=0.5, beta=-1.5, extra=1, shift=3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("transw", [False, True])
@pytest.mark.parametrize("extra,shift", [(1, 0), (8, 8), (3, 1), (0, 4), (5, 2)])
def test_forward_strides_and_alignment(extra, shift, transw, dtype):
    forward([70, 0, 200, 3], 136, 72, getattr(_torch(), dtype), transw, extra=extra, shift=shift)
    forward([70, 0, 200, 3], 131, 77, getattr(_torch(), dtype), transw, extra=extra, shift=shift)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("transw", [False, True])
def test_forward_alpha_beta_and_rows_of_no_group(transw, dtype):
    dt = getattr(_torch(), dtype)
    forward([40, 0, 130], 144, 80, dt, transw, alpha=0.7, beta=-1.3, before=9, after=11)
    forward([40, 0, 130], 144, 80, dt, transw, alpha=2.0, beta=0.0, before=3, after=200)
    forward([40, 0, 130], 33, 80, dt, transw, alpha=0.0, beta=0.5)
    forward([40, 0, 130], 33, 0, dt, transw, beta=1.0)


def weight_gradient(sizes, M, N, dtype, out, alpha=1.0, beta=0.0, extra=0, shift=0, before=0, after=0):
    torch = _torch()
    g = torch.Generator().manual_seed(M * 3 + N)
    E, rows = len(sizes), sum(sizes) + before + after
    p = torch.randn(rows, M, generator=g).to(dtype)
    q = torch.randn(rows, N, generator=g).to(dtype)
    # Rows of no group must not be read into any result.
    p[:before] = float("nan")
    p[rows - after:] = float("nan")
    q[:before] = float("inf")
    q[rows - after:] = float("inf")
    d0 = torch.randn(E, M, N, generator=g).to(out) if beta else torch.full((E, M, N), float("nan")).to(out)
    dp, _ = placed(p, extra, shift)
    dq, _ = placed(q, extra, shift)
    dd, buf = placed(d0, extra, shift)
    sg.sgemm_grouped_wgrad_tensors(alpha, dp, dq, offsets_of(sizes, before), beta, dd)
    sg.check_status()
    pd, qd = p.cuda().double(), q.cuda().double()
    at = before
    for e, n in enumerate(sizes):
        ref = alpha * (pd[at:at + n].t() @ qd[at:at + n])
        size = abs(alpha) * (pd[at:at + n].abs().t() @ qd[at:at + n].abs())
        if beta:
            ref = ref + beta * d0[e].cuda().double()
            size = size + abs(beta) * d0[e].cuda().double().abs()
        err = (dd[e].double() - ref).abs()
        assert bool((err <= tolerance(ref, size, n, out)).all()), e
        at += n
    ld = N + extra
    outside = torch.ones_like(buf, dtype=torch.bool)
    outside[shift:shift + E * M * ld].view(E, M, ld)[:, :, :N] = False
    assert torch.isnan(buf[outside]).all()


WGRAD = [("float32", "float32"), ("bfloat16", "float32"), ("bfloat16", "bfloat16")]


@pytest.mark.parametrize("dtype,out", WGRAD)
@pytest.mark.parametrize("sizes,M,N", SIZES, ids=lambda v: str(v)[:24])
def test_weight_gradient(sizes, M, N, dtype, out):
    torch = _torch()
    weight_gradient(sizes, M, N, getattr(torch, dtype), getattr(torch, out))


@pytest.mark.parametrize("dtype,out", WGRAD)
@pytest.mark.parametrize("extra,shift", [(1, 0), (8, 8), (3, 1), (0, 4), (5, 2)])
def test_weight_gradient_strides(extra, shift, dtype, out):
    torch = _torch()
    weight_gradient([70, 0, 200, 3], 136, 72, getattr(torch, dtype), getattr(torch, out), extra=extra, shift=shift)
    weight_gradient([70, 0, 200, 3], 131, 77, getattr(torch, dtype), getattr(torch, out), extra=extra, shift=shift)


@pytest.mark.parametrize("dtype,out", WGRAD)
def test_weight_gradient_accumulates(dtype, out):
    torch = _torch()
    dt, ot = getattr(torch, dtype), getattr(torch, out)
    weight_gradient([40, 0, 130], 144, 80, dt, ot, alpha=0.7, beta=1.0, before=9, after=11)
    weight_gradient([40, 0, 130], 33, 80, dt, ot, alpha=0.0, beta=0.5)
    weight_gradient([0, 0], 33, 80, dt, ot)
    weight_gradient([0, 0], 33, 80, dt, ot, beta=-2.0)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_nan_stays_in_its_group(dtype):
    torch = _torch()
    dt = getattr(torch, dtype)
    sizes, N, K = [30, 50, 20], 100, 72
    x = torch.randn(100, K).to(dt).cuda()
    w = torch.randn(3, N, K).to(dt).cuda()
    off = offsets_of(sizes)
    for bad_x, bad_w in ((float("nan"), 1.0), (float("inf"), 1.0), (1.0, float("nan"))):
        xb, wb = x.clone(), w.clone()
        xb[30:80] *= bad_x
        wb[1] *= bad_w
        y = torch.empty(100, N, dtype=dt, device="cuda")
        sg.sgemm_grouped_tensors(1.0, xb, wb, off, 0.0, y, transw=True)
        d = torch.empty(3, N, K, device="cuda")
        sg.sgemm_grouped_wgrad_tensors(1.0, xb[:, :K].new_ones(100, N) * (1.0 if bad_x == 1.0 else 2.0), xb, off,
                                       0.0, d)
        sg.check_status()
        assert torch.isfinite(y[:30].float()).all() and torch.isfinite(y[80:].float()).all()
        assert not torch.isfinite(y[30:80].float()).any()
        assert torch.isfinite(d[0]).all() and torch.isfinite(d[2]).all()


def test_gradients_against_differences():
    # Two-sided differences of L = sum(Y * C) in float64 against the kernels' gradients.
    torch = _torch()
    sizes, N, K = [3, 0, 4], 5, 6
    g = torch.Generator().manual_seed(11)
    x, w = torch.randn(7, K, generator=g), torch.randn(3, N, K, generator=g)
    c = torch.randn(7, N, generator=g)
    off = offsets_of(sizes)
    dx = torch.empty(7, K, device="cuda")
    dw = torch.empty(3, N, K, device="cuda")
    sg.sgemm_grouped_tensors(1.0, c.cuda(), w.cuda(), off, 0.0, dx)          # input gradient: C W
    sg.sgemm_grouped_wgrad_tensors(1.0, c.cuda(), x.cuda(), off, 0.0, dw)
    sg.check_status()

    def loss(xd, wd):
        total, at = 0.0, 0
        for e, n in enumerate(sizes):
            total += float(((xd[at:at + n] @ wd[e].t()) * c[at:at + n].double()).sum())
            at += n
        return total

    h = 1e-3                                     # L is bilinear: differences are exact but for rounding
    for i in range(7):
        for k in range(K):
            d = torch.zeros(7, K, dtype=torch.float64)
            d[i, k] = h
            diff = (loss(x.double() + d, w.double()) - loss(x.double() - d, w.double())) / (2 * h)
            assert abs(diff - float(dx[i, k])) <= 1e-5
    for e in range(3):
        for n in range(N):
            for k in range(K):
                d = torch.zeros(3, N, K, dtype=torch.float64)
                d[e, n, k] = h
                diff = (loss(x.double(), w.double() + d) - loss(x.double(), w.double() - d)) / (2 * h)
                assert abs(diff - float(dw[e, n, k])) <= 1e-5


@pytest.mark.parametrize("dtype", TYPES)
def test_bad_offsets_are_reported(dtype):
    torch = _torch()
    dt = getattr(torch, dtype)
    x = torch.randn(50, 64).to(dt).cuda()
    w = torch.randn(4, 64, 96).to(dt).cuda()
    good = offsets_of([10, 20, 10, 10])
    want = torch.empty(50, 96, dtype=dt, device="cuda")
    sg.sgemm_grouped_tensors(1.0, x, w, good, 0.0, want)
    sg.check_status()
    for bad in ([0, 20, 10, 10, 10], [0, 10, 30, 40, 51], [-1, 10, 30, 40, 50], [0, 10, 30, 2 ** 31 - 1, 50]):
        off = torch.tensor(bad, dtype=torch.int32).cuda()
        y = torch.full((50, 96), 3.0, dtype=dt, device="cuda")
        sg.sgemm_grouped_tensors(1.0, x, w, off, 0.0, y)
        rc, bits = sg.sgemm_check_status(torch.cuda.current_stream().cuda_stream)
        assert rc == sg.SGEMM_ERR_DEVICE_CHECK and bits == 32
        if bad[0] == 0:
            assert torch.equal(y[:10], want[:10])      # the groups that are right are computed
        d = torch.full((4, 64, 96), 3.0, device="cuda")
        sg.sgemm_grouped_wgrad_tensors(1.0, x, want, off, 0.0, d)
        rc, bits = sg.sgemm_check_status(torch.cuda.current_stream().cuda_stream)
        assert rc == sg.SGEMM_ERR_DEVICE_CHECK and bits == 32
        lengths = [b - a if 0 <= a <= b <= 50 else 0 for a, b in zip(bad, bad[1:])]
        for e, n in enumerate(lengths):
            assert bool((d[e] == 0).all()) == (n == 0)


@pytest.mark.parametrize("dtype", TYPES)
def test_many_groups(dtype):
    sizes = [(i * 7) % 5 for i in range(1024)]
    forward(sizes, 72, 40, getattr(_torch(), dtype), True)


@pytest.mark.parametrize("dtype", TYPES)
def test_captured_in_a_graph_with_new_offsets(dtype):
    # Offsets are read when the graph runs: a replay follows what they hold then.
    torch = _torch()
    dt = getattr(torch, dtype)
    x = torch.randn(300, 128).to(dt).cuda()
    w = torch.randn(4, 200, 128).to(dt).cuda()
    y = torch.empty(300, 200, dtype=dt, device="cuda")
    d = torch.empty(4, 200, 128, device="cuda")
    off = offsets_of([100, 50, 0, 150])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sg.sgemm_grouped_tensors(1.0, x, w, off, 0.0, y, transw=True)
        sg.sgemm_grouped_wgrad_tensors(1.0, y, x, off, 0.0, d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sg.sgemm_grouped_tensors(1.0, x, w, off, 0.0, y, transw=True)
        sg.sgemm_grouped_wgrad_tensors(1.0, y, x, off, 0.0, d)
    for sizes in ([100, 50, 0, 150], [1, 0, 299, 0], [75, 75, 75, 75]):
        off.copy_(offsets_of(sizes))
        graph.replay()
        sg.check_status()
        y2, d2 = torch.empty_like(y), torch.empty_like(d)
        sg.sgemm_grouped_tensors(1.0, x, w, off, 0.0, y2, transw=True)
        sg.sgemm_grouped_wgrad_tensors(1.0, y2, x, off, 0.0, d2)
        sg.check_status()
        assert torch.equal(y, y2) and torch.equal(d, d2)


# Few tiles and long sums: the sums are split and joined.
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("transw", [False, True])
@pytest.mark.parametrize("sizes,N,K", [([40], 72, 4096), ([16, 0, 20], 200, 5000), ([300], 130, 2500),
                                       ([9], 500, 8190)], ids=lambda v: str(v))
def test_forward_split_sums(sizes, N, K, transw, dtype):
    dt = getattr(_torch(), dtype)
    forward(sizes, N, K, dt, transw)
    forward(sizes, N, K, dt, transw, alpha=0.5, beta=2.0, extra=3, shift=1, before=5, after=6)


@pytest.mark.parametrize("dtype,out", WGRAD)
@pytest.mark.parametrize("sizes,M,N", [([5000], 130, 70), ([3000, 0, 77], 64, 200), ([1027], 256, 128)],
                         ids=lambda v: str(v))
def test_weight_gradient_split_sums(sizes, M, N, dtype, out):
    torch = _torch()
    dt, ot = getattr(torch, dtype), getattr(torch, out)
    weight_gradient(sizes, M, N, dt, ot)
    weight_gradient(sizes, M, N, dt, ot, alpha=0.5, beta=2.0, extra=3, shift=1, before=5, after=6)


@pytest.mark.parametrize("dtype", TYPES)
def test_same_bits_on_every_call_and_another_stream(dtype):
    torch = _torch()
    dt = getattr(torch, dtype)
    for sizes, N, K in (([30, 1, 90], 300, 4096), ([500, 0, 40], 264, 136)):
        x = torch.randn(sum(sizes), K).to(dt).cuda()
        w = torch.randn(3, N, K).to(dt).cuda()
        off = offsets_of(sizes)
        got = []
        for stream in (None, None, torch.cuda.Stream()):
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
            y = torch.empty(sum(sizes), N, dtype=dt, device="cuda")
            d = torch.empty(3, N, K, device="cuda")
            torch.cuda.synchronize()
            sg.sgemm_grouped_tensors(1.0, x, w, off, 0.0, y, transw=True, stream=stream)
            sg.sgemm_grouped_wgrad_tensors(1.0, y, x, off, 0.0, d, stream=stream)
            sg.check_status(stream=stream)
            got.append((y, d))
        for y, d in got[1:]:
            assert torch.equal(y, got[0][0]) and torch.equal(d, got[0][1])


@pytest.mark.parametrize("dtype,out", WGRAD)
@pytest.mark.parametrize("alpha", [float("inf"), float("nan"), -3e38])
@pytest.mark.parametrize("beta", [0.0, -2.0])
def test_alpha_has_no_part_in_empty_sums(dtype, out, alpha, beta):
    # A group without rows gets beta * D, and K = 0 beta * Y, whatever alpha is.
    torch = _torch()
    dt, ot = getattr(torch, dtype), getattr(torch, out)
    for sizes in ([70, 0, 5, 0], [0, 0], [0, 4001]):
        p, q = torch.ones(sum(sizes), 70, device="cuda").to(dt), torch.ones(sum(sizes), 136, device="cuda").to(dt)
        d0 = torch.randn(len(sizes), 70, 136, device="cuda").to(ot)
        d = d0.clone() if beta else torch.full_like(d0, float("nan"))
        sg.sgemm_grouped_wgrad_tensors(alpha, p, q, offsets_of(sizes), beta, d)
        sg.check_status()
        for e, n in enumerate(sizes):
            if n == 0:
                assert torch.equal(d[e], (beta * d0[e].float()).to(ot) if beta else torch.zeros_like(d[e]))
    y0 = torch.randn(9, 40, device="cuda").to(dt)
    y = y0.clone() if beta else torch.full_like(y0, float("nan"))
    sg.sgemm_grouped_tensors(alpha, y0[:, :0], torch.empty(2, 0, 40, device="cuda", dtype=dt), offsets_of([4, 5]), beta, y)
    sg.check_status()
    assert torch.equal(y, (beta * y0.float()).to(dt) if beta else torch.zeros_like(y))


def test_a_copy_without_memory_is_an_error():
    # Rows of one bfloat16 each, copied to rows of 16 bytes: eight times what the
    # weights take (51 GB), more than the GPU has. The call says so; nothing ran.
    torch = _torch()
    N, E = sg.SGEMM_GROUPED_MAX_DIM, 12
    w = torch.empty(E, N, 1, device="cuda", dtype=torch.bfloat16)
    x = torch.ones(1, 1, device="cuda", dtype=torch.bfloat16)
    y = torch.empty(1, N, device="cuda", dtype=torch.bfloat16)
    y[0, :1000] = 3.0
    off = torch.tensor([0] + [1] * E, dtype=torch.int32, device="cuda")
    assert E * N * 16 > torch.cuda.get_device_properties(0).total_memory
    try:
        with pytest.raises(sg.SgemmError) as error:
            sg.sgemm_grouped_tensors(1.0, x, w, off, 0.0, y, transw=True)
        assert error.value.code == sg.SGEMM_ERR_CUDA
        sg.check_status()
        assert torch.all(y[0, :1000] == 3.0)
    finally:
        del w, y
        torch.cuda.empty_cache()
    forward([70, 0, 200, 3], 131, 77, torch.bfloat16, True)
