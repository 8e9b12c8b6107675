"""Products with 4-bit weights against the definition in 64 bits."""
import numpy as np
import pytest

import dense_fp32_matrix_strict_gb300 as sg

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def make(tokens, N, K, group, dtype, zeros, experts=0, seed=0, pad=0):
    """Host tensors; Q's rows lie `pad` bytes further apart than they are long."""
    torch = _torch()
    g = torch.Generator().manual_seed(seed + N + K)
    lead = (experts,) if experts else ()
    nb, ng = (K + 1) // 2, -(-K // group)
    x = torch.randn(tokens, K, generator=g).to(dtype)
    q = torch.randint(0, 256, lead + (N, nb + pad), generator=g, dtype=torch.uint8)
    s = (torch.rand(*lead, N, ng, generator=g) * 0.02 + 0.001).to(dtype)
    z = torch.randint(0, 16, lead + (N, ng), generator=g, dtype=torch.uint8) if zeros else None
    return x, q, s, z


def reference(x, q, s, z, group, K):
    """(y, sum of |terms|) for one set of weights."""
    q = q[:, :(K + 1) // 2].numpy().astype(np.int64)
    code = np.empty((q.shape[0], 2 * q.shape[1]), np.int64)
    code[:, 0::2] = q & 15
    code[:, 1::2] = q >> 4
    of = np.arange(K) // group
    zero = z.numpy().astype(np.int64)[:, of] if z is not None else 8
    w = s.double().numpy()[:, of] * (code[:, :K] - zero)
    x = x.double().numpy()
    return x @ w.T, np.abs(x) @ np.abs(w).T


def close(y, ref, size, dtype, K):
    torch = _torch()
    # FP32 sums of exact products (4 K 2^-24 sum|terms|), then the output's rounding.
    tol = 4 * max(K, 8) * 2.0 ** -24 * size + 1e-37
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref)
    return bool(np.all(np.abs(y.double().cpu().numpy() - ref) <= tol))


def call(x, q, s, z, group, K, N, pairs=None, experts=None, pad_y=3):
    torch = _torch()
    pairs = pairs or x.shape[0]
    buf = torch.full((pairs, N + pad_y), -5.0, dtype=x.dtype, device="cuda")
    sg.sgemv_w4_tensors(x.cuda(), q.cuda()[..., :(K + 1) // 2], s.cuda(), buf[:, :N], group,
                        zeros=None if z is None else z.cuda(), experts=experts)
    sg.check_status()
    assert torch.all(buf[:, N:] == -5.0)
    return buf[:, :N]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("tokens,N,K,pad", [(1, 1, 1, 0), (1, 17, 31, 0), (1, 64, 512, 0), (2, 100, 513, 15),
                                            (3, 333, 1531, 0), (5, 256, 4096, 0), (8, 40, 2000, 8),
                                            (9, 128, 1024, 0), (16, 48, 700, 2), (33, 20, 1100, 0)])
def test_products(tokens, N, K, pad, group, dtype):
    dtype = getattr(_torch(), dtype)
    for zeros in (False, True):
        x, q, s, z = make(tokens, N, K, group, dtype, zeros, pad=pad)
        y = call(x, q, s, z, group, K, N)
        assert close(y, *reference(x, q, s, z, group, K), dtype, K)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("K", [12288, 16384])
def test_long_inputs(K, dtype):
    dtype = getattr(_torch(), dtype)
    x, q, s, z = make(6, 50, K, 64, dtype, True)
    y = call(x, q, s, z, 64, K, 50)
    assert close(y, *reference(x, q, s, z, 64, K), dtype, K)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("tokens,N,K", [(10, 70, 6184), (16, 33, 9001), (40, 20, 12345), (1, 18, 70001)])
def test_long_inputs_of_many_tokens(tokens, N, K, dtype):
    # k in slabs, their sums joined.
    dtype = getattr(_torch(), dtype)
    x, q, s, z = make(tokens, N, K, 128, dtype, True)
    y = call(x, q, s, z, 128, K, N)
    assert close(y, *reference(x, q, s, z, 128, K), dtype, K)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_long_inputs_of_experts(dtype):
    torch = _torch()
    dtype = getattr(torch, dtype)
    K, N = 40000, 50
    x, q, s, z = make(2, N, K, 64, dtype, False, experts=3)
    ids = torch.tensor([2, -1, 0, 1], dtype=torch.int32)
    y = call(x, q, s, z, 64, K, N, pairs=4, experts=ids.cuda())
    assert torch.all(y[1] == 0)
    for p in (0, 2, 3):
        e = int(ids[p])
        ref, size = reference(x[p // 2:p // 2 + 1], q[e], s[e], None, 64, K)
        assert close(y[p:p + 1], ref, size, dtype, K)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("tokens,repeat,N,K", [(1, 1, 64, 512), (2, 8, 200, 1024), (3, 2, 77, 999)])
def test_experts(tokens, repeat, N, K, dtype):
    torch = _torch()
    dtype = getattr(torch, dtype)
    E, group = 7, 32
    x, q, s, z = make(tokens, N, K, group, dtype, True, experts=E)
    pairs = tokens * repeat
    ids = torch.randint(0, E, (pairs,), generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    ids[-1] = -1
    y = call(x, q, s, z, group, K, N, pairs=pairs, experts=ids.cuda())
    for p, e in enumerate(ids.tolist()):
        if e < 0:
            assert torch.all(y[p] == 0)
            continue
        ref, size = reference(x[p // repeat:p // repeat + 1], q[e], s[e], z[e], group, K)
        assert close(y[p:p + 1], ref, size, dtype, K)


def test_bad_expert_index_is_reported():
    torch = _torch()
    x, q, s, z = make(2, 40, 128, 32, torch.float32, False, experts=3)
    y = torch.full((2, 40), 9.0, device="cuda")
    ids = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    sg.sgemv_w4_tensors(x.cuda(), q.cuda(), s.cuda(), y, 32, experts=ids)
    rc, bits = sg.sgemm_check_status(torch.cuda.current_stream().cuda_stream)
    assert rc == sg.SGEMM_ERR_DEVICE_CHECK and bits == 32
    assert torch.all(y[0] == 0)
    assert close(y[1:], *reference(x[1:], q[1], s[1], None, 32, 128), torch.float32, 128)


def test_float32_inputs_keep_their_low_bits():
    # Values that differ in the last bits of their significands, in all three pieces.
    torch = _torch()
    K = 64
    x = (1.0 + torch.arange(K) * 2.0 ** -23).view(1, K).float()
    q = torch.full((1, K // 2), 0x79, dtype=torch.uint8)        # +1, -1, +1, -1, ...
    s = torch.ones(1, 1)
    y = call(x, q, s, None, 64, K, 1)
    assert float(y) == -(K // 2) * 2.0 ** -23


def test_infinities_and_nan_reach_their_rows():
    torch = _torch()
    x, q, s, _ = make(3, 20, 256, 64, torch.float32, False)
    q[:] = 0x99                                                # every weight +1
    x[1, 100] = float("inf")
    x[2, 7] = float("nan")
    x[0, 3] = 3e38
    y = call(x, q, s, None, 64, 256, 20).cpu()
    assert torch.isfinite(y[0]).all() and torch.all(y[1] == float("inf")) and torch.isnan(y[2]).all()


def test_no_inputs_give_zeros():
    torch = _torch()
    y = call(torch.empty(2, 0), torch.empty(5, 0, dtype=torch.uint8), torch.empty(5, 0), None, 32, 0, 5)
    assert torch.all(y == 0)


def test_same_bits_on_every_call_and_another_stream():
    torch = _torch()
    x, q, s, z = make(4, 500, 3000, 64, torch.float32, True)
    first = call(x, q, s, z, 64, 3000, 500).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = call(x, q, s, z, 64, 3000, 500)
    side.synchronize()
    assert torch.equal(first, again)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("offset,ldq,K", [(0, 0, 600), (1, 0, 513), (3, 301, 600), (4, 300, 599), (7, 0, 1031),
                                          (8, 520, 1030), (12, 516, 1025), (15, 529, 1058), (16, 528, 1024)])
def test_weights_and_inputs_at_any_alignment(offset, ldq, K, dtype):
    # Rows of Q and X anywhere in a larger buffer whose other bytes change.
    torch = _torch()
    dtype = getattr(torch, dtype)
    N, E, group, nb = 37, 2, 32, (K + 1) // 2
    ldq = ldq or nb
    x, q, s, z = make(2, N, K, group, dtype, True, experts=E)
    ids = torch.tensor([1, 0], dtype=torch.int32)
    got = []
    for fill in (0, 255):
        buf = torch.full((offset + E * N * ldq + 64,), fill, dtype=torch.uint8)
        rows = buf.as_strided((E, N, nb), (N * ldq, ldq, 1), offset)
        rows.copy_(q)
        xbuf = torch.full((offset + 2 * (K + 3) + 8,), float("nan"), dtype=dtype)
        xs = xbuf.as_strided((2, K), (K + 3, 1), offset)
        xs.copy_(x)
        y = torch.empty(2, N, dtype=dtype, device="cuda")
        sg.sgemv_w4_tensors(xbuf.cuda().as_strided((2, K), (K + 3, 1), offset),
                            buf.cuda().as_strided((E, N, nb), (N * ldq, ldq, 1), offset), s.cuda(), y, group,
                            zeros=z.cuda(), experts=ids.cuda())
        sg.check_status()
        got.append(y.cpu())
    assert torch.equal(got[0], got[1])
    for p, e in enumerate(ids.tolist()):
        ref, size = reference(x[p:p + 1], q[e], s[e], z[e], group, K)
        assert close(got[0][p:p + 1], ref, size, dtype, K)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("tokens,N,K", [(8, 130, 8192), (10, 33, 6144), (16, 500, 4096), (3, 700, 6200), (12, 16, 5632)])
def test_few_rows_of_long_inputs(tokens, N, K, dtype):
    # Sums in slabs where one slab would fit too, warps shared out over the units.
    dtype = getattr(_torch(), dtype)
    x, q, s, z = make(tokens, N, K, 128, dtype, False)
    y = call(x, q, s, z, 128, K, N)
    assert close(y, *reference(x, q, s, z, 128, K), dtype, K)


# Calls one entry point `loops` times from each of `n` threads without
# Python's lock between them; returns how many calls were refused.
CALLER = r"""
#include <pthread.h>
#include <stdint.h>
typedef int (*Entry)(int, int64_t, int64_t, int64_t, int64_t, int64_t, const void*, int64_t, const void*, int64_t,
                     int64_t, const void*, const void*, int64_t, const void*, void*, int64_t, void*);
struct Args { int64_t K; const void *x, *q, *s; void *y, *stream; };
static Entry entry;
static int loops, rows, group;
static pthread_barrier_t start;
static void* work(void* arg) {
    const struct Args* a = arg;
    intptr_t refused = 0;
    pthread_barrier_wait(&start);
    for (int i = 0; i < loops; ++i)
        refused += entry(1, 1, 1, rows, a->K, group, a->x, a->K, a->q, a->K / 2, 0, a->s, 0, 1, 0, a->y, rows,
                         a->stream) != 0;
    return (void*)refused;
}
int call_from_threads(void* fn, int n, int times, int N, int per, const struct Args* args) {
    pthread_t threads[16];
    int refused = 0;
    entry = (Entry)fn; loops = times; rows = N; group = per;
    pthread_barrier_init(&start, 0, n);
    for (int i = 0; i < n; ++i) pthread_create(&threads[i], 0, work, (void*)&args[i]);
    for (int i = 0; i < n; ++i) {
        void* r;
        pthread_join(threads[i], &r);
        refused += (int)(intptr_t)r;
    }
    pthread_barrier_destroy(&start);
    return refused;
}
"""


def test_host_threads_call_concurrently(tmp_path):
    # Threads whose calls need different amounts of shared memory of the same
    # kernel: no call is refused for another's sake, and each gets its result.
    import ctypes
    import subprocess
    torch = _torch()
    (tmp_path / "caller.c").write_text(CALLER)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-pthread", "-o", str(tmp_path / "caller.so"),
                    str(tmp_path / "caller.c")], check=True)
    caller = ctypes.CDLL(str(tmp_path / "caller.so"))

    class Args(ctypes.Structure):
        _fields_ = [("K", ctypes.c_int64)] + [(n, ctypes.c_void_p) for n in ("x", "q", "s", "y", "stream")]

    N, group, kept = 48, 128, []
    sizes = (512, 1024, 4096, 6144)
    args = (Args * len(sizes))()
    for i, K in enumerate(sizes):
        x, q, s, _ = make(1, N, K, group, torch.bfloat16, False, seed=i)
        want = call(x, q, s, None, group, K, N).contiguous()
        x, q, s, y, stream = x.cuda(), q.cuda(), s.cuda(), torch.empty_like(want), torch.cuda.Stream()
        args[i] = Args(K, x.data_ptr(), q.data_ptr(), s.data_ptr(), y.data_ptr(), stream.cuda_stream)
        kept.append((x, q, s, y, stream, want))
    torch.cuda.synchronize()
    entry = ctypes.cast(sg.load().sgemv_w4, ctypes.c_void_p)
    assert caller.call_from_threads(entry, len(sizes), 2000, N, group, args) == 0
    sg.check_status()
    torch.cuda.synchronize()
    for x, q, s, y, stream, want in kept:
        assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_every_code_with_every_zero_point(group, dtype):
    # q - z for all 16 codes and 256 zero points: integers below 2^8, which the
    # unpacking and the sum of a one-input token keep exactly.
    torch = _torch()
    dtype = getattr(torch, dtype)
    N, K = 256, 16
    x = torch.eye(K).to(dtype)
    q = torch.tensor([2 * i | (2 * i + 1) << 4 for i in range(8)], dtype=torch.uint8).repeat(N, 1)
    z = torch.arange(N, dtype=torch.uint8).view(N, 1)
    y = call(x, q, torch.ones(N, 1, dtype=dtype), z, group, K, N)
    assert torch.equal(y.cpu().float(), torch.arange(K).view(K, 1).float() - torch.arange(N).float())
