"""Long sums of the expert-layer products on small integers and powers of two,
whose FP32 sums are exact in any order: every result has to be equal, so that a
part of a sum that is left out, or taken twice, shows at any length."""
import numpy as np
import pytest

import dense_fp32_matrix_strict_gb300 as sg

pytestmark = pytest.mark.gpu

TYPES = ["float32", "bfloat16"]


def _torch():
    import torch
    return torch


def shows_every_block(terms_of, length, block, dtype):
    """Leaving out any block of the sum changes the rounded result."""
    torch = _torch()
    whole = terms_of(0, length)
    for lo in range(0, length, block):
        less = whole - terms_of(lo, min(length, lo + block))
        assert not torch.equal(less.to(dtype), whole.to(dtype)), lo


def quantised(lead, N, K, group, pad, gen):
    """Codes, scales of 1/2 or 1, zero points, and the weights that they stand for."""
    torch = _torch()
    q = torch.randint(0, 256, (*lead, N, (K + 1) // 2 + pad), generator=gen, dtype=torch.uint8)
    s = torch.randint(0, 2, (*lead, N, -(-K // group)), generator=gen) * 0.5 + 0.5
    z = torch.randint(0, 16, s.shape, generator=gen, dtype=torch.uint8)
    codes = torch.stack([q & 15, q >> 4], -1).flatten(-2)[..., :K].double()
    of = torch.arange(K) // group
    return q, s, z, (codes - z.double()[..., of]) * s.double()[..., of], codes, of


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", [0, 1, 4])
@pytest.mark.parametrize("tokens,N,K,group", [(1, 18, 70001, 128), (6, 50, 16384, 64), (10, 70, 6184, 128),
                                              (16, 33, 9001, 32), (40, 20, 12345, 128), (8, 130, 8192, 64),
                                              (3, 333, 1531, 32), (33, 20, 1100, 64)])
def test_4_bit_products(tokens, N, K, group, pad, dtype):
    # At most 15 K in steps of 1/2: below 2^24 steps.
    torch = _torch()
    dt = getattr(torch, dtype)
    gen = torch.Generator().manual_seed(K + N)
    x = torch.randint(-1, 2, (tokens, K), generator=gen)
    q, s, z, w, codes, of = quantised((), N, K, group, pad, gen)
    xd = x.double()
    for zeros in (z, None):
        if zeros is None:
            w = (codes - 8) * s.double()[..., of]
        shows_every_block(lambda lo, hi: xd[:, lo:hi] @ w[:, lo:hi].t(), K, 512, dt)
        y = torch.empty(tokens, N, dtype=dt, device="cuda")
        sg.sgemv_w4_tensors(x.to(dt).cuda(), q.cuda()[:, :(K + 1) // 2], s.to(dt).cuda(), y, group,
                            zeros=None if zeros is None else zeros.cuda())
        sg.check_status()
        assert torch.equal(y.cpu(), (xd @ w.t()).to(dt))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,K,group", [(50, 40000, 64), (200, 1024, 32), (77, 999, 128)])
def test_4_bit_products_of_experts(N, K, group, dtype):
    torch = _torch()
    dt = getattr(torch, dtype)
    gen = torch.Generator().manual_seed(K)
    x = torch.randint(-1, 2, (3, K), generator=gen)
    q, s, z, w, _, _ = quantised((5,), N, K, group, 0, gen)
    ids = [4, -1, 0, 2, 2, 1]
    y = torch.empty(6, N, dtype=dt, device="cuda")
    sg.sgemv_w4_tensors(x.to(dt).cuda(), q.cuda(), s.to(dt).cuda(), y, group, zeros=z.cuda(),
                        experts=torch.tensor(ids, dtype=torch.int32).cuda())
    sg.check_status()
    for p, e in enumerate(ids):
        ref = torch.zeros(N).double() if e < 0 else w[e] @ x[p // 2].double()
        assert torch.equal(y[p].cpu(), ref.to(dt))
        if e >= 0:
            shows_every_block(lambda lo, hi: w[e][:, lo:hi] @ x[p // 2, lo:hi].double(), K, 512, dt)


def integers(shape, most, gen, dtype, shift):
    """Whole numbers up to `most`, `shift` elements into their buffer on the GPU."""
    torch = _torch()
    v = torch.randint(-most, most + 1, shape, generator=gen).to(dtype)
    buf = torch.zeros(v.numel() + shift, dtype=dtype, device="cuda")
    buf[shift:].copy_(v.flatten())
    return buf[shift:].view(shape)


def offsets_of(sizes):
    return _torch().tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=_torch().int32).cuda()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("transw", [False, True])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("sizes,N,K", [([40], 72, 4096), ([16, 0, 20], 200, 5000), ([300], 130, 2500), ([9], 500, 8190),
                                       ([8, 8, 8], 512, 2048), ([30, 0, 0, 3], 129, 9000), ([600, 0, 70], 260, 1032),
                                       ([1], 40, 30000)], ids=str)
def test_grouped_products(sizes, N, K, shift, transw, dtype):
    # At most 2 K, times a quarter: exact.
    torch = _torch()
    dt = getattr(torch, dtype)
    gen = torch.Generator().manual_seed(N + K)
    x = integers((sum(sizes), K), 1, gen, dt, shift)
    w = integers((len(sizes), N, K) if transw else (len(sizes), K, N), 2, gen, dt, shift)
    y0 = integers((sum(sizes), N), 3, gen, dt, shift)
    for alpha, beta in ((1.0, 0.0), (0.25, -2.0)):
        y = y0.clone()
        sg.sgemm_grouped_tensors(alpha, x, w, offsets_of(sizes), beta, y, transw=transw)
        sg.check_status()
        at = 0
        for e, n in enumerate(sizes):
            if n == 0:
                continue
            xd, wd = x[at:at + n].double(), w[e].double().t() if transw else w[e].double()
            ref = alpha * (xd @ wd) + beta * y0[at:at + n].double()
            assert torch.equal(y[at:at + n], ref.to(dt))
            if beta == 0:
                shows_every_block(lambda lo, hi: xd[:, lo:hi] @ wd[lo:hi], K, 32, dt)
            at += n


@pytest.mark.parametrize("dtype,out", [("float32", "float32"), ("bfloat16", "float32"), ("bfloat16", "bfloat16")])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("sizes,M,N", [([5000], 130, 70), ([3000, 0, 77], 64, 200), ([1027], 256, 128), ([9, 700, 65], 300, 136)],
                         ids=str)
def test_grouped_weight_gradients(sizes, M, N, shift, dtype, out):
    # At most the rows of a group, times a quarter: exact.
    torch = _torch()
    dt, ot = getattr(torch, dtype), getattr(torch, out)
    gen = torch.Generator().manual_seed(M + N)
    p, q = integers((sum(sizes), M), 1, gen, dt, shift), integers((sum(sizes), N), 1, gen, dt, shift)
    d0 = integers((len(sizes), M, N), 3, gen, ot, shift)
    for alpha, beta in ((1.0, 0.0), (0.25, -2.0)):
        d = d0.clone()
        sg.sgemm_grouped_wgrad_tensors(alpha, p, q, offsets_of(sizes), beta, d)
        sg.check_status()
        at = 0
        for e, n in enumerate(sizes):
            pd, qd = p[at:at + n].double(), q[at:at + n].double()
            assert torch.equal(d[e], (alpha * (pd.t() @ qd) + beta * d0[e].double()).to(ot))
            if beta == 0 and n > 0:
                shows_every_block(lambda lo, hi: pd[lo:hi].t() @ qd[lo:hi], n, 32, ot)
            at += n


@pytest.mark.parametrize("dtype,sizes,N,K", [
    # Tiles for 90 % of the workers, sums below and above what cutting the round costs,
    ("float32", [128] * 8, 2176, 1024), ("float32", [128] * 8, 2176, 4096),
    # for half and three quarters of them in 32-row tiles,
    ("float32", [40] * 4, 2432, 2048), ("float32", [40] * 6, 2432, 1024), ("float32", [40, 39, 41, 70], 2432, 600),
    # for more than half of the pairs, low tiles and tall ones, and after whole rounds.
    ("bfloat16", [32] * 4, 2816, 16384), ("bfloat16", [256] * 4, 2816, 4096), ("bfloat16", [70, 256, 31, 200], 5632, 4096),
], ids=str)
def test_last_rounds_whole_and_cut(dtype, sizes, N, K):
    torch = _torch()
    dt = getattr(torch, dtype)
    gen = torch.Generator(device="cuda").manual_seed(N + K)

    def integers_of(*shape, most):
        return torch.randint(-most, most + 1, shape, generator=gen, device="cuda").to(dt)

    x, w = integers_of(sum(sizes), K, most=1), integers_of(len(sizes), N, K, most=2)
    y = torch.full((sum(sizes), N), float("nan"), device="cuda", dtype=dt)
    sg.sgemm_grouped_tensors(1.0, x, w, offsets_of(sizes), 0.0, y, transw=True)
    sg.check_status()
    at = 0
    for e, n in enumerate(sizes):
        ref = x[at:at + n].double() @ w[e].double().t()
        assert torch.equal(y[at:at + n], ref.to(dt))
        at += n


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes,M,N", [([256, 256], 1024, 1024), ([2048, 100], 1024, 1536), ([300, 0, 2500], 1000, 2000)],
                         ids=str)
def test_last_rounds_of_weight_gradients_whole_and_cut(dtype, sizes, M, N):
    torch = _torch()
    dt = getattr(torch, dtype)
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    p, q = (torch.randint(-1, 2, (sum(sizes), n), generator=gen, device="cuda").to(dt) for n in (M, N))
    d = torch.full((len(sizes), M, N), float("nan"), device="cuda")
    sg.sgemm_grouped_wgrad_tensors(1.0, p, q, offsets_of(sizes), 0.0, d)
    sg.check_status()
    at = 0
    for e, n in enumerate(sizes):
        assert torch.equal(d[e], (p[at:at + n].double().t() @ q[at:at + n].double()).float())
        at += n
