"""The router against a plain implementation in 64 bits: choices, weights and
grouping exactly, gradients against the formula and against differences."""
import numpy as np
import pytest

import dense_fp32_matrix_strict_gb300 as sg

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def route(logits, top, renorm, ldl=None, stream=None):
    torch = _torch()
    T, E = logits.shape
    dev = torch.full((T, ldl or E), float("nan"), dtype=logits.dtype, device="cuda")
    dev[:, :E] = logits.cuda()
    out = {"weights": torch.full((T, top), -7.0, device="cuda"),
           "experts": torch.full((T, top), -7, dtype=torch.int32, device="cuda"),
           "offsets": torch.full((E + 1,), -7, dtype=torch.int32, device="cuda"),
           "order": torch.full((T * top,), -7, dtype=torch.int32, device="cuda"),
           "place": torch.full((T, top), -7, dtype=torch.int32, device="cuda")}
    sg.sgemm_route_tensors(dev[:, :E], out["weights"], out["experts"], out["offsets"], out["order"],
                           out["place"], renorm=renorm, stream=stream)
    sg.check_status(stream=stream)
    return dev[:, :E], {k: v.cpu().numpy() for k, v in out.items()}, out


def plain(logits, top, renorm):
    """Loops over tokens in float64."""
    z = logits.astype(np.float64)
    T, E = z.shape
    weights = np.zeros((T, top))
    experts = np.full((T, top), -1, np.int32)
    probs = np.zeros((T, E))
    for t in range(T):
        able = [e for e in range(E) if z[t, e] > -np.inf]
        able.sort(key=lambda e: (-z[t, e], e))
        picked = able[:top]
        if not picked:
            continue
        m = z[t, picked[0]]
        raised = {e: np.exp(z[t, e] - m) for e in able}
        total = sum(raised[e] for e in (picked if renorm else able))
        for j, e in enumerate(picked):
            experts[t, j] = e
            weights[t, j] = raised[e] / total
        for e in (picked if renorm else able):
            probs[t, e] = raised[e] / total
    flat = experts.reshape(-1)
    order = [p for e in range(E) for p in np.nonzero(flat == e)[0]]
    place = np.full(flat.shape, -1, np.int32)
    for row, p in enumerate(order):
        place[p] = row
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])])
    order = np.array(order + [-1] * (flat.size - len(order)), np.int32)
    return weights, experts, offsets, order, place.reshape(T, top), probs


def check_forward(got, want):
    weights, experts, offsets, order, place, _ = want
    assert np.array_equal(got["experts"], experts)
    assert np.array_equal(got["offsets"], offsets)
    assert np.array_equal(got["order"], order)
    assert np.array_equal(got["place"], place)
    # exp's argument error (one rounding of l - m, |l - m| < 2^7 here) and a sum of
    # up to E terms: 2^7 * 2^-24 + (E + 4) * 2^-24 relative covers both.
    E = len(offsets) - 1
    assert np.all(np.abs(got["weights"] - weights) <= (132 + E) * 2.0 ** -24 * weights + 1e-37)


SHAPES = [(1, 1, 1), (1, 8, 2), (33, 8, 8), (64, 128, 8), (128, 60, 6), (129, 60, 6), (1000, 32, 1),
          (4097, 256, 8), (700, 512, 3), (300, 1024, 32), (37, 33, 32), (9000, 7, 2)]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,top", SHAPES)
def test_choices_weights_and_grouping(T, E, top, renorm):
    torch = _torch()
    g = torch.Generator().manual_seed(T * 7 + E)
    logits = torch.randn(T, E, generator=g) * 3
    _, got, _ = route(logits, top, renorm, ldl=E + 5)
    check_forward(got, plain(logits.numpy(), top, renorm))


@pytest.mark.parametrize("T", [50, 2000])
def test_ties_go_to_the_lowest_index(T):
    torch = _torch()
    g = torch.Generator().manual_seed(T)
    logits = torch.randint(-2, 3, (T, 96), generator=g).to(torch.bfloat16)
    logits[:, ::5] *= -0.0                     # zeros of both signs are equal
    for renorm in (True, False):
        _, got, _ = route(logits, 8, renorm)
        check_forward(got, plain(logits.float().numpy(), 8, renorm))


@pytest.mark.parametrize("T", [70, 900])
def test_masked_logits(T):
    # -inf and NaN are never chosen, whole rows of them leave the token without
    # experts; the type's lowest value is a number like any other.
    torch = _torch()
    g = torch.Generator().manual_seed(T)
    logits = torch.randn(T, 40, generator=g)
    logits[torch.rand(T, 40, generator=g) < 0.8] = float("-inf")
    logits[3::7] = float("-inf")
    logits[5, :] = float("nan")
    logits[6, ::3] = float("nan")
    logits[8, :] = torch.finfo(torch.float32).min
    logits[9, :] = float("-inf")
    logits[9, 17] = torch.finfo(torch.float32).min
    for renorm in (True, False):
        dev, got, raw = route(logits, 5, renorm)
        ref = logits.numpy().copy()
        ref[np.isnan(ref)] = -np.inf
        want = plain(ref, 5, renorm)
        check_forward(got, want)
        dw = torch.randn(T, 5, generator=g).cuda()
        dl = torch.full((T, 40), 9.0, device="cuda")
        sg.sgemm_route_backward_tensors(dev, raw["experts"], dw, dl, renorm=renorm)
        sg.check_status()
        dl = dl.cpu().numpy()
        assert np.all(np.isfinite(dl))
        assert np.all(dl[want[5] == 0] == 0)


def test_infinite_logit_gives_nan_weights():
    torch = _torch()
    logits = torch.zeros(4, 8)
    logits[2, 3] = float("inf")
    _, got, _ = route(logits, 2, True)
    assert np.isnan(got["weights"][2]).all() and np.isfinite(got["weights"][[0, 1, 3]]).all()
    assert got["experts"][2, 0] == 3


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,top", [(1, 1, 1), (5, 40, 3), (600, 256, 8), (40, 1024, 32)])
def test_gradient_of_the_formula(T, E, top, renorm, dtype):
    torch = _torch()
    dt = getattr(torch, dtype)
    g = torch.Generator().manual_seed(E)
    logits = (torch.randn(T, E, generator=g) * 2).to(dt)
    dev, got, raw = route(logits, top, renorm, ldl=E + 3)
    want = plain(logits.float().numpy(), top, renorm)
    dw = torch.randn(T, top, generator=g)
    buf = torch.full((T, E + 2), 9.0, dtype=dt, device="cuda")
    sg.sgemm_route_backward_tensors(dev, raw["experts"], dw.cuda(), buf[:, :E], renorm=renorm)
    sg.check_status()
    p, ids = want[5], want[1]
    d = dw.numpy().astype(np.float64)
    s = (d * want[0]).sum(1, keepdims=True)
    up = np.zeros_like(p)
    np.put_along_axis(up, ids.astype(np.int64), d, 1)
    ref = p * (up - s)
    out = buf.float().cpu().numpy()
    assert np.all(out[:, E:] == 9.0)
    # p as the weights above; s sums top terms of size <= max|d|.
    size = p * (np.abs(d).max() * 2)
    tol = (200 + E) * 2.0 ** -24 * size + (2.0 ** -8 * np.abs(ref) if dtype == "bfloat16" else 0) + 1e-37
    assert np.all(np.abs(out[:, :E] - ref) <= tol)


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(renorm):
    torch = _torch()
    g = torch.Generator().manual_seed(2)
    E, top = 12, 3
    logits = torch.randn(1, E, generator=g)
    dw = torch.randn(1, top, generator=g)
    dev, _, raw = route(logits, top, renorm)
    dl = torch.empty(1, E, device="cuda")
    sg.sgemm_route_backward_tensors(dev, raw["experts"], dw.cuda(), dl, renorm=renorm)
    sg.check_status()
    ids = raw["experts"].cpu().numpy()[0]
    h = 1e-6
    for e in range(E):
        def loss(x):
            z = logits.numpy().astype(np.float64)[0].copy()
            z[e] += x
            r = np.exp(z - z.max())
            return float((dw.numpy()[0] * r[ids]).sum() / (r[ids].sum() if renorm else r.sum()))
        # The central difference's own error: h^2 times a third derivative of order 1,
        # and 2^-52 / h of rounding.
        assert abs((loss(h) - loss(-h)) / (2 * h) - float(dl[0, e])) <= 1e-9 + 300 * 2.0 ** -24


def test_bad_expert_index_is_reported():
    torch = _torch()
    logits = torch.randn(4, 8, device="cuda")
    ids = torch.tensor([[0, 1], [2, 8], [-1, 3], [4, 5]], dtype=torch.int32, device="cuda")
    dw = torch.ones(4, 2, device="cuda")
    dl = torch.empty(4, 8, device="cuda")
    sg.sgemm_route_backward_tensors(logits, ids, dw, dl)
    rc, bits = sg.sgemm_check_status(torch.cuda.current_stream().cuda_stream)
    assert rc == sg.SGEMM_ERR_DEVICE_CHECK and bits == 32
    assert torch.isfinite(dl).all()


def test_same_result_on_every_call_and_another_stream():
    torch = _torch()
    logits = torch.randn(5000, 128)
    _, first, _ = route(logits, 8, False)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        _, again, _ = route(logits, 8, False, stream=side)
    for k in first:
        assert np.array_equal(first[k], again[k])


def test_no_tokens():
    torch = _torch()
    _, got, _ = route(torch.empty(0, 8), 2, True)
    assert np.array_equal(got["offsets"], np.zeros(9, np.int32))


@pytest.mark.parametrize("T", [256, 257])
@pytest.mark.parametrize("E,top", [(300, 32), (128, 8)])
def test_many_equal_logits(T, E, top):
    # More equal keys than a warp has lanes, in both forms of the call.
    torch = _torch()
    logits = torch.zeros(T, E)
    logits[:, E // 2] = 1.0
    logits[1::2, : E // 3] = -1.0
    for renorm in (True, False):
        _, got, _ = route(logits, top, renorm)
        check_forward(got, plain(logits.numpy(), top, renorm))


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("T", [40, 700])
def test_weight_gradients_of_choices_without_an_expert_are_not_used(T, dtype, renorm):
    # No row stands behind such a choice, so what a caller has there may be
    # anything: the other choices' gradients are those of the formula.
    torch = _torch()
    dt = getattr(torch, dtype)
    E, top = 30, 6
    g = torch.Generator().manual_seed(T)
    logits = torch.randn(T, E, generator=g).to(dt)
    logits[torch.rand(T, E, generator=g) < 0.85] = float("-inf")
    logits[::9] = float("-inf")
    dev, got, raw = route(logits, top, renorm)
    want = plain(logits.float().numpy(), top, renorm)
    none = torch.from_numpy(want[1] < 0)
    assert bool(none.any()) and not bool(none.all())
    dw = torch.randn(T, top, generator=g)
    d = np.where(none, 0.0, dw.numpy().astype(np.float64))
    s = (d * want[0]).sum(1, keepdims=True)
    up = np.zeros_like(want[5])
    for t in range(T):
        for j in range(top):
            if want[1][t, j] >= 0:
                up[t, want[1][t, j]] = d[t, j]
    ref = want[5] * (up - s)
    # As for the gradient of the formula above: p, s and the output's rounding.
    size = want[5] * (np.abs(d).max() * 2)
    tol = (200 + E) * 2.0 ** -24 * size + (2.0 ** -8 * np.abs(ref) if dtype == "bfloat16" else 0) + 1e-37
    for bad in (float("nan"), float("inf"), float("-inf")):
        dl = torch.full((T, E), 9.0, dtype=dt, device="cuda")
        sg.sgemm_route_backward_tensors(dev, raw["experts"], dw.masked_fill(none, bad).cuda(), dl, renorm=renorm)
        sg.check_status()
        assert np.all(np.abs(dl.float().cpu().numpy() - ref) <= tol)


@pytest.mark.parametrize("renorm", [True, False])
def test_weight_gradient_of_a_masked_logit_is_not_used(renorm):
    # A choice whose logit is -inf or NaN has weight 0, whoever chose it.
    torch = _torch()
    logits = torch.zeros(3, 8)
    logits[0, 2], logits[1, 2] = float("-inf"), float("nan")
    ids = torch.tensor([[2, 5]] * 3, dtype=torch.int32, device="cuda")
    out = []
    for dw in (0.0, float("nan"), float("inf")):
        dl = torch.empty(3, 8, device="cuda")
        sg.sgemm_route_backward_tensors(logits.cuda(), ids, torch.tensor([[dw, 1.5]] * 3).cuda(), dl, renorm=renorm)
        sg.check_status()
        out.append(dl[:2])
    assert torch.isfinite(out[0]).all()
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
