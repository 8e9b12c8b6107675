"""The example's expert layer, its operators together: against autograd in
64 bits, and the decode form against the dequantised weights."""
import importlib.util
import os

import pytest

import dense_fp32_matrix_strict_gb300 as sg

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def reference(layer, x, experts, up, down):
    """Output in float64 for the experts that were chosen, differentiable."""
    import torch
    logits = x @ layer["router"].t()
    chosen = logits.gather(1, experts.long())
    weights = torch.softmax(chosen, 1)
    out = torch.zeros_like(x)
    for j in range(experts.shape[1]):
        for e in range(up.shape[0]):
            t = experts[:, j] == e
            out = out.index_add(0, t.nonzero()[:, 0],
                                (torch.relu(x[t] @ up[e].t()) @ down[e].t()) * weights[t, j, None])
    return out


def relative(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("tokens,hidden,inner,experts,top", [(50, 64, 96, 6, 2), (300, 100, 37, 16, 4)])
def test_training_step_in_float32(tokens, hidden, inner, experts, top):
    import torch
    layer = example().ExpertLayer(hidden, inner, experts, top, dtype=torch.float32)
    x = torch.randn(tokens, hidden, device="cuda")
    out, kept = layer.forward(x)
    dout = torch.randn_like(out)
    grads = layer.backward(dout, kept)
    sg.check_status()
    leaves = [t.double().requires_grad_() for t in (x, layer.router, layer.up, layer.down)]
    ref = reference({"router": leaves[1]}, leaves[0], kept[1]["experts"], leaves[2], leaves[3])
    # Sums of at most a few hundred FP32 terms in a row of four products:
    # 4 * sqrt(300) * 2^-24 relative in the mean, taken ten times over.
    assert relative(out, ref.detach()) <= 4e-5
    ref.backward(dout.double())
    for got, leaf in zip(grads, leaves):
        assert relative(got, leaf.grad) <= 4e-5


def test_training_step_in_bfloat16():
    import torch
    layer = example().ExpertLayer(256, 512, 8, 2)
    x = torch.randn(400, 256, device="cuda").bfloat16()
    out, kept = layer.forward(x)
    dout = torch.randn(400, 256, device="cuda").bfloat16()
    grads = layer.backward(dout, kept)
    sg.check_status()
    leaves = [t.double().requires_grad_() for t in (x, layer.router, layer.up, layer.down)]
    ref = reference({"router": leaves[1]}, leaves[0], kept[1]["experts"], leaves[2], leaves[3])
    # Each tensor between two products is rounded to 8 bits of significand
    # (2^-9 relative, half of that in the mean); at most five roundings meet.
    assert relative(out, ref.detach()) <= 5 * 2.0 ** -9
    ref.backward(dout.double())
    for got, leaf in zip(grads, leaves):
        assert relative(got, leaf.grad) <= 5 * 2.0 ** -9


def test_decode_is_the_layer_with_dequantised_weights():
    import torch
    m = example()
    layer = m.ExpertLayer(256, 384, 8, 2, dtype=torch.float32)
    layer.quantise(64)
    x = torch.randn(3, 256, device="cuda")
    got = layer.decode(x)
    experts = layer.route(x)["experts"]
    sg.check_status()
    up, down = (m.dequantise(*layer.q[n], 64).double() for n in ("up", "down"))
    ref = reference({"router": layer.router.double()}, x.double(), experts, up, down)
    assert relative(got, ref) <= 4e-5
    # And the quantised layer is near the layer.
    assert relative(got, layer.forward(x)[0].double()) <= 0.3


def test_masked_experts_leave_no_trace(monkeypatch):
    # Tokens with fewer experts than choices, one with none: rows that no group
    # writes are uninitialised (here NaN) and reach neither output nor gradient.
    import torch
    m = example()
    layer = m.ExpertLayer(64, 96, 6, 3, dtype=torch.float32)
    gen = torch.Generator().manual_seed(3)
    masked = (torch.rand(50, 6, generator=gen) < 0.6).cuda()
    masked[7] = True
    masked[8] = False
    route, empty, empty_like = sg.sgemm_route_tensors, torch.empty, torch.empty_like

    def spoiled(t):
        return t.fill_(float("nan")) if t.is_floating_point() else t

    def masked_route(logits, *outputs):
        logits.masked_fill_(masked[:logits.shape[0]], float("-inf"))
        route(logits, *outputs)

    with monkeypatch.context() as patch:
        patch.setattr(torch, "empty", lambda *a, **k: spoiled(empty(*a, **k)))
        patch.setattr(torch, "empty_like", lambda *a, **k: spoiled(empty_like(*a, **k)))
        patch.setattr(m.sg, "sgemm_route_tensors", masked_route)
        x = torch.randn(50, 64, device="cuda")
        out, kept = layer.forward(x)
        dout = torch.randn(50, 64, device="cuda")
        grads = layer.backward(dout, kept)
        layer.quantise(32)
        few = layer.decode(x[:9])
    sg.check_status()
    leaves = [t.double().requires_grad_() for t in (x, layer.router, layer.up, layer.down)]
    logits = (leaves[0] @ leaves[1].t()).masked_fill(masked, float("-inf"))
    ref = torch.zeros_like(leaves[0])
    experts = kept[1]["experts"]
    assert bool((experts[7] < 0).all()) and bool((experts[8] >= 0).all())
    for t in range(50):
        ids = [e for e in experts[t].tolist() if e >= 0]
        if not ids:
            continue
        weights = torch.softmax(logits[t, ids], 0)
        row = sum(w * (torch.relu(leaves[0][t] @ leaves[2][e].t()) @ leaves[3][e].t())
                  for w, e in zip(weights, ids))
        ref = ref.index_add(0, torch.tensor([t], device="cuda"), row[None])
    # As for the training step in float32 above.
    assert torch.all(out[7] == 0) and relative(out, ref.detach()) <= 4e-5
    ref.backward(dout.double())
    for got, leaf in zip(grads, leaves):
        assert relative(got, leaf.grad) <= 4e-5
    assert torch.isfinite(few).all() and torch.all(few[7] == 0)


def test_host_threads_train_concurrently():
    # Each thread runs steps of its own sizes and type on its own stream; all
    # get the bits of a run by themselves.
    import threading

    import torch
    m = example()
    shapes = [(50, 64, 96, 6, 2, torch.float32), (300, 100, 37, 16, 4, torch.bfloat16),
              (700, 256, 384, 8, 2, torch.bfloat16), (20, 512, 256, 12, 3, torch.float32)]
    cases = []
    for i, (tokens, hidden, inner, experts, top, dtype) in enumerate(shapes):
        layer = m.ExpertLayer(hidden, inner, experts, top, dtype=dtype, seed=i)
        x = torch.randn(tokens, hidden, device="cuda").to(dtype)

        def step(layer=layer, x=x):
            out, kept = layer.forward(x)
            return (out, *layer.backward(torch.ones_like(out), kept))

        cases.append((step, [t.clone() for t in step()], torch.cuda.Stream()))
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(len(cases))

    def work(step, want, stream):
        try:
            start.wait()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got = step()
                stream.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        except Exception as e:                  # reported below, on the main thread
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    sg.check_status()
