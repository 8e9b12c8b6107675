"""A mixture-of-experts layer on the library's entry points: forward and
backward for training, and single-token decode with 4-bit weights.

    logits = x @ router.T                          sgemm
    weights, experts, offsets, order, place        sgemm_route
    h = x[token of each row] @ up[e].T             sgemm_grouped
    y = relu(h) @ down[e].T                        sgemm_grouped
    out[t] = sum_j weights[t, j] * y[place[t, j]]      over the choices with an expert

Nothing waits for the device between the calls: the sizes of the groups stay
there. Torch does the gathers, the activation and the weighted sums. Run it
(python examples/expert_layer.py) for one training step and one decode step
with their times.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_fp32_matrix_strict_gb300 as sg  # noqa: E402


class ExpertLayer:
    """router (E, H) float32; up (E, F, H) and down (E, H, F) of `dtype`; top experts per token."""

    def __init__(self, hidden, inner, experts, top, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=gen, device="cuda") * shape[-1] ** -0.5

        self.top = top
        self.router = normal(experts, hidden)
        self.up = normal(experts, inner, hidden).to(dtype)
        self.down = normal(experts, hidden, inner).to(dtype)

    def route(self, x):
        tokens, experts = x.shape[0], self.router.shape[0]
        r = {"logits": torch.empty(tokens, experts, device="cuda"),
             "weights": torch.empty(tokens, self.top, device="cuda"),
             "experts": torch.empty(tokens, self.top, dtype=torch.int32, device="cuda"),
             "offsets": torch.empty(experts + 1, dtype=torch.int32, device="cuda"),
             "order": torch.empty(tokens * self.top, dtype=torch.int32, device="cuda"),
             "place": torch.empty(tokens, self.top, dtype=torch.int32, device="cuda")}
        sg.sgemm_tensors(1.0, x.float(), self.router, 0.0, r["logits"], transb=True)
        sg.sgemm_route_tensors(r["logits"], r["weights"], r["experts"], r["offsets"], r["order"], r["place"])
        return r

    def forward(self, x):
        """Returns the output and what backward needs."""
        r = self.route(x)
        rows = x[r["order"] // self.top]
        h = torch.empty(rows.shape[0], self.up.shape[1], dtype=x.dtype, device="cuda")
        sg.sgemm_grouped_tensors(1.0, rows, self.up, r["offsets"], 0.0, h, transw=True)
        a = h.relu()
        y = torch.empty_like(rows)
        sg.sgemm_grouped_tensors(1.0, a, self.down, r["offsets"], 0.0, y, transw=True)
        out = (rows_of(y, r["place"]) * r["weights"][:, :, None]).sum(1).to(x.dtype)
        return out, (x, r, rows, h, a, y)

    def backward(self, dout, kept):
        """Gradients of x, router, up and down; the weights' in float32."""
        x, r, rows, h, a, y = kept
        off, order, place = r["offsets"], r["order"], r["place"]
        dweights = (dout.float()[:, None, :] * rows_of(y, place)).sum(-1)
        dy = (dout.float()[order // self.top] * r["weights"].flatten()[order][:, None]).to(x.dtype)
        ddown = torch.empty(self.down.shape, device="cuda")
        sg.sgemm_grouped_wgrad_tensors(1.0, dy, a, off, 0.0, ddown)
        da = torch.empty_like(a)
        sg.sgemm_grouped_tensors(1.0, dy, self.down, off, 0.0, da)
        dh = da * (h > 0)
        dup = torch.empty(self.up.shape, device="cuda")
        sg.sgemm_grouped_wgrad_tensors(1.0, dh, rows, off, 0.0, dup)
        drows = torch.empty_like(rows)
        sg.sgemm_grouped_tensors(1.0, dh, self.up, off, 0.0, drows)
        dlogits = torch.empty_like(r["logits"])
        sg.sgemm_route_backward_tensors(r["logits"], r["experts"], dweights, dlogits)
        dx = rows_of(drows, place).sum(1)
        sg.sgemm_tensors(1.0, dlogits, self.router, 1.0, dx)
        drouter = torch.empty_like(self.router)
        sg.sgemm_tensors(1.0, dlogits, x.float(), 0.0, drouter, transa=True)
        return dx.to(x.dtype), drouter, dup, ddown

    def quantise(self, group=64):
        """up and down in 4 bits, with scales and zero points for decode()."""
        self.group = group
        self.q = {name: quantise(w, group) for name, w in (("up", self.up), ("down", self.down))}

    def decode(self, x):
        """The layer's output for a few tokens, weights in 4 bits."""
        r = self.route(x)
        ids = r["experts"].view(-1)
        q, s, z = self.q["up"]
        h = torch.empty(ids.numel(), q.shape[1], dtype=x.dtype, device="cuda")
        sg.sgemv_w4_tensors(x, q, s, h, self.group, zeros=z, experts=ids)
        q, s, z = self.q["down"]
        y = torch.empty(ids.numel(), q.shape[1], dtype=x.dtype, device="cuda")
        sg.sgemv_w4_tensors(h.relu(), q, s, y, self.group, zeros=z, experts=ids)
        y = y.view(x.shape[0], self.top, -1).float()
        return (y * r["weights"][:, :, None]).sum(1).to(x.dtype)


def rows_of(y, place):
    """The rows of y (rows, N) at place (tokens, top) in float32; zeros for a choice without an
    expert (place -1), whose row no product wrote."""
    return y[place].float().masked_fill((place < 0)[:, :, None], 0.0)


def quantise(w, group):
    """w (..., N, K), K a multiple of group: codes (..., N, K / 2), scales and zero points."""
    g = w.float().unflatten(-1, (-1, group))
    low, high = g.amin(-1).clamp(max=0.0), g.amax(-1).clamp(min=0.0)
    scale = ((high - low) / 15).clamp(min=1e-8).to(w.dtype)
    zero = (-low / scale.float()).round().clamp(0, 15)
    code = (g / scale.float()[..., None] + zero[..., None]).round().clamp(0, 15).flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale, zero.to(torch.uint8)


def dequantise(q, scale, zero, group):
    code = torch.stack([q & 15, q >> 4], -1).flatten(-2).float().unflatten(-1, (-1, group))
    return ((code - zero.float()[..., None]) * scale.float()[..., None]).flatten(-2)


def _milliseconds(f):
    for _ in range(3):
        f()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(10):
        f()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / 10


def main():
    layer = ExpertLayer(hidden=4096, inner=2048, experts=32, top=4)
    x = torch.randn(4096, 4096, device="cuda").bfloat16()

    def step():
        out, kept = layer.forward(x)
        return layer.backward(out, kept)

    print(f"training step, 4096 tokens: {_milliseconds(step):.3f} ms")
    layer.quantise()
    print(f"decode, 2 tokens: {_milliseconds(lambda: layer.decode(x[:2])):.3f} ms")
    sg.check_status()


if __name__ == "__main__":
    main()
