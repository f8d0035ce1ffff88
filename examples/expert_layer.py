"""An expert layer from its training to its answers, with the library's operators.

A layer of experts y = W2_e gelu(W1_e x), each token sent to `top` of them, learns
to reproduce the outputs of a fixed random layer:

  forward   grouped_gemm, twice
  backward  grouped_gemm with transposed weights, grouped_gemm_wgrad
  update    newton_schulz of the momentum, one batch over the experts
  answer    w4_gemm on the weights quantised to 4 bits, token by token

PyTorch routes the tokens (top-k, sort) and does the element-wise parts.

    python examples/expert_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_gemm_bf16_gb300 as dg  # noqa: E402


def route(x, gate, top):
    """Rows of x in the order of their experts: (token of each row, its share,
    offsets of the experts' rows)."""
    share, expert = torch.softmax(x.float() @ gate, dim=-1).topk(top, dim=-1)
    share = (share / share.sum(dim=-1, keepdim=True)).reshape(-1)
    order = torch.argsort(expert.reshape(-1), stable=True)
    counts = torch.bincount(expert.reshape(-1), minlength=gate.shape[1])
    offsets = torch.zeros(gate.shape[1] + 1, dtype=torch.int32, device=x.device)
    offsets[1:] = torch.cumsum(counts, 0)
    return order // top, share[order], offsets


def gelu(h):
    return torch.nn.functional.gelu(h.float(), approximate="tanh").to(h.dtype)


def gelu_grad(h, g):
    x = h.float()
    c, k = 0.7978845608028654, 0.044715
    t = torch.tanh(c * (x + k * x ** 3))
    return (g.float() * (0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * k * x * x))).to(h.dtype)


def layer(x, w1, w2, plan):
    """Outputs per token, and what the backward pass needs."""
    token, share, offsets = plan
    rows = x[token]
    h = dg.grouped_gemm(rows, w1, offsets)
    z = gelu(h)
    y = dg.grouped_gemm(z, w2, offsets)
    out = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
    out.index_add_(0, token, y.float() * share[:, None])
    return out, (rows, h, z)


def gradients(d_out, saved, w2, plan):
    token, share, offsets = plan
    rows, h, z = saved
    d_y = (d_out[token] * share[:, None]).to(rows.dtype)
    d_w2 = dg.grouped_gemm_wgrad(z, d_y, offsets, out_dtype=torch.float32)
    d_h = gelu_grad(h, dg.grouped_gemm(d_y, w2.transpose(1, 2), offsets))
    d_w1 = dg.grouped_gemm_wgrad(rows, d_h, offsets, out_dtype=torch.float32)
    return d_w1, d_w2


def quantise(w, group=64):
    """[experts, K, N] weights to 4 bits along K: (q [experts, N, K / 2], scales, zeros)."""
    t = w.transpose(1, 2).float()
    e, n, k = t.shape
    t = t.reshape(e, n, k // group, group)
    lo, hi = t.amin(-1, keepdim=True).clamp(max=0), t.amax(-1, keepdim=True).clamp(min=0)
    scale = ((hi - lo) / 15).clamp(min=1e-8).to(w.dtype).float()
    zero = (-lo / scale).round().clamp(0, 15)
    q = (t / scale + zero).round().clamp(0, 15).to(torch.uint8).reshape(e, n, k)
    return ((q[..., 0::2] | (q[..., 1::2] << 4)).contiguous(), scale.squeeze(-1).to(w.dtype),
            zero.squeeze(-1).to(torch.uint8))


def main(tokens=4096, width=1024, hidden=2048, experts=16, top=2, steps=30, quiet=False):
    """Returns the first and the last step's loss, and the relative distance of the
    4-bit layer's answers from the 16-bit layer's."""
    gen = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * scale

    gate = normal(width, experts, scale=width ** -0.5)
    target = [normal(experts, width, hidden, scale=width ** -0.5).bfloat16(),
              normal(experts, hidden, width, scale=hidden ** -0.5).bfloat16()]
    master = [normal(experts, width, hidden, scale=width ** -0.5),
              normal(experts, hidden, width, scale=hidden ** -0.5)]
    momentum = [torch.zeros_like(w) for w in master]
    losses = []
    for step in range(steps):
        x = normal(tokens, width).bfloat16()
        plan = route(x, gate, top)
        w1, w2 = (w.bfloat16() for w in master)
        want, _ = layer(x, *target, plan)
        out, saved = layer(x, w1, w2, plan)
        diff = out - want
        losses.append(float((diff * diff).mean()))
        for w, m, g in zip(master, momentum, gradients(diff * (2.0 / diff.numel()), saved, w2, plan)):
            m.mul_(0.9).add_(g)
            # a step of fixed size in every direction of the weights
            w.add_(dg.newton_schulz(m).float(), alpha=-0.02 * max(1.0, w.shape[1] / w.shape[2]) ** 0.5)
        if not quiet:
            print(f"step {step:3d}  loss {losses[-1]:.5f}")
    w1, w2 = (w.bfloat16() for w in master)
    (q1, s1, z1), (q2, s2, z2) = quantise(w1), quantise(w2)
    far = size = 0.0
    for _ in range(4):
        x = normal(1, width).bfloat16()
        token, share, offsets = route(x, gate, top)
        full, _ = layer(x, w1, w2, (token, share, offsets))
        h = dg.w4_gemm(x[token], q1, s1, zeros=z1, offsets=offsets, epilogue="gelu_tanh")
        y = dg.w4_gemm(h, q2, s2, zeros=z2, offsets=offsets)
        four = torch.zeros_like(full).index_add_(0, token, y.float() * share[:, None])
        far += float((four - full).square().sum())
        size += float(full.square().sum())
    gap = (far / size) ** 0.5
    if not quiet:
        print(f"4-bit answers differ from the 16-bit ones by {gap:.3f} of their size")
    return losses[0], losses[-1], gap


if __name__ == "__main__":
    main()
