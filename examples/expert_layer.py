"""An expert layer from its training to its answers, with the library's operators.

A layer of experts y = W2_e gelu(W1_e x), each token sent to `top` of them, learns
to reproduce the outputs of a fixed random layer:

  forward   expert_dispatch (tokens to their experts' rows), grouped_gemm twice, expert_combine
  backward  expert_combine_grad, grouped_gemm with transposed weights, grouped_gemm_wgrad
  update    newton_schulz of the momentum, one batch over the experts
  answer    w4_gemm on the weights quantised to 4 bits, token by token, and i8_gemm on
            weights and activations in 8 bits

PyTorch chooses the experts (softmax, top-k) and does the element-wise parts.

    python examples/expert_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_gemm_bf16_gb300 as dg  # noqa: E402


def route(x, gate, top):
    """(experts of every token, their shares)."""
    share, expert = torch.softmax(x.float() @ gate, dim=-1).topk(top, dim=-1)
    return expert, share / share.sum(dim=-1, keepdim=True)


def gelu(h):
    return torch.nn.functional.gelu(h.float(), approximate="tanh").to(h.dtype)


def gelu_grad(h, g):
    x = h.float()
    c, k = 0.7978845608028654, 0.044715
    t = torch.tanh(c * (x + k * x ** 3))
    return (g.float() * (0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * k * x * x))).to(h.dtype)


def layer(x, w1, w2, plan):
    """Outputs per token, and what the backward pass needs."""
    expert, share = plan
    rows, offsets, slots = dg.expert_dispatch(x, expert, w1.shape[0])
    h = dg.grouped_gemm(rows, w1, offsets)
    z = gelu(h)
    y = dg.grouped_gemm(z, w2, offsets)
    out = dg.expert_combine(y, slots, share, out_dtype=torch.float32)
    return out, (rows, h, z, offsets, slots)


def gradients(d_out, saved, w2, plan):
    rows, h, z, offsets, slots = saved
    d_y, _ = dg.expert_combine_grad(d_out, slots, plan[1])
    d_y = d_y.to(rows.dtype)
    d_w2 = dg.grouped_gemm_wgrad(z, d_y, offsets, out_dtype=torch.float32)
    d_h = gelu_grad(h, dg.grouped_gemm(d_y, w2.transpose(1, 2), offsets))
    d_w1 = dg.grouped_gemm_wgrad(rows, d_h, offsets, out_dtype=torch.float32)
    return d_w1, d_w2


def answer_in_8_bits(x, w1, w2, plan):
    """The layer with 8-bit weights (q [experts, N, K], scales) and activations: a token is
    quantised once and its bytes go to its experts' rows."""
    (q1, s1), (q2, s2) = w1, w2
    expert, share = plan
    xq, xs = dg.i8_quantize(x)
    rows, offsets, slots, rows_scales = dg.expert_dispatch(xq, expert, q1.shape[0], scales=xs)
    h = dg.i8_gemm(rows, q1, s1, x_scales=rows_scales, offsets=offsets, epilogue="gelu_tanh")
    y = dg.i8_gemm(h, q2, s2, offsets=offsets)
    return dg.expert_combine(y, slots, share, out_dtype=torch.float32)


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
    in_8_bits = [dg.i8_quantize(w.transpose(1, 2).contiguous()) for w in (w1, w2)]
    far = far8 = size = 0.0
    for _ in range(4):
        x = normal(1, width).bfloat16()
        expert, share = route(x, gate, top)
        full, _ = layer(x, w1, w2, (expert, share))
        rows, offsets, slots = dg.expert_dispatch(x, expert, experts)
        h = dg.w4_gemm(rows, q1, s1, zeros=z1, offsets=offsets, epilogue="gelu_tanh")
        y = dg.w4_gemm(h, q2, s2, zeros=z2, offsets=offsets)
        four = dg.expert_combine(y, slots, share, out_dtype=torch.float32)
        eight = answer_in_8_bits(x, *in_8_bits, (expert, share))
        far += float((four - full).square().sum())
        far8 += float((eight - full).square().sum())
        size += float(full.square().sum())
    gap = (far / size) ** 0.5
    if not quiet:
        print(f"4-bit answers differ from the 16-bit ones by {gap:.3f} of their size, 8-bit ones "
              f"by {(far8 / size) ** 0.5:.3f}")
    return losses[0], losses[-1], gap


if __name__ == "__main__":
    main()
