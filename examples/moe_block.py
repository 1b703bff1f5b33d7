"""A mixture-of-experts block on the library's calls, run against plain torch.

serve():  a projection with one low-rank adapter per request, the router, the
          experts in FP8 (contiguous rows for prefill, masked rows for decode)
          and the weighted sum back to tokens.
train():  forward and backward of a routed linear layer in bfloat16: the
          gradients of the tokens and of the router's weights.

    python examples/moe_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_grouped_gemm_act_amd as fg  # noqa: E402

H, I, E, K, R, ADAPTERS = 512, 256, 8, 2, 16, 4  # hidden, expert width, experts, choices, rank


def quantize_weight(w):
    """[..., N, K] bfloat16 -> e4m3fn codes and 128x128 block scales"""
    n, k = w.shape[-2:]
    b = w.float().reshape(*w.shape[:-2], n // 128, 128, k // 128, 128)
    s = b.abs().amax((-3, -1)) / 448
    q = (b / s[..., :, None, :, None]).reshape(w.shape).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), s.contiguous()


def make(seed=0, device="cuda"):
    g = torch.Generator().manual_seed(seed)

    def n(*shape):
        return (torch.randn(*shape, generator=g) * shape[-1] ** -0.5).to(torch.bfloat16).to(device)
    p = dict(wo=n(H, H), la=n(ADAPTERS, R, H), lb=n(ADAPTERS, H, R), scale=torch.ones(ADAPTERS, device=device),
             wr=n(E, H), w13=n(E, 2 * I, H), w2=n(E, H, I), w=n(E, H, H))
    p["w13_q"], p["s13"] = quantize_weight(p["w13"])
    p["w2_q"], p["s2"] = quantize_weight(p["w2"])
    return p


def serve(p, x, adapter, decode):
    """x [T,H] bfloat16, adapter [T] int32 (-1: none) -> [T,H] bfloat16"""
    h = fg.gemm_bf16_nt_lora(x, p["wo"], p["la"], p["lb"], adapter, p["scale"])
    ids, w = fg.moe_topk(fg.gemm_bf16_nt(h, p["wr"]), K)
    if decode:  # fixed shapes for graph replay: room for every token at every expert
        cap = x.shape[0]
        row, masked_m = fg.moe_sort_masked(ids, E, cap)
        a, sa = fg.moe_dispatch_fp8(h, row, (E, cap))
        y, sy = fg.grouped_masked_swiglu_fp8(a, sa, p["w13_q"], p["s13"], masked_m, cap)
        d = fg.grouped_masked(y, sy, p["w2_q"], p["s2"], masked_m, cap)
    else:
        row, m_indices, _ = fg.moe_sort_contiguous(ids, E)
        a, sa = fg.moe_dispatch_fp8(h, row, m_indices.numel())
        y, sy = fg.grouped_contiguous_swiglu_fp8(a, sa, p["w13_q"], p["s13"], m_indices)
        d = fg.grouped_contiguous(y, sy, p["w2_q"], p["s2"], m_indices)
    return fg.moe_combine(d, row, w)


def serve_plain(p, x, adapter):
    xf = x.float()
    h = xf @ p["wo"].float().t()
    for a in range(ADAPTERS):
        at = adapter == a
        h[at] += p["scale"][a] * (xf[at] @ p["la"][a].float().t()) @ p["lb"][a].float().t()
    h = h.to(torch.bfloat16).float()
    logits = (h @ p["wr"].float().t()).to(torch.bfloat16).float()
    top, ids = logits.topk(K)
    w = torch.softmax(top, 1)
    out = torch.zeros_like(h)
    for e in range(E):
        gate, up = (h @ p["w13"][e].float().t()).split(I, 1)
        y = (torch.nn.functional.silu(gate) * up) @ p["w2"][e].float().t()
        out += (w * (ids == e)).sum(1, keepdim=True) * y
    return out


class Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits):
        ids, w = fg.moe_topk(logits, K)
        ctx.save_for_backward(logits, ids, w)
        ctx.mark_non_differentiable(ids)
        return ids, w

    @staticmethod
    def backward(ctx, _, dw):
        return fg.moe_topk_backward(*ctx.saved_tensors, dw.contiguous())


class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, row, rows):
        ctx.save_for_backward(row)
        return fg.moe_dispatch_bf16(x, row, rows)

    @staticmethod
    def backward(ctx, da):
        return fg.moe_dispatch_backward(da.contiguous(), *ctx.saved_tensors), None, None


class Experts(torch.autograd.Function):
    """one bfloat16 linear layer per expert; its input's gradient is the same
    product with transposed weights (the weights' own gradient is not formed)"""

    @staticmethod
    def forward(ctx, a, w, m_indices):
        ctx.save_for_backward(w, m_indices)
        return fg.grouped_contiguous_bf16(a, w, m_indices)

    @staticmethod
    def backward(ctx, dy):
        w, m_indices = ctx.saved_tensors
        return fg.grouped_contiguous_bf16(dy, w.transpose(1, 2).contiguous(), m_indices), None, None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, row, w):
        ctx.save_for_backward(y, row, w)
        return fg.moe_combine(y, row, w)

    @staticmethod
    def backward(ctx, dout):
        dy, dw = fg.moe_combine_backward(dout.contiguous(), *ctx.saved_tensors)
        return dy, None, dw


def train(p, x, wr, dout):
    """gradients of <dout, layer(x)> by x and by the router's weights wr [E,H] (float32)"""
    x, wr = x.clone().requires_grad_(), wr.clone().requires_grad_()
    ids, w = Route.apply(x.float() @ wr.t())
    row, m_indices, _ = fg.moe_sort_contiguous(ids, E)
    a = Dispatch.apply(x, row, m_indices.numel())
    out = Combine.apply(Experts.apply(a, p["w"], m_indices), row, w)
    (out.float() * dout.float()).sum().backward()
    return out.detach(), x.grad, wr.grad


def train_plain(p, x, wr, dout):
    x, wr = x.float().requires_grad_(), wr.clone().requires_grad_()
    top, ids = (x @ wr.t()).topk(K)
    w = torch.softmax(top, 1)
    out = 0
    for e in range(E):
        out = out + (w * (ids == e)).sum(1, keepdim=True) * (x @ p["w"][e].float().t())
    (out * dout.float()).sum().backward()
    return out.detach(), x.grad, wr.grad


def far(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def main():
    p = make()
    g = torch.Generator().manual_seed(1)
    worst = {}
    for T, decode in ((300, False), (24, True), (1, True)):
        x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
        adapter = torch.randint(-1, ADAPTERS, (T,), generator=g, dtype=torch.int32).cuda()
        out = serve(p, x, adapter, decode)
        worst[f"serve {T} tokens, {'masked' if decode else 'contiguous'}"] = far(out, serve_plain(p, x, adapter))
    x, dout = (torch.randn(300, H, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    wr = (torch.randn(E, H, generator=g) * H ** -0.5).cuda()
    for name, a, b in zip(("out", "dx", "dwr"), train(p, x, wr, dout), train_plain(p, x, wr, dout)):
        worst[f"train {name}"] = far(a, b)
    for name, v in worst.items():
        print(f"{name}: relative difference from plain torch {v:.1e}")
    return worst


if __name__ == "__main__":
    main()
