"""A mixture-of-experts layer with per-request adapters, forward and backward,
on the library's grouped operators.

    h   = x W + s (x LA_a) LB_a          a = the request's adapter     gemm_lora
    e, weight = the top experts of each token, by the router's scores  route
    off, order, pos = rows grouped by expert                           group_rows
    u   = gelu(h[token] W1_e + b1_e)     rows gathered by token        gemm_grouped
    y   = u W2_e                                                       gemm_grouped
    out = sum over a token's experts of weight * y                     combine

`forward` serves (any number of tokens, one included); `gradients` is the
backward pass of the expert layers without the activation: the grouped products
with the other storage order, and the weight gradients over each expert's rows.

    python examples/mixture_layer.py [tokens]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_08_gb300 as lib  # noqa: E402


def make(width=1024, hidden=2048, experts=16, adapters=8, rank=16, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, sigma):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0, sigma, generator=g)

    return dict(W=normal(width, width, sigma=width ** -0.5),           # [out, in]
                LA=normal(adapters, rank, width, sigma=width ** -0.5),  # [rank, in]
                LB=normal(adapters, width, rank, sigma=0.1),            # [out, rank]
                scale=torch.full((adapters,), 2.0, device="cuda"),
                router=normal(width, experts, sigma=width ** -0.5),
                W1=normal(experts, hidden, width, sigma=width ** -0.5),
                b1=torch.zeros(experts, hidden, device="cuda"),
                W2=normal(experts, width, hidden, sigma=hidden ** -0.5))


def route(p, h, top):
    """Experts of each token's rows, grouped: (offsets, token of each row, place, weights)."""
    scores = lib.gemm(h, p["router"])  # FP32
    chosen, weights = lib.route(scores, top, renormalize=False)
    offsets, order, place = lib.group_rows(chosen.view(-1), p["W1"].shape[0])
    return offsets, order // top, place, weights


def forward(p, x, adapter, top=2):
    h = lib.gemm_lora(x, p["W"].t(), p["LA"].transpose(1, 2), p["LB"].transpose(1, 2), adapter,
                      scale=p["scale"])
    offsets, token, place, weights = route(p, h, top)
    u = lib.gemm_grouped(h, p["W1"].transpose(1, 2), offsets, row_index=token, bias=p["b1"],
                         activation=lib.GEMM_ACT_GELU)
    y = lib.gemm_grouped(u, p["W2"].transpose(1, 2), offsets, out_dtype=torch.float32)
    return lib.combine(y, place.view_as(weights), weights=weights)


def gradients(p, h, offsets, token, dv):
    """For v = h[token] W1_e (a row per place) and its gradient dv: (dh per place, dW1 [out, in])."""
    dh = lib.gemm_grouped(dv, p["W1"], offsets, out_dtype=torch.float32)
    dW1 = lib.gemm_grouped_wgrad(h, dv, offsets, row_index=token)  # [in, out]
    return dh, dW1.transpose(1, 2)


def main():
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 512
    p = make()
    x = torch.randn(tokens, p["W"].shape[1], device="cuda").to(torch.bfloat16)
    adapter = (torch.arange(tokens, device="cuda") % (p["LA"].shape[0] + 1) - 1).to(torch.int32)
    forward(p, x, adapter)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(10):
        out = forward(p, x, adapter)
    end.record()
    torch.cuda.synchronize()
    assert lib.gemm_last_device_status() == lib.GEMM_OK
    print(f"{tokens} tokens: {start.elapsed_time(end) * 100:.1f} us a pass, |out| "
          f"{out.norm().item():.4g}")


if __name__ == "__main__":
    main()
