"""A training step of a block with routed experts and a shared one, on the library's
operators: forward, and the gradients of its input and of every weight.

    s, c = scores of x Wr; the chosen experts of each token, their weights   gemm, route
    off, order, pos = rows grouped by expert                                 group_rows
    y   = x[token] We_e                          the routed experts          gemm_grouped
    m   = x + sum over a token's experts of weight * y                       combine
    h   = gelu(z), z = m W1 + b1                 the shared expert           gemm_fused
    out = m + h W2 + b2                                                      gemm_fused

Back: gemm_fused_grad (dz and db1), gemm_fused with a residual (dm), combine_grad (dy and
the weights' gradients), the grouped products, combine (the gradient of the gather),
route_grad, and gemm for the dense weights.

    python examples/mixture_block.py [tokens]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_08_gb300 as lib  # noqa: E402

RULE = dict(score=lib.GEMM_SCORE_SIGMOID, renormalize=True, scale=1.5)


def make(width=1024, hidden=2048, experts=32, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, sigma, kind=dtype):
        return torch.empty(shape, dtype=kind, device="cuda").normal_(0, sigma, generator=g)

    return dict(Wr=normal(experts, width, sigma=width ** -0.5),              # [out, in]
                balance=normal(experts, sigma=0.05, kind=torch.float32),
                We=normal(experts, width, width, sigma=width ** -0.5),       # [out, in] each
                W1=normal(hidden, width, sigma=width ** -0.5),
                b1=normal(hidden, sigma=0.1, kind=torch.float32),
                W2=normal(width, hidden, sigma=hidden ** -0.5),
                b2=normal(width, sigma=0.1, kind=torch.float32))


def forward(p, x, top=4):
    """(out, what the backward pass needs)."""
    logits = lib.gemm(x, p["Wr"].t())  # FP32
    chosen, weights = lib.route(logits, top, bias=p["balance"], groups=4, groups_kept=2, group_top=2,
                                **RULE)
    offsets, order, place = lib.group_rows(chosen.view(-1), p["We"].shape[0])
    place, token = place.view_as(chosen), order // top
    y = lib.gemm_grouped(x, p["We"].transpose(1, 2), offsets, row_index=token)
    m = lib.combine(y, place, weights=weights, residual=x)
    h, z = lib.gemm_fused(m, p["W1"].t(), bias=p["b1"], activation=lib.GEMM_ACT_GELU, keep_pre=True)
    out = lib.gemm_fused(h, p["W2"].t(), bias=p["b2"], residual=m)
    return out, (x, logits, chosen, weights, offsets, token, place, y, m, h, z)


def backward(p, saved, dout):
    """The gradients of x and of the weights, each laid out as what it belongs to."""
    x, logits, chosen, weights, offsets, token, place, y, m, h, z = saved
    ones = torch.ones((1, dout.shape[0]), dtype=dout.dtype, device="cuda")
    dz, db1 = lib.gemm_fused_grad(dout, p["W2"], z, activation=lib.GEMM_ACT_GELU, bias_grad=True)
    dm = lib.gemm_fused(dz, p["W1"], residual=dout)
    d = dict(W1=lib.gemm(dz.t(), m), b1=db1, W2=lib.gemm(dout.t(), h), b2=lib.gemm(ones, dout)[0])
    # (rows of dropped tokens, behind the last group, are not read below)
    dy, dweights = lib.combine_grad(dm, y, place, weights=weights, out=torch.empty_like(y))
    d["We"] = lib.gemm_grouped_wgrad(x, dy, offsets, row_index=token).transpose(1, 2)
    rows = lib.gemm_grouped(dy, p["We"], offsets)
    dx = lib.combine(rows, place, residual=dm)  # (of the gather: no weights)
    dlogits = lib.route_grad(logits, chosen, dweights, **RULE).to(x.dtype)
    d["Wr"] = lib.gemm(dlogits.t(), x)
    d["x"] = lib.gemm_fused(dlogits, p["Wr"], residual=dx)
    return d


def main():
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 4096
    p = make()
    x = torch.randn(tokens, p["Wr"].shape[1], device="cuda").to(torch.bfloat16)
    dout = torch.randn_like(x)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for timed in (False, True):
        if timed:
            start.record()
        for _ in range(10 if timed else 2):
            out, saved = forward(p, x)
            d = backward(p, saved, dout)
    end.record()
    torch.cuda.synchronize()
    assert lib.gemm_last_device_status() == lib.GEMM_OK
    print(f"{tokens} tokens: {start.elapsed_time(end) * 100:.1f} us a step, |out| "
          f"{out.float().norm().item():.4g}, |dx| {d['x'].float().norm().item():.4g}")


if __name__ == "__main__":
    main()
