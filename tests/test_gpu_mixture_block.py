"""The block of routed and shared experts (examples/mixture_block.py): the router, the grouped
products, the combination and the fused products run together, forward and backward, against
the same block in 64 bits with gradients by torch's autograd."""
import math
import os
import sys

import pytest
import torch

import dense_gemm_08_gb300 as lib

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def reference(p, x, chosen, dout, top):
    """The block with the same choice of experts."""
    q = {k: v.double().requires_grad_() for k, v in p.items() if k != "balance"}
    xd = x.double().requires_grad_()
    s = torch.sigmoid(xd @ q["Wr"].t())
    w = s.gather(1, chosen.long())
    w = 1.5 * w / w.sum(1, keepdim=True)
    m = xd
    for j in range(top):
        y = torch.einsum("tk,tnk->tn", xd, q["We"][chosen[:, j].long()])
        m = m + w[:, j:j + 1] * y
    z = m @ q["W1"].t() + q["b1"]
    h = 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    out = m + h @ q["W2"].t() + q["b2"]
    out.backward(dout.double())
    return out, dict({k: v.grad for k, v in q.items()}, x=xd.grad)


def off(got, ref):
    """Relative to the largest value: sums of values of one size."""
    return float((got.double() - ref.detach()).abs().max() / ref.detach().abs().max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens", [1, 5, 130, 700])
def test_forward_and_backward(dtype, tokens):
    import mixture_block as ex
    p = ex.make(width=128, hidden=264, experts=16, dtype=dtype, seed=tokens)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens, 128, device="cuda", generator=g).to(dtype)
    dout = torch.randn(tokens, 128, device="cuda", generator=g).to(dtype)
    out, saved = ex.forward(p, x)
    d = ex.backward(p, saved, dout)
    torch.cuda.synchronize()
    assert lib.gemm_last_device_status() == lib.GEMM_OK
    chosen = saved[2]
    # the choice follows the rule, from the logits that the block computed
    c = torch.sigmoid(saved[1].double()) + p["balance"].double()
    best = c.view(tokens, 4, 4).topk(2, 2).values.sum(2).topk(2, 1).indices
    allowed = torch.zeros(tokens, 4, dtype=torch.bool, device="cuda").scatter_(1, best, True)
    c = c.masked_fill(~allowed.repeat_interleave(4, 1), -math.inf)
    assert torch.equal(chosen.long(), c.topk(4, 1).indices)
    ref, grads = reference(p, x, chosen, dout, 4)
    # Each value on the way is rounded to the type (half a step u): out through y, m, h and itself,
    # the gradients through those and dz, dm, dy, their rows and dx; a rounding's share of a result of
    # many terms of random sign is at most its own size, so 8 u and 16 u of the largest value, and as
    # much again for values beside the largest ones (heavy tails: the ratio of the largest value to
    # the terms' root mean square stays above 1).
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    assert off(out, ref) <= 8 * u
    assert set(d) == set(grads)
    for k in grads:
        assert d[k].shape == grads[k].shape
        assert off(d[k], grads[k]) <= 32 * u, k


def test_a_captured_step_is_replayed_with_other_values():
    """The whole step in a graph: the sizes of the groups are on the device only."""
    import mixture_block as ex
    p = ex.make(width=128, hidden=256, experts=16)
    x = torch.randn(300, 128, device="cuda").bfloat16()
    dout = torch.randn(300, 128, device="cuda").bfloat16()
    out, saved = ex.forward(p, x)
    ex.backward(p, saved, dout)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gout, gsaved = ex.forward(p, x)
        gd = ex.backward(p, gsaved, dout)
    for _ in range(2):
        x.copy_(torch.randn(300, 128, device="cuda").bfloat16())
        graph.replay()
        out, saved = ex.forward(p, x)
        d = ex.backward(p, saved, dout)
        assert torch.equal(gout, out) and torch.equal(gsaved[2], saved[2])
        for k in d:
            assert torch.equal(gd[k], d[k]), k


def test_padded_tokens():
    """Rows of a padded batch whose logits are masked: no expert, and the residual alone."""
    g = torch.Generator(device="cuda").manual_seed(2)
    logits = torch.randn(40, 16, device="cuda", generator=g)
    logits[25:] = -math.inf
    chosen, w = lib.route(logits, 3)
    offsets, order, place = lib.group_rows(chosen.view(-1), 16)
    assert int(offsets[-1]) == 75 and (place.view(40, 3)[25:] == -1).all()
    x = torch.randn(40, 64, device="cuda", generator=g)
    W = torch.randn(16, 64, 64, device="cuda", generator=g)
    y = torch.full((120, 64), math.nan, device="cuda")
    lib.gemm_grouped(x, W, offsets, row_index=order // 3, out=y)  # (rows past the groups: left NaN)
    out = lib.combine(y, place.view(40, 3), weights=w, residual=x)
    assert torch.equal(out[25:], x[25:]) and torch.isfinite(out).all()
    dY = torch.zeros_like(y)
    _, dw = lib.combine_grad(out, y, place.view(40, 3), weights=w, out=dY)
    assert (dw[25:] == 0).all() and torch.isfinite(dw).all() and (dY[75:] == 0).all()
    dl = lib.route_grad(logits, chosen, dw)
    assert (dl[25:] == 0).all() and torch.isfinite(dl).all()
