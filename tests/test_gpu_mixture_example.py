"""The mixture-of-experts example against the same layer written out in 64 bits."""
import math
import os
import sys

import pytest
import torch

import dense_gemm_08_gb300 as lib

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 7, 200])
def test_forward_and_gradients(tokens):
    import mixture_layer as ex
    p = ex.make(width=256, hidden=384, experts=6, adapters=3, seed=tokens)
    x = torch.randn(tokens, 256, device="cuda").to(torch.bfloat16)
    adapter = (torch.arange(tokens, device="cuda") % 4 - 1).to(torch.int32)
    got = ex.forward(p, x, adapter)
    torch.cuda.synchronize()
    assert lib.gemm_last_device_status() == lib.GEMM_OK
    # the layer in 64 bits, from the BF16 values each step starts with
    h = lib.gemm_lora(x, p["W"].t(), p["LA"].transpose(1, 2), p["LB"].transpose(1, 2), adapter,
                      scale=p["scale"])
    want_h = x.double() @ p["W"].double().t()
    for i, a in enumerate(adapter.tolist()):
        if a >= 0:
            want_h[i] += 2.0 * (x[i].double() @ p["LA"][a].double().t()) @ p["LB"][a].double().t()
    # BF16 results of sums of unit size: half an ulp of the result, and of the first product
    assert torch.allclose(h.double(), want_h, rtol=2.0 ** -7, atol=2.0 ** -6)
    offsets, token, place, weights = ex.route(p, h, 2)
    out = torch.zeros(tokens, 256, dtype=torch.float64, device="cuda")
    bounds = offsets.tolist()
    assert bounds[-1] == 2 * tokens
    for e in range(6):
        for r in range(bounds[e], bounds[e + 1]):
            t = int(token[r])
            z = h[t].double() @ p["W1"][e].double().t()
            u = 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
            slot = int((place.view(tokens, 2)[t] == r).nonzero()[0])
            out[t] += weights[t, slot].double() * (u.to(torch.bfloat16).double() @ p["W2"][e].double().t())
    assert torch.allclose(got.double(), out, rtol=2.0 ** -7, atol=2.0 ** -7)
    dv = torch.randn(2 * tokens, 384, device="cuda").to(torch.bfloat16)
    dh, dW1 = ex.gradients(p, h, offsets, token, dv)
    torch.cuda.synchronize()
    for e in range(6):
        lo, hi = bounds[e], bounds[e + 1]
        rows = h[token[lo:hi].long()].double()
        want = dv[lo:hi].double().t() @ rows
        assert torch.allclose(dW1[e].double(), want, rtol=1e-4, atol=1e-4 * math.sqrt(max(hi - lo, 1)))
        assert torch.allclose(dh[lo:hi].double(), dv[lo:hi].double() @ p["W1"][e].double(), rtol=1e-4,
                              atol=1e-4 * math.sqrt(384))
