"""The gradients of the block of routed and shared experts against central differences of the block in 64
bits (the choice of experts fixed), and each as a whole against the formulas'."""
import math
import os
import sys

import pytest
import torch

import dense_gemm_08_gb300 as lib
from test_gpu_mixture_block import reference

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu

# In units u of half a step of the type, as 2-norms.  On the way to a gradient y, m, z, h, dz, dm, dy, the
# experts' rows and dx or dlogits are rounded, nine at most, each off by u of itself; the weights' gradient is a
# difference of terms of one size (dw - sum of q dw), which can double what they are off by.
UNITS = 18


def block(p, x, chosen):
    """out in 64 bits."""
    s = torch.sigmoid(x @ p["Wr"].t()).gather(1, chosen)
    w = 1.5 * s / s.sum(1, keepdim=True)
    m = x
    for j in range(chosen.shape[1]):
        m = m + w[:, j:j + 1] * torch.einsum("tk,tnk->tn", x, p["We"][chosen[:, j]])
    z = m @ p["W1"].t() + p["b1"]
    h = 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return m + h @ p["W2"].t() + p["b2"]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens", [3, 130])
def test_gradients(dtype, tokens):
    import mixture_block as ex
    p = ex.make(width=128, hidden=264, experts=16, dtype=dtype, seed=tokens)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(tokens, 128, device="cuda", generator=g).to(dtype)
    dout = torch.randn(tokens, 128, device="cuda", generator=g).to(dtype)
    _, saved = ex.forward(p, x)
    d = ex.backward(p, saved, dout)
    torch.cuda.synchronize()
    assert lib.gemm_last_device_status() == lib.GEMM_OK
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    _, grads = reference(p, x, saved[2], dout, 4)
    chosen = saved[2].long()
    wide = {k: v.double() for k, v in p.items() if k != "balance"}
    wide["x"] = x.double()
    assert set(d) == set(wide)

    def value(name, at):
        q = dict(wide, **{name: at})
        return (block(q, q["x"], chosen) * dout.double()).sum()

    for name in d:
        mine = d[name].double()
        assert (mine - grads[name]).norm() <= UNITS * u * grads[name].norm(), name
        # along the library's gradient, and along one drawn at random.  (h^2 times the third derivative, and
        # 2^-52 of the sum / h, are far below the roundings)
        for v in (mine / mine.norm(), torch.randn(mine.shape, dtype=torch.float64, device="cuda", generator=g)):
            v = v / v.norm()
            h = 1e-4
            slope = (value(name, wide[name] + h * v) - value(name, wide[name] - h * v)) / (2 * h)
            assert abs(float(slope - (mine * v).sum())) <= (UNITS * u + 1e-6) * float(mine.norm()), name
