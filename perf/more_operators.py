"""Cases of the operators around a mixture's grouped products: routing tokens to
experts, the experts' rows back to the tokens, and dense products with bias,
activation and residual; each with its gradient.

Each case is a dict of plain values.  `prepare` makes what a program holds
before the call, `run` makes one pass (the framework's call where `own` is
true, elementary torch operations where it is not), `work` counts the bytes
and operations a pass cannot do without, and `exact` computes the same results
from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
NONE, RELU, GELU, SILU = 0, 1, 2, 3
SOFTMAX, SIGMOID = 0, 1


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the router of one decode step: 32 tokens, 8 of 64 experts, FP32 logits of the router's product
        dict(name="route_decode", op="route", dtype="f32", tokens=32, experts=64, k=8,
             score=SOFTMAX, bias=False, groups=1, kept=1, top=1, renorm=True, scale=1.0),
        # a prefill or training batch with sigmoid scores, a bias for balance, 8 groups of which 4 stay
        dict(name="route_groups", op="route", dtype="f32", tokens=16384, experts=256, k=8,
             score=SIGMOID, bias=True, groups=8, kept=4, top=2, renorm=True, scale=2.5),
        # the gradient of a softmax router's logits, the weights not renormalised: every expert has one
        dict(name="route_grad_softmax", op="route_grad", dtype="bf16", tokens=16384, experts=128, k=8,
             score=SOFTMAX, renorm=False, scale=1.0),
        # the gradient of a sigmoid router with renormalised weights, an odd number of tokens
        dict(name="route_grad_sigmoid", op="route_grad", dtype="f32", tokens=4097, experts=160, k=6,
             score=SIGMOID, renorm=True, scale=2.5),
        # the experts' rows of a decode step back to its 16 tokens, with the residual stream
        dict(name="combine_decode", op="combine", dtype="bf16", tokens=16, k=8, N=4096, dropped=0,
             weights=True, residual=True, out="bf16"),
        # a prefill of 16384 tokens, 8 experts each; some rows dropped (an expert over its capacity)
        dict(name="combine_prefill", op="combine", dtype="bf16", tokens=16384, k=8, N=4096,
             dropped=1311, weights=True, residual=True, out="bf16"),
        # a training step: gradients of the experts' rows and of the weights
        dict(name="combine_grad_bf16", op="combine_grad", dtype="bf16", tokens=8192, k=8, N=4096,
             dropped=0, weights=True),
        # a small ragged batch: odd numbers of tokens and columns, dropped rows
        dict(name="combine_grad_f16", op="combine_grad", dtype="f16", tokens=4095, k=2, N=2049,
             dropped=100, weights=True),
        # one token through a projection with bias and residual: the weights are the traffic
        dict(name="fused_token_f16", op="fused", dtype="f16", M=1, K=4096, N=4096, order="col",
             bias=True, act=NONE, residual=True, pre=False),
        # training forward of an MLP's first product: bias, GELU, the value before it kept
        dict(name="fused_up_bf16", op="fused", dtype="bf16", M=8192, K=4096, N=14336, order="col",
             bias=True, act=GELU, residual=False, pre=True),
        # its backward: the second product's input gradient times GELU', and the bias gradient
        dict(name="fused_grad_bf16", op="fused_grad", dtype="bf16", M=8192, K=4096, N=14336,
             order="row", act=GELU, dbias=True),
        # the same for a small layer of odd sizes
        dict(name="fused_grad_f16", op="fused_grad", dtype="f16", M=1000, K=1408, N=2049, order="row",
             act=SILU, dbias=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "combine", "combine_grad", "fused", "fused", "fused_grad",
                     "fused_grad"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * _log_int(rng, max(1, 8 // groups), 512 // groups)
        kept = rng.randint(max(1, groups // 2), groups)
        k = min(rng.choice([1, 2, 4, 6, 8]), experts // groups * kept)
        case = dict(op=op, dtype=rng.choice(["f32", "f32", "bf16", "f16"]),
                    tokens=_log_int(rng, 1, 32768), experts=experts, k=k,
                    score=rng.choice([SOFTMAX, SIGMOID]), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]))
        if op == "route":
            case.update(bias=rng.random() < 0.5, groups=groups, kept=kept,
                        top=rng.choice([1, 2]) if groups > 1 else 1)
        return case
    dtype = rng.choice(["bf16", "bf16", "f16", "f16", "f32"])
    if op in ("combine", "combine_grad"):
        k = rng.choice([1, 2, 4, 8])
        N = _log_int(rng, 32, 8192)
        most = 16384 * 8 * 4096 // (k * N) // (2 if op == "combine_grad" else 1) * 2 // BYTES[dtype]
        tokens = _log_int(rng, 1, min(16384, most))
        case = dict(op=op, dtype=dtype, tokens=tokens, k=k, N=N, weights=rng.random() < 0.8,
                    dropped=rng.choice([0, tokens * k // 50]))
        if op == "combine":
            case.update(residual=rng.random() < 0.5, out=rng.choice([dtype, dtype, "f32"]))
        return case
    small = dtype == "f32"
    while True:
        M = _log_int(rng, 1, 2000 if small else 8192)
        K = _log_int(rng, 64, 1000 if small else 14336)
        N = _log_int(rng, 64, 1024 if small else 14336)
        if M * K * N <= 8192 * 4096 * 14336:
            break
    case = dict(op=op, dtype=dtype, M=M, K=K, N=N, order=rng.choice(["col", "row"]),
                act=rng.choice([NONE, RELU, GELU, SILU]))
    if op == "fused":
        case.update(bias=rng.random() < 0.6, residual=rng.random() < 0.5, pre=rng.random() < 0.4)
    else:
        case.update(dbias=rng.random() < 0.6)
    return case


# ----------------------------------------------------------------- prepare
def _normal(gen, shape, sigma, dtype, pad_to=1):
    """Normal values; the innermost extent is stored padded to a multiple of pad_to elements."""
    stored = list(shape)
    stored[-1] = -(-shape[-1] // pad_to) * pad_to
    t = torch.empty(stored, dtype=DTYPES[dtype], device="cuda")
    t.normal_(0.0, sigma, generator=gen)
    return t[..., :shape[-1]]


def _places(gen, case):
    """Where each (token, choice) lies among the experts' rows, which are sorted by expert and then
    by token: random distinct experts (four times as many as a token takes), some rows -1."""
    T, k = case["tokens"], case["k"]
    experts = torch.rand((T, 4 * k), generator=gen, device="cuda").argsort(1)[:, :k].reshape(-1)
    order = torch.sort(experts, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device="cuda")
    if case["dropped"]:  # rows of an expert past its capacity have no place
        place = torch.where(place < T * k - case["dropped"], place, torch.full_like(place, -1))
    return place.to(torch.int32).view(T, k)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, dt = case["op"], case["dtype"]
    vec = 16 // BYTES[dt]
    s = {"case": case}
    if op in ("route", "route_grad"):
        T, E, k = case["tokens"], case["experts"], case["k"]
        s["logits"] = _normal(gen, (T, E), 1.5, dt)
        if op == "route":
            s["bias"] = _normal(gen, (E,), 0.05, "f32") if case["bias"] else None
        else:
            # what the router chose: the k largest logits, in order
            chosen = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True).indices
            s["chosen"] = chosen[:, :k].to(torch.int32).contiguous()
            s["dweights"] = _normal(gen, (T, k), 1.0, "f32")
        return s
    if op in ("combine", "combine_grad"):
        T, k, N = case["tokens"], case["k"], case["N"]
        s["Y"] = _normal(gen, (T * k, N), 1.0, dt, vec)
        s["place"] = _places(gen, case)
        s["weights"] = None
        if case["weights"]:
            w = torch.rand((T, k), generator=gen, device="cuda") + 0.05
            s["weights"] = w / w.sum(1, keepdim=True)
        if op == "combine":
            s["residual"] = None
            if case["residual"]:
                s["residual"] = _normal(gen, (T, N), 1.0, case["out"], 16 // BYTES[case["out"]])
        else:
            s["dD"] = _normal(gen, (T, N), 1.0, dt, vec)
            # the gradient of the experts' rows; rows that no token has keep what they hold (0).
            # (one row more: where the plain form puts the rows without a place)
            pitch = -(-N // vec) * vec
            s["store"] = torch.zeros((T * k + 1, pitch), dtype=DTYPES[dt], device="cuda")[:, :N]
        return s
    M, K, N = case["M"], case["K"], case["N"]
    s["A"] = _normal(gen, (M, K), 1.0, dt, vec)
    if case["order"] == "col":  # [out, in] storage, as linear layers keep it
        s["B"] = _normal(gen, (N, K), K ** -0.5, dt, vec).t()
    else:
        s["B"] = _normal(gen, (K, N), K ** -0.5, dt, vec)
    if op == "fused":
        s["bias"] = _normal(gen, (N,), 0.5, "f32") if case["bias"] else None
        s["residual"] = _normal(gen, (M, N), 1.0, dt, vec) if case["residual"] else None
    else:
        s["Z"] = _normal(gen, (M, N), 1.0, dt, vec)
    return s


# --------------------------------------------------------------------- run
def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"route": _plain_route, "route_grad": _plain_route_grad, "combine": _plain_combine,
                "combine_grad": _plain_combine_grad, "fused": _plain_fused,
                "fused_grad": _plain_fused_grad}[op](s, case)
    import dense_gemm_08_gb300 as lib
    if op == "route":
        return lib.route(s["logits"], case["k"], score=case["score"], bias=s["bias"],
                         groups=case["groups"], groups_kept=case["kept"], group_top=case["top"],
                         renormalize=case["renorm"], scale=case["scale"])
    if op == "route_grad":
        return lib.route_grad(s["logits"], s["chosen"], s["dweights"], score=case["score"],
                              renormalize=case["renorm"], scale=case["scale"])
    if op == "combine":
        return lib.combine(s["Y"], s["place"], weights=s["weights"], residual=s["residual"],
                           out_dtype=DTYPES[case["out"]])
    if op == "combine_grad":
        return lib.combine_grad(s["dD"], s["Y"], s["place"], weights=s["weights"],
                                out=s["store"][:-1])
    if op == "fused":
        return lib.gemm_fused(s["A"], s["B"], bias=s["bias"], activation=case["act"],
                              residual=s["residual"], keep_pre=case["pre"])
    return lib.gemm_fused_grad(s["A"], s["B"], s["Z"], activation=case["act"],
                               bias_grad=case["dbias"])


def _first(x, k):
    """The k largest of each row and where they are, ties by index."""
    v, i = torch.sort(x, dim=-1, descending=True, stable=True)
    return v[..., :k], i[..., :k]


def _plain_route(s, case):
    x = s["logits"]
    T, E, k = case["tokens"], case["experts"], case["k"]
    wide = x.double()
    p = _scores(wide, case["score"])
    # the choice goes by values that may lie close together: 64 bits.  (Without a bias the scores'
    # order is the logits' own.)
    c = p + s["bias"].double() if s["bias"] is not None else wide
    if case["groups"] > 1:
        rank = c if case["top"] == 1 else (c if s["bias"] is not None else p)
        g = _first(rank.view(T, case["groups"], -1), case["top"])[0].sum(-1)
        best = _first(g, case["kept"])[1]
        keep = torch.zeros_like(g).scatter_(1, best, 1.0).repeat_interleave(E // case["groups"], 1)
        c = torch.where(keep > 0, c, torch.full_like(c, -math.inf))
    chosen = _first(c, k)[1]
    w = _scores(x.float(), case["score"]).gather(1, chosen)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return chosen.to(torch.int32), w * case["scale"]


def _scores(x, score):
    if score == SIGMOID:
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route_grad(s, case):
    at = s["chosen"].long()
    p = _scores(s["logits"].float(), case["score"])
    mine, d = p.gather(1, at), s["dweights"] * case["scale"]
    if case["renorm"]:
        total = mine.sum(1, keepdim=True)
        d = (d - (d * mine / total).sum(1, keepdim=True)) / total
    dp = torch.zeros_like(p).scatter_(1, at, d)
    if case["score"] == SIGMOID:
        dx = dp * p * (1.0 - p)
    else:
        dx = p * (dp - (dp * p).sum(1, keepdim=True))
    return dx.to(DTYPES[case["dtype"]])


def _plain_combine(s, case):
    at = s["place"].long()
    w = (at >= 0).float()
    if s["weights"] is not None:
        w = w * s["weights"]
    d = (s["Y"][at.clamp(min=0)].float() * w[..., None]).sum(1)
    if s["residual"] is not None:
        d = d + s["residual"].float()
    return d.to(DTYPES[case["out"]])


def _plain_combine_grad(s, case):
    at = s["place"].long()
    kept = at >= 0
    d = s["dD"].float()
    wide = d[:, None, :] if s["weights"] is None else d[:, None, :] * s["weights"][..., None]
    wide = wide.expand(-1, case["k"], -1).to(DTYPES[case["dtype"]])
    store = s["store"]
    store[torch.where(kept, at, torch.full_like(at, store.shape[0] - 1)).view(-1)] = wide.reshape(
        -1, case["N"])
    dw = (d[:, None, :] * s["Y"][at.clamp(min=0)].float()).sum(-1) * kept
    return store[:-1], dw


def _activate(z, act):
    if act == RELU:
        return torch.clamp(z, min=0.0)
    if act == GELU:
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == SILU:
        return z / (1.0 + torch.exp(-z))
    return z


def _slope(z, act):
    if act == RELU:
        return (z > 0).to(z.dtype)
    if act == GELU:
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if act == SILU:
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _plain_fused(s, case):
    z = s["A"].float() @ s["B"].float()
    if s["bias"] is not None:
        z = z + s["bias"]
    d = _activate(z, case["act"])
    if s["residual"] is not None:
        d = d + s["residual"].float()
    dt = DTYPES[case["dtype"]]
    return (d.to(dt), z.to(dt)) if case["pre"] else d.to(dt)


def _plain_fused_grad(s, case):
    d = (s["A"].float() @ s["B"].float()) * _slope(s["Z"].float(), case["act"])
    dt = DTYPES[case["dtype"]]
    return (d.to(dt), d.sum(0)) if case["dbias"] else d.to(dt)


# -------------------------------------------------------------------- work
def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["k"]
        return {"bytes": e * T * E + 8 * T * k + (4 * E if case["bias"] else 0), "flops": 0}
    if op == "route_grad":
        T, E, k = case["tokens"], case["experts"], case["k"]
        # renormalised weights and sigmoid scores depend on the chosen logits alone
        read = T * E if case["score"] == SOFTMAX and not case["renorm"] else T * k
        return {"bytes": e * (read + T * E) + 8 * T * k, "flops": 0}
    if op in ("combine", "combine_grad"):
        T, k, N = case["tokens"], case["k"], case["N"]
        rows = T * k - case["dropped"]
        small = 4 * T * k * (2 if case["weights"] else 1)
        if op == "combine":
            o = BYTES[case["out"]]
            return {"bytes": e * rows * N + o * T * N * (2 if case["residual"] else 1) + small,
                    "flops": 2 * rows * N}
        return {"bytes": e * (2 * rows * N + T * N) + small + 4 * T * k, "flops": 3 * rows * N}
    M, K, N = case["M"], case["K"], case["N"]
    if op == "fused":
        outs = 1 + (1 if case["residual"] else 0) + (1 if case["pre"] else 0)
        return {"bytes": e * (M * K + K * N + outs * M * N) + (4 * N if case["bias"] else 0),
                "flops": 2 * M * K * N}
    return {"bytes": e * (M * K + K * N + 2 * M * N) + (4 * N if case["dbias"] else 0),
            "flops": 2 * M * K * N}


# ------------------------------------------------------------------- exact
def _p64(x, score):
    return torch.sigmoid(x) if score == SIGMOID else torch.softmax(x, 1)


def exact(case, seed):
    op = case["op"]
    if op in ("fused", "fused_grad") and work(case)["flops"] > 2.5e12:
        return None
    s = prepare(case, seed)
    if op == "route":
        x = s["logits"].double()
        p = _p64(x, case["score"])
        # without a bias the logits' order is the scores' own
        c = x if s["bias"] is None else p + s["bias"].double()
        E, G = case["experts"], case["groups"]
        if G > 1:
            by = p if s["bias"] is None and case["top"] > 1 else c
            size = E // G
            best = torch.topk(by.view(-1, G, size), min(case["top"], size), dim=2).values.sum(2)
            order = torch.argsort(best, dim=1, descending=True, stable=True)[:, :case["kept"]]
            allowed = torch.zeros_like(best, dtype=torch.bool)
            allowed.scatter_(1, order, True)
            c = c.masked_fill(~allowed.repeat_interleave(size, 1), -math.inf)
        chosen = torch.argsort(c, dim=1, descending=True, stable=True)[:, :case["k"]]
        w = torch.gather(p, 1, chosen)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return chosen.to(torch.int32), w * case["scale"]
    if op == "route_grad":
        # by the chain rule, through the Jacobian of each step
        x, at = s["logits"].double(), s["chosen"].long()
        p, dw = _p64(x, case["score"]), s["dweights"].double() * case["scale"]
        q = p.gather(1, at)
        dq = dw
        if case["renorm"]:
            S = q.sum(1, keepdim=True)
            dq = dw / S - (dw * q).sum(1, keepdim=True) / (S * S)
        dx = torch.zeros_like(x)
        if case["score"] == SIGMOID:
            dx.scatter_add_(1, at, dq * q * (1 - q))
        else:
            dx.scatter_add_(1, at, dq * q)
            dx -= p * (dq * q).sum(1, keepdim=True)
        return dx
    if op == "combine":
        d = torch.zeros((case["tokens"], case["N"]), dtype=torch.float64, device="cuda")
        if s["residual"] is not None:
            d += s["residual"].double()
        for j in range(case["k"]):
            at = s["place"][:, j].long()
            has = torch.nonzero(at >= 0)[:, 0]
            y = s["Y"][at[has]].double()
            if s["weights"] is not None:
                y *= s["weights"][has, j].double()[:, None]
            d[has] += y
        return d
    if op == "combine_grad":
        T, k, N = case["tokens"], case["k"], case["N"]
        dY = torch.zeros((T * k, N), dtype=torch.float64, device="cuda")
        dw = torch.zeros((T, k), dtype=torch.float64, device="cuda")
        for j in range(k):
            at = s["place"][:, j].long()
            has = torch.nonzero(at >= 0)[:, 0]
            g = s["dD"][has].double()
            dw[has, j] = torch.einsum("tn,tn->t", g, s["Y"][at[has]].double())
            if s["weights"] is not None:
                g = g * s["weights"][has, j].double()[:, None]
            dY[at[has]] = g
        return dY, dw
    z = s["A"].double() @ s["B"].double()
    if op == "fused":
        if s["bias"] is not None:
            z += s["bias"].double()
        d = _act64(z, case["act"])[0]
        if s["residual"] is not None:
            d = d + s["residual"].double()
        return (d, z) if case["pre"] else d
    d = z * _act64(s["Z"].double(), case["act"])[1]
    return (d, d.sum(0)) if case["dbias"] else d


def _act64(z, act):
    """(activation, its derivative)."""
    if act == NONE:
        return z, 1.0
    if act == RELU:
        return torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0).to(z.dtype)
    if act == SILU:
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    # GELU, tanh form: z times the logistic function of 2u
    c = (2.0 / math.pi) ** 0.5
    p = torch.sigmoid(2 * c * (z + 0.044715 * z ** 3))
    return z * p, p + z * p * (1 - p) * 2 * c * (1 + 3 * 0.044715 * z ** 2)
