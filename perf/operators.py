"""Cases of the grouped operators: rows grouped by a number, matrix products
grouped by expert, their weight gradients, and low-rank adapters of many
requests beside a shared projection.

Each case is a dict of plain values.  `prepare` makes what a program holds
before the call, `run` makes one pass (the framework's call where `own` is
true, elementary torch operations in 32 bits where it is not), `work` counts
the bytes and operations a pass cannot do without, and `exact` computes the
same results from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
NONE, RELU, GELU = 0, 1, 2


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the router's rows of one decode step: 32 tokens, 8 experts each, 64 experts
        dict(name="group_decode", op="group", rows=256, groups=64, skew=0.6, dropped=0),
        # a prefill or training batch of 16384 tokens, 8 of 128 experts each, some rows dropped
        # (an expert over its capacity)
        dict(name="group_prefill", op="group", rows=131072, groups=128, skew=0.5, dropped=1311),
        # decode: 16 tokens x 8 experts over 64 experts, up projection with GELU; the experts'
        # weights are the traffic
        dict(name="experts_decode_bf16", op="grouped", dtype="bf16", rows=128, groups=64, K=4096,
             N=2048, skew=0.7, topk=8, order="col", bias=False, act=GELU, out="bf16"),
        # prefill or training forward: 8192 tokens x 2 of 8 experts, the MLP shape 4096 -> 14336,
        # rows gathered from the tokens, bias and GELU fused
        dict(name="experts_up_bf16", op="grouped", dtype="bf16", rows=16384, groups=8, K=4096,
             N=14336, skew=0.4, topk=2, order="col", bias=True, act=GELU, out="bf16"),
        # input gradient of many small experts (the other storage order of the weights), ragged
        # and odd: 64 experts, an odd number of rows and columns, some experts empty
        dict(name="experts_dgrad_f16", op="grouped", dtype="f16", rows=8191, groups=64, K=1408,
             N=2049, skew=1.1, topk=0, order="row", bias=False, act=NONE, out="f16"),
        # FP32 experts of a small model
        dict(name="experts_f32", op="grouped", dtype="f32", rows=2000, groups=16, K=1000, N=1024,
             skew=0.5, topk=0, order="row", bias=True, act=RELU, out="f32"),
        # weight gradient of the large experts' up projection, FP32 gradients
        dict(name="wgrad_bf16", op="wgrad", dtype="bf16", rows=16384, groups=8, M=4096, N=14336,
             skew=0.4, topk=2, beta=0.0, out="f32"),
        # weight gradient accumulated over micro-batches (beta = 1), many small experts
        dict(name="wgrad_accumulate_f16", op="wgrad", dtype="f16", rows=4097, groups=64, M=1024,
             N=2048, skew=0.9, topk=0, beta=1.0, out="f32"),
        # FP32 weight gradient of a small model
        dict(name="wgrad_f32", op="wgrad", dtype="f32", rows=2000, groups=16, M=1000, N=1024,
             skew=0.5, topk=0, beta=0.0, out="f32"),
        # one token of one request, square projection
        dict(name="lora_token_f16", op="lora", dtype="f16", M=1, K=4096, N=4096, rank=16,
             adapters=32, skew=0.0, base=0, mixed=True, order="col", out="f16"),
        # a decode step of 64 requests over 48 adapters, some requests without one
        dict(name="lora_decode_bf16", op="lora", dtype="bf16", M=64, K=4096, N=14336, rank=16,
             adapters=48, skew=0.5, base=7, mixed=True, order="col", out="bf16"),
        # a prefill of 8192 tokens of about 20 requests, each with its own adapter
        dict(name="lora_prefill_bf16", op="lora", dtype="bf16", M=8192, K=4096, N=14336, rank=64,
             adapters=20, skew=0.5, base=300, mixed=False, order="col", out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["group", "grouped", "grouped", "wgrad", "wgrad", "lora", "lora"])
    if op == "group":
        rows = _log_int(rng, 8, 131072)
        return dict(op=op, rows=rows, groups=_log_int(rng, 2, 256), skew=rng.choice([0.0, 0.5, 1.2]),
                    dropped=rng.choice([0, rows // 50]))
    dtype = rng.choice(["bf16", "bf16", "f16", "f16", "f32"])
    small = dtype == "f32"
    if op == "lora":
        dtype = "bf16" if small else dtype
        M = _log_int(rng, 1, 8192)
        adapters = _log_int(rng, 1, 64)
        return dict(op=op, dtype=dtype, M=M, K=_log_int(rng, 128, 8192), N=_log_int(rng, 128, 14336),
                    rank=rng.choice([8, 16, 16, 32, 64]), adapters=adapters,
                    skew=rng.choice([0.0, 0.6, 1.1]), base=rng.choice([0, M // 7]),
                    mixed=M <= 256, order=rng.choice(["col", "row"]),
                    out=rng.choice([dtype, dtype, "f32"]))
    while True:
        rows = _log_int(rng, 16, 2000 if small else 16384)
        groups = _log_int(rng, 1, 64)
        K = _log_int(rng, 64, 1000 if small else 8192)
        N = _log_int(rng, 64, 1024 if small else 14336)
        if rows * K * N <= 16384 * 4096 * 14336 and groups * K * N <= (1 << 29):
            break
    skew = rng.choice([0.0, 0.5, 1.0])
    out = "f32" if small else rng.choice([dtype, dtype, "f32"])
    if op == "wgrad":
        return dict(op=op, dtype=dtype, rows=rows, groups=groups, M=K, N=N, skew=skew,
                    topk=rng.choice([0, 0, 2]), beta=rng.choice([0.0, 1.0]), out=out)
    return dict(op=op, dtype=dtype, rows=rows, groups=groups, K=K, N=N, skew=skew,
                topk=rng.choice([0, 0, 2]), order=rng.choice(["col", "row"]),
                bias=rng.random() < 0.5, act=rng.choice([NONE, RELU, GELU]), out=out)


def _ragged(rows, groups, skew):
    """Rows of each group: proportional to (g + 1)^-skew, whole numbers that add up to rows."""
    w = [(g + 1.0) ** -skew for g in range(groups)]
    total = sum(w)
    share = [rows * x / total for x in w]
    sizes = [int(s) for s in share]
    by_rest = sorted(range(groups), key=lambda g: (sizes[g] - share[g], g))
    for g in by_rest[:rows - sum(sizes)]:
        sizes[g] += 1
    return sizes


# ----------------------------------------------------------------- prepare
def _normal(gen, shape, sigma, dtype, pad_to=1):
    """Normal values; the innermost extent is stored padded to a multiple of pad_to elements."""
    stored = list(shape)
    stored[-1] = -(-shape[-1] // pad_to) * pad_to
    t = torch.empty(stored, dtype=DTYPES[dtype], device="cuda")
    t.normal_(0.0, sigma, generator=gen)
    return t[..., :shape[-1]]


def _ids(gen, sizes, none, mixed):
    """A group number per row: sizes[g] rows of each group (which group gets which size goes by
    the seed), `none` rows of -1; shuffled, or in runs."""
    groups = len(sizes)
    perm = torch.randperm(groups, generator=gen, device="cuda")
    numbers = torch.cat([perm, torch.full((1,), -1, dtype=perm.dtype, device="cuda")])
    counts = torch.tensor(list(sizes) + [none], device="cuda")
    ids = torch.repeat_interleave(numbers, counts)
    if mixed:
        ids = ids[torch.randperm(ids.numel(), generator=gen, device="cuda")]
    return ids.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op == "group":
        sizes = _ragged(case["rows"] - case["dropped"], case["groups"], case["skew"])
        s["ids"] = _ids(gen, sizes, case["dropped"], True)
        return s
    dt = case["dtype"]
    vec = 16 // BYTES[dt]
    if op == "lora":
        M, K, N, r, n = (case[k] for k in ("M", "K", "N", "rank", "adapters"))
        s["ids"] = _ids(gen, _ragged(M - case["base"], n, case["skew"]), case["base"], case["mixed"])
        s["X"] = _normal(gen, (M, K), 1.0, dt, vec)
        if case["order"] == "col":  # [out, in] storage, as linear layers keep it
            s["W"] = _normal(gen, (N, K), 0.02, dt, vec).t()
            s["LA"] = _normal(gen, (n, r, K), 0.02, dt, vec).transpose(1, 2)
            s["LB"] = _normal(gen, (n, N, r), 0.05, dt, vec).transpose(1, 2)
        else:
            s["W"] = _normal(gen, (K, N), 0.02, dt, vec)
            s["LA"] = _normal(gen, (n, K, r), 0.02, dt, vec)
            s["LB"] = _normal(gen, (n, r, N), 0.05, dt, vec)
        s["scale"] = torch.rand(n, generator=gen, device="cuda") + 0.5
        return s
    rows, groups = case["rows"], case["groups"]
    sizes = _ragged(rows, groups, case["skew"])
    ids = _ids(gen, sizes, 0, True).long()
    order = torch.sort(ids, stable=True).indices
    s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"),
                              torch.bincount(ids, minlength=groups).cumsum(0)]).to(torch.int32)
    s["most"] = max(sizes)  # rows of the largest group (the plain form pads to it)
    stored = rows
    s["row_index"] = None
    if case["topk"] > 1:  # rows of the tokens, each used by topk rows of the product
        stored = -(-rows // case["topk"])
        s["row_index"] = (order // case["topk"]).to(torch.int32)
    if op == "grouped":
        K, N = case["K"], case["N"]
        s["A"] = _normal(gen, (stored, K), 1.0, dt, vec)
        if case["order"] == "col":
            s["B"] = _normal(gen, (groups, N, K), 0.02, dt, vec).transpose(1, 2)
        else:
            s["B"] = _normal(gen, (groups, K, N), 0.02, dt, vec)
        s["bias"] = _normal(gen, (groups, N), 0.5, "f32") if case["bias"] else None
    else:
        M, N = case["M"], case["N"]
        s["A"] = _normal(gen, (stored, M), 1.0, dt, vec)
        s["B"] = _normal(gen, (rows, N), 0.02, dt, vec)
        s["C"] = _normal(gen, (groups, M, N), 0.1, "f32") if case["beta"] else None
    return s


# --------------------------------------------------------------------- run
def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"group": _plain_group, "grouped": _plain_grouped, "wgrad": _plain_wgrad,
                "lora": _plain_lora}[op](s, case)
    import dense_gemm_08_gb300 as lib
    if op == "group":
        return lib.group_rows(s["ids"], case["groups"])
    out = DTYPES[case["out"]]
    if op == "grouped":
        return lib.gemm_grouped(s["A"], s["B"], s["offsets"], row_index=s["row_index"],
                                bias=s["bias"], activation=case["act"], out_dtype=out)
    if op == "wgrad":
        return lib.gemm_grouped_wgrad(s["A"], s["B"], s["offsets"], row_index=s["row_index"],
                                      C=s["C"], beta=case["beta"], out_dtype=out)
    return lib.gemm_lora(s["X"], s["W"], s["LA"], s["LB"], s["ids"], scale=s["scale"],
                         out_dtype=out)


def _activate(x, act):
    if act == RELU:
        return torch.clamp(x, min=0.0)
    if act == GELU:
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _plain_group(s, case):
    # one line per group: a row's place is its group's start plus the rows of its group before it
    ids, groups = s["ids"].long(), case["groups"]
    hot = (ids[None, :] == torch.arange(groups, device=ids.device)[:, None]).to(torch.int32)
    upto = torch.cumsum(hot, 1, dtype=torch.int32)
    offsets = torch.zeros(groups + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.cumsum(upto[:, -1], 0)
    kept = ids >= 0
    at = ids.clamp(min=0)
    place = offsets[at] + upto.gather(0, at[None, :])[0] - 1
    position = torch.where(kept, place, torch.full_like(place, -1))
    order = torch.full((ids.numel() + 1,), -1, dtype=torch.int32, device=ids.device)
    order[torch.where(kept, place, torch.full_like(place, ids.numel())).long()] = torch.arange(
        ids.numel(), dtype=torch.int32, device=ids.device)
    return offsets, order[:-1], position


def _padded(s, x):
    """The groups' rows as [groups, most rows, ...] in 32 bits, zeros past a group's end; and
    where each row of the product lies in it."""
    offsets = s["offsets"].long()
    groups, most = offsets.numel() - 1, s["most"]
    j = torch.arange(most, device=x.device)
    rows = offsets[:-1, None] + j
    inside = rows < offsets[1:, None]
    wide = x[torch.where(inside, rows, torch.zeros_like(rows))].float() * inside[..., None]
    r = torch.arange(x.shape[0], device=x.device)
    g = (r[:, None] >= offsets[1:]).sum(1)
    return wide, g * most + r - offsets[g]


def _plain_grouped(s, case):
    x = s["A"] if s["row_index"] is None else s["A"][s["row_index"].long()]
    wide, at = _padded(s, x)
    y = torch.bmm(wide, s["B"].float())
    if s["bias"] is not None:
        y = y + s["bias"][:, None, :]
    y = y.reshape(-1, y.shape[-1])[at]
    return _activate(y, case["act"]).to(DTYPES[case["out"]])


def _plain_wgrad(s, case):
    x = s["A"] if s["row_index"] is None else s["A"][s["row_index"].long()]
    a, _ = _padded(s, x)
    b, _ = _padded(s, s["B"])
    d = torch.bmm(a.transpose(1, 2), b)
    if s["C"] is not None:
        d = d + case["beta"] * s["C"]
    return d.to(DTYPES[case["out"]])


def _plain_lora(s, case):
    ids, n, r = s["ids"].long(), case["adapters"], case["rank"]
    x = s["X"].float()
    y = x @ s["W"].float()
    # every adapter's first product side by side; a row keeps its own adapter's
    u = (x @ s["LA"].float().permute(1, 0, 2).reshape(x.shape[1], n * r)).view(-1, n, r)
    keep = (ids[:, None] == torch.arange(n, device=ids.device)).float() * s["scale"]
    y = y + (u * keep[..., None]).view(-1, n * r) @ s["LB"].float().reshape(n * r, -1)
    return y.to(DTYPES[case["out"]])


# -------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "group":  # the numbers in; offsets, order and positions out
        return {"bytes": 4 * case["rows"] * 3 + 4 * (case["groups"] + 1), "flops": 0}
    e, o = BYTES[case["dtype"]], BYTES[case["out"]]
    if op == "lora":
        M, K, N, r = (case[k] for k in ("M", "K", "N", "rank"))
        active = sum(1 for x in _ragged(M - case["base"], case["adapters"], case["skew"]) if x)
        return {"bytes": e * (M * K + K * N + active * r * (K + N)) + o * M * N + 4 * M,
                "flops": 2 * M * K * N + 2 * (M - case["base"]) * r * (K + N)}
    rows, groups, N = case["rows"], case["groups"], case["N"]
    active = sum(1 for x in _ragged(rows, groups, case["skew"]) if x)
    stored = -(-rows // case["topk"]) if case["topk"] > 1 else rows
    index = 4 * rows if case["topk"] > 1 else 0
    if op == "grouped":
        K = case["K"]
        return {"bytes": e * (stored * K + active * K * N) + o * rows * N + index +
                4 * (groups + 1) + (4 * active * N if case["bias"] else 0),
                "flops": 2 * rows * K * N}
    M = case["M"]
    return {"bytes": e * (stored * M + rows * N) + groups * M * N * (o + (4 if case["beta"] else 0)) +
            index + 4 * (groups + 1),
            "flops": 2 * rows * M * N}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    if case["op"] == "group" or work(case)["flops"] > 2.5e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "lora":
        x = s["X"].double()
        y = x @ s["W"].double()
        ids = s["ids"].tolist()
        for a in sorted(set(ids)):
            if a < 0:
                continue
            mine = torch.tensor([i for i, b in enumerate(ids) if b == a], device=x.device)
            low = x[mine] @ s["LA"][a].double() * s["scale"][a].double()
            y[mine] += low @ s["LB"][a].double()
        return y
    bounds = s["offsets"].tolist()
    index = s["row_index"].long() if s["row_index"] is not None else None
    groups = case["groups"]
    if case["op"] == "grouped":
        y = torch.zeros((case["rows"], case["N"]), dtype=torch.float64, device="cuda")
    else:
        y = torch.zeros((groups, case["M"], case["N"]), dtype=torch.float64, device="cuda")
    for g in range(groups):
        lo, hi = bounds[g], bounds[g + 1]
        a = s["A"][lo:hi] if index is None else s["A"][index[lo:hi]]
        if case["op"] == "grouped":
            z = a.double() @ s["B"][g].double()
            if s["bias"] is not None:
                z = z + s["bias"][g].double()
            if case["act"] == RELU:
                z = torch.where(z > 0, z, torch.zeros_like(z))
            elif case["act"] == GELU:
                inner = (2.0 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)
                z = z / 2 * (1 + torch.tanh(inner))
            y[lo:hi] = z
        else:
            y[g] = a.double().t() @ s["B"][lo:hi].double()
            if s["C"] is not None:
                y[g] += case["beta"] * s["C"][g].double()
    return y
