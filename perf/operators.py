"""Measured cases of the operators around the expert layer: the experts'
unquantised products and their gradients, the norms before and after the block,
and the 4-bit matrix-vector product.

`run` computes an operator in its plain form (elementary torch operations in
fp32, rounded once) or, where `own` is true, calls the framework's kernels.
"""
import random

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64

# 384 experts over 8 ranks leave 48 on a rank; H = 7168 and I = 2048 are widths
# of the repository's own workloads, 2I = 4096 rows of gate and up.
LARGEST_PRODUCT = 6144 * 4096 * 7168
LARGEST_EXPERTS = 48 * 4096 * 7168
LARGEST_ROWS = 8192 * 7168
LARGEST_MATRIX = 16384 * 7168


def listed():
    return [
        # one token's eight experts on a rank, gate and up product: latency and the weight stream
        {"name": "product, one token", "op": "product", "E": 48, "rows": 8, "spare": 0, "N": 4096, "K": 7168,
         "load": "uniform"},
        # a 1024-token prefill with top-6, 128 rows an expert
        {"name": "product, prefill", "op": "product", "E": 48, "rows": 6144, "spare": 0, "N": 4096, "K": 7168,
         "load": "uniform"},
        # popular and idle experts, odd sizes, a batch padded to its capacity
        {"name": "product, ragged", "op": "product", "E": 37, "rows": 4999, "spare": 121, "N": 1416, "K": 2056,
         "load": "zipf"},
        # a fine-tuning step's backward pass: the gradient of the rows
        {"name": "input gradient", "op": "input gradient", "E": 16, "rows": 16384, "spare": 0, "N": 4096, "K": 2048,
         "load": "uniform"},
        # and of the weights, with uneven experts
        {"name": "weight gradient", "op": "weight gradient", "E": 16, "rows": 16384, "spare": 0, "N": 4096, "K": 2048,
         "load": "zipf"},
        # a decode batch's norm into the layer's quantised input
        {"name": "norm before, decode", "op": "norm before", "T": 8, "H": 7168, "out": "both"},
        # the same for a prefill
        {"name": "norm before, prefill", "op": "norm before", "T": 8192, "H": 7168, "out": "fp8"},
        # training: forward, then the gradients joined with the residual's
        {"name": "norm before, training", "op": "norm before training", "T": 4099, "H": 4096},
        # a decode batch's norm of the block's output, gated per channel, into the residual stream
        {"name": "norm after, decode", "op": "norm after", "T": 8, "H": 7168, "gate": "channel"},
        # training with a gate of the rows' own
        {"name": "norm after, training", "op": "norm after training", "T": 8192, "H": 7168, "gate": "channel"},
        # one token through a dense projection held in 4 bits
        {"name": "matvec, one token", "op": "matvec", "T": 1, "N": 14336, "K": 7168, "fmt": "mx"},
        # a few tokens, the other format, an odd number of outputs
        {"name": "matvec, odd", "op": "matvec", "T": 7, "N": 4099, "K": 2080, "fmt": "nvfp4"},
    ]


def _log(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def draw(rng):
    op = rng.choice(["product", "product", "input gradient", "weight gradient", "norm before", "norm before training",
                     "norm after", "norm after training", "matvec", "matvec"])
    if op in ("product", "input gradient", "weight gradient"):
        E, rows = _log(rng, 1, 64), _log(rng, 1, 16384)
        N, K = 8 * _log(rng, 8, 896), 8 * _log(rng, 8, 896)
        while E * N * K > LARGEST_EXPERTS:
            E = max(1, E // 2)
        while rows * N * K > LARGEST_PRODUCT:
            rows = rows * 2 // 3
        return {"op": op, "E": E, "rows": rows, "spare": rng.choice([0, 0, rng.randint(1, 200)]), "N": N, "K": K,
                "load": rng.choice(["uniform", "zipf"])}
    if op == "matvec":
        N, K = _log(rng, 17, 16384), 32 * _log(rng, 4, 256)
        while N * K > LARGEST_MATRIX:
            N = N * 2 // 3
        return {"op": op, "T": _log(rng, 1, 16), "N": N, "K": K, "fmt": rng.choice(["mx", "nvfp4"])}
    T, H = _log(rng, 1, 16384), 32 * _log(rng, 4, 512)
    while T * H > LARGEST_ROWS:
        T = T * 2 // 3
    if op == "norm before":
        return {"op": op, "T": T, "H": H, "out": rng.choice(["bf16", "fp8", "both"])}
    if op == "norm before training":
        return {"op": op, "T": T, "H": H}
    return {"op": op, "T": T, "H": H, "gate": rng.choice(["none", "channel", "token", "full"])}


def _sizes(case):
    """Rows of each expert: every row goes to an expert drawn uniformly or by a
    popularity that falls with the expert's rank; experts may stay empty."""
    rng = random.Random(case["rows"] * 1000003 + case["E"])
    E = case["E"]
    weights = [1.0 / (e + 1) ** 1.2 if case["load"] == "zipf" else 1.0 for e in range(E)]
    rng.shuffle(weights)
    sizes = [0] * E
    for e in rng.choices(range(E), weights, k=case["rows"]):
        sizes[e] += 1
    return sizes


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, mean=0.0):
        t = torch.randn(shape, dtype=BF16, device="cuda", generator=g).mul_(scale)
        return t.add_(mean) if mean else t

    s = dict(case)
    op = case["op"]
    if op in ("product", "input gradient", "weight gradient"):
        E, N, K = case["E"], case["N"], case["K"]
        R = case["rows"] + case["spare"]
        ends = [0]
        for n in _sizes(case):
            ends.append(ends[-1] + n)
        s["ends"] = ends
        s["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        if op != "input gradient":
            s["x"] = normal(R, K, scale=0.5)
        if op != "product":
            s["dy"] = normal(R, N, scale=0.5)
        if op != "weight gradient":
            s["w"] = normal(E, N, K, scale=0.04)
    elif op == "matvec":
        T, N, K = case["T"], case["N"], case["K"]
        s["x"] = normal(T, K, scale=0.5)
        s["w"] = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
        # scales as quantised weights of deviation 0.04 have them: 2^-8 to 2^-5
        if case["fmt"] == "mx":
            s["w_sf"] = torch.randint(119, 123, (N, K // 32), dtype=torch.uint8, device="cuda", generator=g)
        else:
            s["w_sf"] = torch.randint(1, 17, (N, K // 16), dtype=torch.uint8, device="cuda", generator=g)
    else:
        T, H = case["T"], case["H"]
        s["x"] = normal(T, H, scale=0.5)
        s["weight"] = normal(H, scale=0.1, mean=1.0)
        if op == "norm before training":
            s["dy"], s["dresidual"] = normal(T, H), normal(T, H)
        if op.startswith("norm after"):
            s["residual"] = normal(T, H)
            s["gate_kind"] = case["gate"]
            shape = {"channel": (H,), "token": (T, 1), "full": (T, H)}.get(case["gate"])
            s["gate"] = normal(*shape, scale=0.2, mean=0.5) if shape else None
            if op.endswith("training"):
                s["dout"] = normal(T, H)
    return s


EPS = 1e-6
RESIDUAL_SCALE = 0.75


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import moe_expert_layer_08_b200 as moe

    op = s["op"]
    if op == "product":
        return moe.grouped_matmul(s["x"], s["w"], s["offsets"])
    if op == "input gradient":
        return moe.grouped_matmul_grad_input(s["dy"], s["w"], s["offsets"])
    if op == "weight gradient":
        return moe.grouped_matmul_grad_weight(s["dy"], s["x"], s["offsets"])
    if op == "matvec":
        return moe.fp4_matvec(s["x"], s["w"], s["w_sf"], fmt=s["fmt"])
    if op == "norm before":
        n = moe.norm_before(s["x"], s["weight"], EPS, bf16=s["out"] != "fp8", fp8=s["out"] != "bf16")
        out = {} if n.y is None else {"y": n.y}
        if n.x_fp8 is not None:
            out["codes"] = n.x_fp8.view(torch.float8_e4m3fn)
            out["scales"] = n.x_sf.view(torch.float8_e8m0fnu)
        return out
    if op == "norm before training":
        n = moe.norm_before(s["x"], s["weight"], EPS, rstd=True)
        dx, dweight = moe.norm_before_backward(s["dy"], s["x"], s["weight"], n.rstd, dresidual=s["dresidual"])
        return {"y": n.y, "dx": dx, "dweight": dweight}
    if op == "norm after":
        return moe.norm_after(s["x"], s["residual"], s["weight"], EPS, gate=s["gate"],
                              residual_scale=RESIDUAL_SCALE).out
    n = moe.norm_after(s["x"], s["residual"], s["weight"], EPS, gate=s["gate"], residual_scale=RESIDUAL_SCALE,
                       rstd=True)
    dx, dresidual, dweight, dgate = moe.norm_after_backward(s["dout"], s["x"], s["weight"], n.rstd, gate=s["gate"],
                                                            residual_scale=RESIDUAL_SCALE)
    return {"out": n.out, "dx": dx, "dresidual": dresidual, "dweight": dweight, "dgate": dgate}


# ------------------------------------------------------------------ plain forms
def _plain(s):
    op = s["op"]
    if op == "product":
        return _plain_rows(s, s["x"], s["N"], lambda x, w: x @ w.T)
    if op == "input gradient":
        return _plain_rows(s, s["dy"], s["K"], lambda dy, w: dy @ w)
    if op == "weight gradient":
        # an expert without rows has a zero gradient: the product over no rows
        ends = s["ends"]
        return torch.stack([(s["dy"][a:b].to(F32).T @ s["x"][a:b].to(F32)).to(BF16)
                            for a, b in zip(ends[:-1], ends[1:])])
    if op == "matvec":
        return _plain_matvec(s)
    if op == "norm before":
        return _plain_before(s)
    if op == "norm before training":
        x, w, dy = s["x"].to(F32), s["weight"].to(F32), s["dy"].to(F32)
        rstd = _plain_rstd(x)
        xhat = x * rstd
        dxhat = dy * w
        dx = rstd * (dxhat - xhat * (dxhat * xhat).mean(1, keepdim=True)) + s["dresidual"].to(F32)
        return {"y": (xhat * w).to(BF16), "dx": dx.to(BF16), "dweight": (dy * xhat).sum(0)}
    x, w = s["x"].to(F32), s["weight"].to(F32)
    gate = 1.0 if s["gate"] is None else s["gate"].to(F32)
    rstd = _plain_rstd(x)
    xhat = x * rstd
    z = xhat * w
    out = (RESIDUAL_SCALE * s["residual"].to(F32) + gate * z).to(BF16)
    if op == "norm after":
        return out
    dout = s["dout"].to(F32)
    dz = dout * gate
    dxhat = dz * w
    dx = rstd * (dxhat - xhat * (dxhat * xhat).mean(1, keepdim=True))
    dgate = None
    if s["gate"] is not None:
        dgate = dout * z
        dgate = {"channel": lambda v: v.sum(0), "token": lambda v: v.sum(1, keepdim=True),
                 "full": lambda v: v.to(BF16)}[s["gate_kind"]](dgate)
    return {"out": out, "dx": dx.to(BF16), "dresidual": (RESIDUAL_SCALE * dout).to(BF16),
            "dweight": (dz * xhat).sum(0), "dgate": dgate}


def _plain_rows(s, rows, columns, product):
    """The product of each expert's rows with its weights; zeros for the rows
    of no expert."""
    ends = s["ends"]
    parts = [product(rows[a:b].to(F32), s["w"][e].to(F32)).to(BF16)
             for e, (a, b) in enumerate(zip(ends[:-1], ends[1:])) if b > a]
    parts.append(torch.zeros((rows.shape[0] - ends[-1], columns), dtype=BF16, device=rows.device))
    return torch.cat(parts)


def _plain_rstd(x):
    return torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)


def _plain_before(s):
    x = s["x"].to(F32)
    y = (x * _plain_rstd(x) * s["weight"].to(F32)).to(BF16)
    out = {} if s["out"] == "fp8" else {"y": y}
    if s["out"] != "bf16":
        v = y.to(F32).view(s["T"], -1, 32)
        # the smallest e with amax <= 448 * 2^e, 448 = 0.875 * 2^9; a group of zeros has e = 0
        amax = v.abs().amax(2)
        m, e = torch.frexp(amax)
        e = torch.where(amax > 0, e - 8 - (m <= 0.875).to(torch.int32), 0).clamp(-127, 127)
        codes = torch.ldexp(v, -e[:, :, None]).to(torch.float8_e4m3fn)
        out["codes"] = codes.view(s["T"], s["H"])
        out["scales"] = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return out


def _plain_matvec(s):
    T, N, K = s["T"], s["N"], s["K"]
    values = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                          device="cuda")
    codes = torch.stack([s["w"] & 15, s["w"] >> 4], 2).view(N, K)
    if s["fmt"] == "mx":
        scales = torch.ldexp(torch.ones((), device="cuda"), s["w_sf"].to(torch.int32) - 127)
    else:
        scales = s["w_sf"].view(torch.float8_e4m3fn).to(F32)
    w = values[codes.to(torch.int32)].view(N, scales.shape[1], -1) * scales[:, :, None]
    return (s["x"].to(F32) @ w.view(N, K).T).to(BF16)


# ------------------------------------------------------------------ what a pass needs
def work(case):
    op = case["op"]
    if op in ("product", "input gradient", "weight gradient"):
        E, N, K, R, spare = case["E"], case["N"], case["K"], case["rows"], case["spare"]
        used = sum(1 for n in _sizes(case) if n)
        flops = 2.0 * R * N * K
        if op == "weight gradient":
            return {"bytes": 2.0 * (R * (N + K) + E * N * K), "flops": flops}
        written = N if op == "product" else K
        return {"bytes": 2.0 * (R * (N + K) + used * N * K + spare * written), "flops": flops}
    if op == "matvec":
        T, N, K = case["T"], case["N"], case["K"]
        group = 32 if case["fmt"] == "mx" else 16
        return {"bytes": N * K * (0.5 + 1.0 / group) + 2.0 * T * (N + K), "flops": 2.0 * T * N * K}
    T, H = case["T"], case["H"]
    n = float(T) * H
    if op == "norm before":
        y = {"bf16": 2.0, "fp8": 33 / 32, "both": 2.0 + 33 / 32}[case["out"]]
        return {"bytes": n * (2 + y) + 2.0 * H, "flops": 5 * n}
    if op == "norm before training":
        return {"bytes": n * 2 * 5 + 6.0 * H, "flops": 14 * n}
    gate = {"none": 0.0, "channel": 2.0 * H, "token": 2.0 * T, "full": 2.0 * n}[case["gate"]]
    if op == "norm after":
        return {"bytes": n * 2 * 3 + 2.0 * H + gate, "flops": 7 * n}
    # forward: x, residual and out; backward: dout, dx and dresidual; x is read once
    gates = {"none": 0.0, "channel": 6.0 * H, "token": 6.0 * T, "full": 4.0 * n}[case["gate"]]
    return {"bytes": n * 2 * 6 + 6.0 * H + gates, "flops": 20 * n}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("product", "input gradient"):
        source, columns = ("x", case["N"]) if op == "product" else ("dy", case["K"])
        rows = s[source].to(F64)
        out = torch.zeros((rows.shape[0], columns), dtype=F64, device="cuda")
        start = 0
        for e, n in enumerate(_sizes(case)):
            w = s["w"][e].to(F64) if n else None
            if n:
                out[start:start + n] = torch.einsum("rk,nk->rn" if op == "product" else "rn,nk->rk",
                                                    rows[start:start + n], w)
            start += n
        return out
    if op == "weight gradient":
        out = torch.zeros((case["E"], case["N"], case["K"]), dtype=F64, device="cuda")
        start = 0
        for e, n in enumerate(_sizes(case)):
            out[e] = torch.einsum("rn,rk->nk", s["dy"][start:start + n].to(F64), s["x"][start:start + n].to(F64))
            start += n
        return out
    if op == "matvec":
        return _exact_matvec(case, s)
    x, w = s["x"].to(F64), s["weight"].to(F64)
    H = case["H"]
    r = (x.pow(2).sum(1) / H + EPS).pow(-0.5)
    if op == "norm before":
        y = torch.einsum("th,t,h->th", x, r, w)
        out = {} if case["out"] == "fp8" else {"y": y}
        if case["out"] != "bf16":
            # the operator quantises the rounded norm; scales by a search over the powers of two
            v = y.to(BF16).to(F64).reshape(-1, 32)
            amax = v.abs().max(1).values
            powers = torch.pow(torch.tensor(2.0, dtype=F64, device="cuda"),
                               torch.arange(-127, 128, dtype=F64, device="cuda"))
            scale = powers[torch.searchsorted(448.0 * powers, amax).clamp(max=254)]
            scale[amax == 0] = 1.0
            out["codes"] = _to_e4m3(v / scale[:, None]).reshape(case["T"], H)
            out["scales"] = scale.reshape(case["T"], H // 32)
        return out
    if op == "norm before training":
        dy = s["dy"].to(F64)
        dot = torch.einsum("th,h,th->t", dy, w, x) / H
        dx = torch.einsum("th,h,t->th", dy, w, r) - x * (dot * r.pow(3))[:, None] + s["dresidual"].to(F64)
        return {"y": torch.einsum("th,t,h->th", x, r, w), "dx": dx, "dweight": torch.einsum("th,th,t->h", dy, x, r)}
    gate = torch.ones((), dtype=F64, device="cuda") if s["gate"] is None else s["gate"].to(F64)
    gate = gate.expand(case["T"], H)
    z = torch.einsum("th,t,h->th", x, r, w)
    out = gate * z + s["residual"].to(F64) * RESIDUAL_SCALE
    if op == "norm after":
        return out
    dout = s["dout"].to(F64)
    dz = dout * gate
    dot = torch.einsum("th,h,th->t", dz, w, x) / H
    dx = torch.einsum("th,h,t->th", dz, w, r) - x * (dot * r.pow(3))[:, None]
    dgate = {"none": lambda: None, "channel": lambda: torch.einsum("th,th->h", dout, z),
             "token": lambda: torch.einsum("th,th->t", dout, z)[:, None], "full": lambda: dout * z}[case["gate"]]()
    return {"out": out, "dx": dx, "dresidual": dout * RESIDUAL_SCALE, "dweight": torch.einsum("th,th,t->h", dz, x, r),
            "dgate": dgate}


def _to_e4m3(v):
    """Nearest E4M3 value, ties to even: steps of 2^(exponent - 3), 2^-9 below 2^-6."""
    exponent = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.pow(torch.tensor(2.0, dtype=F64, device=v.device), exponent - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_matvec(case, s):
    T, N, K = case["T"], case["N"], case["K"]
    w = torch.empty((N, K), dtype=F64, device="cuda")
    for half, code in enumerate((s["w"] % 16, s["w"] // 16)):
        code = code.to(F64)
        sign = torch.where(code >= 8, -1.0, 1.0)
        mag = code % 8
        field, odd = torch.floor(mag / 2), mag % 2
        w[:, half::2] = sign * torch.where(field > 0, torch.exp2(field - 1) * (1 + odd / 2), odd / 2)
    sf = s["w_sf"].to(F64)
    if case["fmt"] == "mx":
        scale = torch.exp2(sf - 127)
    else:
        field, frac = torch.floor(sf / 8), sf % 8
        scale = torch.where(field > 0, torch.exp2(field - 7) * (1 + frac / 8), frac * 2.0 ** -9)
    w = w * scale.repeat_interleave(K // scale.shape[1], 1)
    return torch.einsum("tk,nk->tn", s["x"].to(F64), w)
