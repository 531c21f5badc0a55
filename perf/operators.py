"""Measured cases of the expert layer's training and few-token operators.

Five operators: the spread of token rows over their expert rows (``dispatch``), the
weighted sum of expert rows per token (``combine``), the gradient of each, the gradient of
the top-k softmax routing (``route``), and the product of a few rows with 4-bit weights
(``matvec``, MXFP4 or NVFP4, one matrix or a bank of experts).

``run`` computes them in plain torch, in 32 bits, rounding once at the end; with ``own`` set
it makes the library's calls instead.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
ALPHA, LIMIT = 1.702, 7.0


def listed():
    return [
        # decode: the down products of one token's four experts, summed into its output
        {"name": "combine one token", "op": "combine", "T": 1, "k": 4, "E": 32, "H": 2880, "dtype": "bf16",
         "rows_dtype": "fp32", "weighted": True, "drop": 0.0},
        # prefill or a training forward pass of the gpt-oss-20b layer, a few pairs over capacity
        {"name": "combine prefill", "op": "combine", "T": 4096, "k": 4, "E": 32, "H": 2880, "dtype": "bf16",
         "rows_dtype": "bf16", "weighted": True, "drop": 0.02},
        # a training step of the gpt-oss-120b layer: gradients of the rows and of the routing weights
        {"name": "combine backward large", "op": "combine_backward", "T": 8192, "k": 4, "E": 128, "H": 2880,
         "dtype": "bf16", "rows_dtype": "bf16", "weighted": True, "drop": 0.0},
        # the same step's tokens on their way to the experts
        {"name": "dispatch large", "op": "dispatch", "T": 8192, "k": 4, "E": 128, "H": 2880, "dtype": "bf16",
         "rows_dtype": "bf16", "weighted": False, "drop": 0.0},
        # router weight on the input, an odd width, dropped pairs, half precision: both gradients
        {"name": "dispatch backward odd", "op": "dispatch_backward", "T": 1021, "k": 3, "E": 17, "H": 1001,
         "dtype": "fp16", "rows_dtype": "fp16", "weighted": True, "drop": 0.1},
        # the router's gradient: one micro batch, and a long one with the most experts per token
        {"name": "route backward", "op": "route", "T": 4096, "k": 4, "E": 32},
        {"name": "route backward long", "op": "route", "T": 65536, "k": 8, "E": 128},
        # one 4-bit projection of one token
        {"name": "matvec one row", "op": "matvec", "fmt": "mxfp4", "T": 1, "k": 1, "E": 1, "N": 2880, "K": 2880,
         "dtype": "bf16", "out": "bf16", "swiglu": False, "bias": True},
        # decode, one token: its four experts' gate and up products with the activation
        {"name": "matvec gate_up one token", "op": "matvec", "fmt": "mxfp4", "T": 1, "k": 4, "E": 32, "N": 5760,
         "K": 2880, "dtype": "bf16", "out": "bf16", "swiglu": True, "bias": True},
        # decode, eight tokens: the down products, one row per pair, kept in 32 bits for the sum
        {"name": "matvec down eight tokens", "op": "matvec", "fmt": "mxfp4", "T": 32, "k": 1, "E": 32, "N": 2880,
         "K": 2880, "dtype": "bf16", "out": "fp32", "swiglu": False, "bias": True},
        # decode, a batch of 64 tokens over the 128 experts of the gpt-oss-120b layer: nearly every expert is read
        {"name": "matvec gate_up batch", "op": "matvec", "fmt": "mxfp4", "T": 64, "k": 4, "E": 128, "N": 5760,
         "K": 2880, "dtype": "bf16", "out": "bf16", "swiglu": True, "bias": True},
        # NVFP4 banks, half precision, eight tokens
        {"name": "matvec nvfp4 gate_up", "op": "matvec", "fmt": "nvfp4", "T": 8, "k": 4, "E": 32, "N": 5760,
         "K": 2880, "dtype": "fp16", "out": "fp16", "swiglu": True, "bias": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_backward", "combine", "combine_backward", "route", "matvec", "matvec"])
    if op == "route":
        E = _log(rng, 1, 256)
        return {"op": op, "T": _log(rng, 1, 65536 if E <= 128 else 32768), "k": rng.randint(1, min(8, E)), "E": E}
    if op == "matvec":
        E, N, K = _log(rng, 1, 64), 2 * _log(rng, 8, 2880), 32 * _log(rng, 1, 180)
        k = rng.randint(1, min(4, E))
        dtype = rng.choice(["bf16", "fp16"])
        return {"op": op, "fmt": rng.choice(["mxfp4", "nvfp4"]), "T": _log(rng, 1, 48), "k": k, "E": E, "N": N, "K": K,
                "dtype": dtype, "out": rng.choice([dtype, "fp32"]), "swiglu": rng.random() < 0.5,
                "bias": rng.random() < 0.7}
    E, H = _log(rng, 1, 256), _log(rng, 32, 2880)
    dtype, rows = rng.choice([("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("bf16", "fp32"), ("fp16", "fp32")])
    if rng.random() < 0.5:
        H = (H + 7) // 8 * 8
    return {"op": op, "T": _log(rng, 1, 4096), "k": rng.randint(1, min(8, E)), "E": E, "H": H, "dtype": dtype,
            "rows_dtype": rows, "weighted": rng.random() < 0.8, "drop": rng.choice([0.0, 0.0, 0.05, 0.5])}


def _routing(gen, T, E, k):
    """Expert ids in decreasing order of random logits, and their softmax weights."""
    logits = torch.randn((T, E), device="cuda", generator=gen)
    val, ids = torch.topk(logits, k, dim=1)
    return ids.to(torch.int32), torch.softmax(val, dim=1)


def _rows(case):
    """Pairs that are not dropped: the expert rows."""
    P = case["T"] * case["k"]
    return max(1, P - int(P * case["drop"]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    T, k, E = case["T"], case["k"], case["E"]
    ids, weights = _routing(gen, T, E, k)
    s = {"case": case, "ids": ids, "weights": weights}
    randn = lambda shape, dtype: torch.randn(shape, device="cuda", generator=gen).to(DTYPES[dtype])  # noqa: E731
    if case["op"] == "route":
        s["dweights"] = randn((T, k), "fp32")
        return s
    if case["op"] == "matvec":
        N, K, block = case["N"], case["K"], 32 if case["fmt"] == "mxfp4" else 16
        s["x"] = randn((T, K), case["dtype"])
        s["row_ids"] = ids.reshape(-1).contiguous() if E > 1 else None
        s["blocks"] = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
        lo, hi = (118, 126) if case["fmt"] == "mxfp4" else (0x08, 0x37)
        s["scales"] = torch.randint(lo, hi + 1, (E, N, K // block), dtype=torch.uint8, device="cuda", generator=gen)
        shape2 = (E, 2) if case["swiglu"] else (E,)
        s["scale2"] = (0.5 + 0.5 * torch.rand(shape2, device="cuda", generator=gen)) if case["fmt"] == "nvfp4" else None
        s["bias"] = 0.02 * randn((E, N), "fp32") if case["bias"] else None
        return s
    H = case["H"]
    n = _rows(case)
    kept = torch.ones(T * k, dtype=torch.bool, device="cuda")
    kept[torch.randperm(T * k, device="cuda", generator=gen)[n:]] = False
    expert = torch.where(kept, ids.reshape(-1).long(), E)              # dropped pairs go behind the last expert
    order = torch.argsort(expert, stable=True)
    row = torch.empty(T * k, dtype=torch.int64, device="cuda")
    row[order] = torch.arange(T * k, device="cuda")
    s["pair_rows"] = torch.where(kept, row, -1).to(torch.int32)
    s["rows_n"] = n
    if not case["weighted"]:
        s["weights"] = None
    tok, rows = case["dtype"], case["rows_dtype"]
    if case["op"] in ("dispatch", "dispatch_backward"):
        s["x"] = randn((T, H), tok)
    if case["op"] == "dispatch_backward":
        s["drows"] = randn((s["rows_n"], H), rows)
    if case["op"] in ("combine", "combine_backward"):
        s["y_rows"] = randn((s["rows_n"], H), rows)
    if case["op"] == "combine_backward":
        s["dout"] = randn((T, H), tok)
    return s


def _spread(a, s, rows_dtype):
    """rows[r(p)] = s_p a[t]"""
    c = s["case"]
    p = (a.float()[:, None, :] * (s["weights"][:, :, None] if c["weighted"] else 1.0)).expand(-1, c["k"], -1)
    valid = s["pair_rows"] >= 0
    rows = torch.zeros((s["rows_n"], c["H"]), dtype=DTYPES[rows_dtype], device="cuda")
    rows[s["pair_rows"][valid].long()] = p.reshape(-1, c["H"])[valid].to(DTYPES[rows_dtype])
    return rows


def _collect(rows, s):
    """The expert rows of every pair in 32 bits, zero where the pair was dropped: [T, k, H]."""
    c = s["case"]
    got = rows.float()[s["pair_rows"].clamp(min=0).long()]
    got = torch.where((s["pair_rows"] >= 0)[:, None], got, torch.zeros((), device="cuda"))
    return got.view(c["T"], c["k"], c["H"])


def _sum(rows, s):
    got = _collect(rows, s)
    got = got * s["weights"][:, :, None] if s["case"]["weighted"] else got
    return got.sum(dim=1).to(DTYPES[s["case"]["dtype"]])


def _dots(a, rows, s):
    return (_collect(rows, s) * a.float()[:, None, :]).sum(dim=2)


def _route_backward(s):
    c, w, dw = s["case"], s["weights"], s["dweights"]
    g = w * (dw - (w * dw).sum(dim=1, keepdim=True))
    return torch.zeros((c["T"], c["E"]), device="cuda").scatter_(1, s["ids"].long(), g)


def _decode(blocks, scales, fmt):
    """The bank's weights in 32 bits: [..., N, K]."""
    value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    codes = torch.stack((blocks & 15, blocks >> 4), dim=-1).flatten(-2)
    w = value[codes.int()]
    if fmt == "mxfp4":
        scale = torch.exp2(scales.float() - 127.0)
        block = 32
    else:
        scale = scales.view(torch.float8_e4m3fn).float()
        block = 16
    return (w.unflatten(-1, (-1, block)) * scale[..., None]).flatten(-2)


def _matvec(s):
    c = s["case"]
    N = c["N"]
    x = s["x"].float()
    if s["row_ids"] is None:
        e = torch.zeros(c["T"] * c["k"], dtype=torch.int64, device="cuda")
    else:
        e = s["row_ids"].long()
    x = x.repeat_interleave(c["k"], dim=0)
    R = e.numel()
    if R <= c["E"]:                      # each row's own matrix
        y = torch.bmm(_decode(s["blocks"][e], s["scales"][e], c["fmt"]), x[:, :, None])[:, :, 0]
    else:                                # every row with every matrix, then its own
        y = torch.matmul(x, _decode(s["blocks"], s["scales"], c["fmt"]).transpose(1, 2))[e, torch.arange(R, device="cuda")]
    if s["scale2"] is not None:
        y = y * (s["scale2"][e].repeat(1, N // 2) if c["swiglu"] else s["scale2"][e][:, None])
    if s["bias"] is not None:
        y = y + s["bias"][e]
    if c["swiglu"]:
        gate = y[:, 0::2].clamp(max=LIMIT)
        up = y[:, 1::2].clamp(min=-LIMIT, max=LIMIT)
        y = (up + 1) * (gate / (1 + torch.exp(-ALPHA * gate)))
    return y.to(DTYPES[c["out"]])


def _own(s):
    import mxfp4_expert_ffn_moe_b200 as moe
    c = s["case"]
    T, k = c["T"], c["k"]
    if c["op"] == "route":
        return moe.moe_route_backward(s["dweights"], s["ids"], s["weights"], c["E"])
    if c["op"] == "matvec":
        args = dict(bias=s["bias"], row_ids=s["row_ids"], rows_per_x=k, swiglu=c["swiglu"], alpha=ALPHA, limit=LIMIT,
                    out_dtype=DTYPES[c["out"]])
        if c["fmt"] == "nvfp4":
            return moe.nvfp4_matvec(s["x"], s["blocks"], s["scales"], s["scale2"], **args)
        return moe.mxfp4_matvec(s["x"], s["blocks"], s["scales"], **args)
    tok, rows = DTYPES[c["dtype"]], DTYPES[c["rows_dtype"]]
    if c["op"] == "dispatch":
        return moe.moe_dispatch_rows(s["x"], s["pair_rows"], k, weights=s["weights"], n_rows=s["rows_n"], dtype=rows)
    if c["op"] == "dispatch_backward":
        return moe.moe_dispatch_rows_backward(s["drows"], s["pair_rows"], T, k, weights=s["weights"],
                                              x=s["x"] if c["weighted"] else None, dtype=tok)
    if c["op"] == "combine":
        return moe.moe_combine_rows(s["y_rows"], s["pair_rows"], T, k, weights=s["weights"], dtype=tok)
    return moe.moe_combine_rows_backward(s["dout"], s["pair_rows"], k, weights=s["weights"],
                                         y_rows=s["y_rows"] if c["weighted"] else None, n_rows=s["rows_n"], dtype=rows)


def run(state):
    if own:
        return _own(state)
    s, c = state, state["case"]
    if c["op"] == "route":
        return _route_backward(s)
    if c["op"] == "matvec":
        return _matvec(s)
    if c["op"] == "dispatch":
        return _spread(s["x"], s, c["rows_dtype"])
    if c["op"] == "dispatch_backward":
        dx = _sum(s["drows"], s)
        return (dx, _dots(s["x"], s["drows"], s)) if c["weighted"] else dx
    if c["op"] == "combine":
        return _sum(s["y_rows"], s)
    drows = _spread(s["dout"], s, c["rows_dtype"])
    return (drows, _dots(s["dout"], s["y_rows"], s)) if c["weighted"] else drows


def work(case):
    c = case
    P = c["T"] * c["k"]
    if c["op"] == "route":
        return {"bytes": 12 * P + 4 * c["T"] * c["E"], "flops": 4 * P}
    if c["op"] == "matvec":
        N, K, E = c["N"], c["K"], c["E"]
        touched = E * (1 - (1 - c["k"] / E) ** c["T"])          # experts that get a row, on average
        per = N * K // 2 + N * K // (32 if c["fmt"] == "mxfp4" else 16) + (4 * N if c["bias"] else 0)
        out = P * (N // 2 if c["swiglu"] else N) * SIZE[c["out"]]
        return {"bytes": int(touched * per) + c["T"] * K * 2 + out + 4 * P, "flops": 2 * P * N * K}
    H, tok, row = c["H"], SIZE[c["dtype"]], SIZE[c["rows_dtype"]]
    rows = _rows(c)
    backward = c["op"].endswith("_backward")
    n = c["T"] * H * tok + rows * H * row + P * (8 if c["weighted"] else 4)
    if backward and c["weighted"]:
        # the other operand of the dots (the token rows again, or the expert rows again) and the weights' gradient
        n += (c["T"] * H * tok if c["op"] == "dispatch_backward" else rows * H * row) + 4 * P
    return {"bytes": n, "flops": rows * H * (4 if backward and c["weighted"] else 2)}


def exact(case, seed):
    """The definitions in 64 bits: pair by pair over the slots, expert by expert over the banks."""
    s, c = prepare(case, seed), case
    T, k, E = c["T"], c["k"], c["E"]
    f64 = torch.float64
    if c["op"] == "route":
        w, dw, ids = s["weights"].to(f64), s["dweights"].to(f64), s["ids"].long()
        out = torch.zeros((T, E), dtype=f64, device="cuda")
        t = torch.arange(T, device="cuda")
        for j in range(k):                 # d w_i / d l_j = w_i (delta_ij - w_j)
            g = torch.zeros(T, dtype=f64, device="cuda")
            for i in range(k):
                g += dw[:, i] * w[:, i] * ((1.0 if i == j else 0.0) - w[:, j])
            out[t, ids[:, j]] += g
        return out
    if c["op"] == "matvec":
        N, K = c["N"], c["K"]
        e = torch.zeros(T * k, dtype=torch.int64, device="cuda") if s["row_ids"] is None else s["row_ids"].long()
        y = torch.zeros((T * k, N), dtype=f64, device="cuda")
        for expert in e.unique().tolist():
            r = (e == expert).nonzero()[:, 0]
            b = s["blocks"][expert].long()
            w = torch.empty((N, K), dtype=f64, device="cuda")
            for half, code in ((0, b % 16), (1, b // 16)):
                m, x2 = code % 2, (code // 2) % 4
                mag = torch.where(x2 == 0, 0.5 * m.to(f64), torch.ldexp(1 + 0.5 * m.to(f64), x2 - 1))
                w[:, half::2] = torch.where(code >= 8, -mag, mag)
            sc = s["scales"][expert].long()
            if c["fmt"] == "mxfp4":
                scale, block = torch.ldexp(torch.ones((), dtype=f64, device="cuda"), sc - 127), 32
            else:
                ex, m = (sc // 8) % 16, (sc % 8).to(f64)
                scale, block = torch.where(ex == 0, torch.ldexp(m, torch.full_like(ex, -9)), torch.ldexp(8 + m, ex - 10)), 16
            w *= scale.repeat_interleave(block, dim=1)
            part = s["x"][r // k].to(f64) @ w.T
            if s["scale2"] is not None:
                s2 = s["scale2"][expert].to(f64)
                if c["swiglu"]:
                    part[:, 0::2] *= s2[0]
                    part[:, 1::2] *= s2[1]
                else:
                    part *= s2
            if s["bias"] is not None:
                part += s["bias"][expert].to(f64)
            y[r] = part
        if not c["swiglu"]:
            return y
        gate, up = torch.minimum(y[:, ::2], torch.full((), LIMIT, dtype=f64, device="cuda")), y[:, 1::2].clamp(-LIMIT, LIMIT)
        return (up + 1) * gate * torch.sigmoid(ALPHA * gate)
    H = c["H"]
    rows_of = s["pair_rows"].view(T, k).long()
    weight = s["weights"].to(f64) if c["weighted"] else torch.ones((T, k), dtype=f64, device="cuda")
    if c["op"] in ("dispatch", "combine_backward"):
        a = s["x" if c["op"] == "dispatch" else "dout"].to(f64)
        rows = torch.zeros((s["rows_n"], H), dtype=f64, device="cuda")
        dots = torch.zeros((T, k), dtype=f64, device="cuda")
        for j in range(k):
            t = (rows_of[:, j] >= 0).nonzero()[:, 0]
            r = rows_of[t, j]
            rows[r] = weight[t, j, None] * a[t]
            if c["op"] == "combine_backward" and c["weighted"]:
                dots[t, j] = torch.einsum("th,th->t", a[t], s["y_rows"][r].to(f64))
        return (rows, dots) if c["op"] == "combine_backward" and c["weighted"] else rows
    src = s["drows" if c["op"] == "dispatch_backward" else "y_rows"]
    out = torch.zeros((T, H), dtype=f64, device="cuda")
    dots = torch.zeros((T, k), dtype=f64, device="cuda")
    for j in range(k):
        t = (rows_of[:, j] >= 0).nonzero()[:, 0]
        part = src[rows_of[t, j]].to(f64)
        out[t] += weight[t, j, None] * part
        if c["op"] == "dispatch_backward" and c["weighted"]:
            dots[t, j] = torch.einsum("th,th->t", s["x"][t].to(f64), part)
    return (out, dots) if c["op"] == "dispatch_backward" and c["weighted"] else out
