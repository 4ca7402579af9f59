"""Cases of the 8-bit integer operators (quantisation per row, dense and grouped products, gate/up with SwiGLU) and of the
rows' way to their experts and back (dispatch, combine, and both backward passes).

`run` computes an operator in its plain form (elementary torch operations), or, where `own` is set, by the library's call.
A row of codes in -127..127 carries one fp32 scale (a token of activations, an output channel of weights); a value is
code * scale.  `inv` gives the grouped row of each (token, slot), as moe_permute writes it.
"""
import math

import torch

own = False
DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
MOST_FLOPS, MOST_BYTES = 1.9e11, 3.4e8   # a drawn case's work stays below the largest listed one's


def listed():
    return [
        # activations of one token of a decode step (latency), from the fp32 residual stream's norm
        {"name": "quant_one_token", "op": "quant", "rows": 1, "cols": 2048, "x": "f32"},
        # h of a prefill on its way to the down projection
        {"name": "quant_prefill_h", "op": "quant", "rows": 8192, "cols": 2816, "x": "bf16"},
        # dense projection of one token: the weights are streamed
        {"name": "gemm_one_token", "op": "gemm", "T": 1, "K": 2048, "N": 5632, "out": "bf16"},
        # the same projection over a prefill: bound by the tensor cores
        {"name": "gemm_prefill", "op": "gemm", "T": 8192, "K": 2048, "N": 5632, "out": "bf16"},
        # down projection of a decode batch over 16 experts, ragged groups of about 4 rows
        {"name": "grouped_decode", "op": "grouped", "T": 64, "E": 16, "k": 1, "K": 2816, "N": 2048, "out": "f32", "gather": False},
        # down projection of a prefill over 64 experts, top-2
        {"name": "grouped_prefill", "op": "grouped", "T": 8192, "E": 64, "k": 2, "K": 512, "N": 1024, "out": "bf16", "gather": False},
        # gate/up + SwiGLU of a decode batch (64 streams x a pair): every expert's weights for 4 rows each
        {"name": "gate_up_decode", "op": "gate_up", "T": 128, "E": 64, "k": 2, "d": 1024, "F": 512, "out": "bf16"},
        # gate/up + SwiGLU of a prefill over 16 wide experts, top-1
        {"name": "gate_up_prefill", "op": "gate_up", "T": 4096, "E": 16, "k": 1, "d": 2048, "F": 2816, "out": "bf16"},
        # a prefill's rows into expert order
        {"name": "dispatch_prefill", "op": "dispatch", "backward": False, "T": 8192, "k": 2, "d": 1024, "x": "bf16"},
        # the gradient of an odd batch in fp32, a width that is no multiple of anything much
        {"name": "dispatch_backward_odd", "op": "dispatch", "backward": True, "T": 999, "k": 3, "d": 1001, "x": "f32"},
        # a decode batch's expert outputs back to tokens, into the fp32 residual stream
        {"name": "combine_decode", "op": "combine", "backward": False, "T": 128, "k": 2, "d": 1024, "x": "bf16", "out": "f32"},
        # the gradients of a training batch's combine: of the expert outputs and of the routing weights
        {"name": "combine_backward_train", "op": "combine", "backward": True, "T": 16384, "k": 2, "d": 2048, "x": "bf16", "out": "bf16"},
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi):   # multiples of 16 (rows of codes are read in 16-byte pieces)
        return 16 * log_int(lo / 16, hi / 16)

    op = rng.choice(["quant", "gemm", "grouped", "gate_up", "dispatch", "combine"])
    kind = rng.choice(["f32", "bf16"])
    if op == "quant":
        case = {"op": op, "rows": log_int(1, 16384), "cols": width(128, 8192), "x": kind}
    elif op == "gemm":
        case = {"op": op, "T": log_int(1, 8192), "K": width(128, 8192), "N": log_int(128, 8192), "out": kind}
    elif op in ("dispatch", "combine"):
        case = {"op": op, "backward": rng.random() < 0.5, "T": log_int(1, 16384), "k": rng.randint(1, 8), "d": log_int(64, 8192), "x": kind}
        if op == "combine":
            case["out"] = rng.choice(["f32", "bf16"])
    else:
        E = log_int(1, 128)
        case = {"op": op, "T": log_int(1, 8192), "E": E, "k": rng.randint(1, min(E, 8)), "out": kind}
        if op == "grouped":
            case |= {"K": width(128, 4096), "N": log_int(128, 4096), "gather": rng.random() < 0.5}
        else:
            case |= {"d": width(128, 4096), "F": log_int(128, 4096)}
    key = "rows" if op == "quant" else "T"
    while work(case)["flops"] > MOST_FLOPS or work(case)["bytes"] > MOST_BYTES:   # few rows first, then fewer experts
        if case[key] > 256 or case.get("E", 1) == 1:
            case[key] = max(1, case[key] // 2)
        else:
            case["E"] = max(1, case["E"] // 2)
            case["k"] = min(case["k"], case["E"])
    return case


def work(case):
    op = case["op"]
    if op == "quant":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (DTYPES[case["x"]].itemsize + 1) + 4 * case["rows"], "flops": 2 * n}
    T, E, k = case["T"], case.get("E", 1), case.get("k", 1)
    rows = T * k
    if op == "dispatch":   # tokens on one side, grouped rows on the other
        n = case["d"] * DTYPES[case["x"]].itemsize
        return {"bytes": (T + rows) * n + 4 * rows, "flops": rows * case["d"] * case["backward"]}
    if op == "combine":   # grouped rows read, tokens written; backward: both read, grouped rows written
        y, out = case["d"] * DTYPES[case["x"]].itemsize, case["d"] * DTYPES[case["out"]].itemsize
        both = 1 + case["backward"]
        return {"bytes": both * rows * y + T * out + 4 * rows * (1 + both), "flops": both * 2 * rows * case["d"]}
    K, N = (case["d"], 2 * case["F"]) if op == "gate_up" else (case["K"], case["N"])
    gathers = op == "gate_up" or case.get("gather", False)
    active = E * (1 - (1 - k / E) ** T)   # experts that have rows, of even loads
    x = (T if gathers else rows) * (K + 4) + 4 * rows * gathers
    y = rows * (case["F"] if op == "gate_up" else N) * DTYPES[case["out"]].itemsize
    return {"bytes": x + active * N * (K + 4) + y, "flops": 2 * rows * N * K}


# ---- the plain forms

def plain_quant(x):
    """[rows, cols] -> codes, fp32 scales [rows]: s = max|x| / 127, c = the nearest whole number to 127 x / max|x|, ties
    to even (in 64 bits: a value of few bits lies on the border of two codes often)."""
    v = x.double()
    top = v.abs().amax(1, keepdim=True)
    codes = torch.round(127.0 * v / torch.where(top == 0, 1.0, top))
    return codes.to(torch.int8), (top[:, 0] / 127.0).float()


def plain_product(x, x_s, w, w_s):
    """Sums of codes, times both scales."""
    return (x.float() @ w.float().transpose(-1, -2)) * x_s[..., None] * w_s[..., None, :]


def plain_grouped(x, x_s, w, w_s, s):
    """Rows of `x` (in group order) times their expert's `w` [E, N, K]: groups padded to the plan's largest."""
    start, count = s["offsets"][:-1, None], (s["offsets"][1:] - s["offsets"][:-1])[:, None]
    at = torch.arange(s["most"], device=x.device)[None, :]
    inside = at < count
    rows = torch.where(inside, start + at, 0)
    y = plain_product(x[rows] * inside[..., None], x_s[rows], w, w_s)
    return y[s["expert"], s["place"]]


def plain(s):
    op = s["op"]
    if op == "quant":
        return plain_quant(s["x"])
    if op == "gemm":
        return plain_product(s["x_q"], s["x_s"], s["w_q"], s["w_s"]).to(s["out_dtype"])
    if op == "dispatch":
        inv, k = s["inv"].long(), s["k"]
        if s["backward"]:
            return s["x"].float()[inv].view(-1, k, s["x"].shape[1]).sum(1).to(s["x"].dtype)
        out = torch.empty(inv.numel(), s["x"].shape[1], dtype=s["x"].dtype, device=DEV)
        out[inv] = s["x"].repeat_interleave(k, 0)
        return out
    if op == "combine":
        inv, w = s["inv"].long(), s["topk_w"]
        y = s["x"].float()[inv].view(*w.shape, -1)
        if not s["backward"]:
            return (w[..., None] * y).sum(1).to(s["out_dtype"])
        grad = s["grad"].float()[:, None, :]
        dy = torch.empty_like(s["x"])
        dy[inv] = (w[..., None] * grad).view(-1, dy.shape[1]).to(dy.dtype)
        return dy, (grad * y).sum(2)
    x, x_s = s["x_q"], s["x_s"]
    if s["perm_tok"] is not None:
        x, x_s = x[s["perm_tok"]], x_s[s["perm_tok"]]
    if op == "grouped":
        return plain_grouped(x, x_s, s["w_q"], s["w_s"], s).to(s["out_dtype"])
    g = plain_grouped(x, x_s, s["g_q"], s["g_s"], s)
    u = plain_grouped(x, x_s, s["u_q"], s["u_s"], s)
    return (g / (1 + torch.exp(-g)) * u).to(s["out_dtype"])


# ---- inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, sd=1.0):
        return torch.randn(*shape, generator=gen, device=DEV) * sd

    def rows_of(rows, cols, sd=1.0, spread=0.0):
        """Codes and scales of normal values, rows of different sizes."""
        x = normal(rows, cols, sd=sd) * torch.exp(normal(rows, 1, sd=spread))
        top = x.abs().amax(1, keepdim=True)
        return torch.round(x * (127.0 / top)).to(torch.int8), top[:, 0] / 127.0

    op = case["op"]
    s = {"op": op}
    if op == "quant":
        x = normal(case["rows"], case["cols"]) * torch.exp(normal(case["rows"], 1, sd=0.5))
        return s | {"x": x.to(DTYPES[case["x"]])}
    T, E, k = case["T"], case.get("E", 1), case.get("k", 1)
    if op in ("dispatch", "combine"):
        d = case["d"]
        grouped = op == "combine" or case["backward"]   # the operand is expert outputs, or a gradient of expert rows
        s |= {"backward": case["backward"], "k": k, "inv": torch.randperm(T * k, generator=gen, device=DEV).int(),
              "x": normal(T * k if grouped else T, d).to(DTYPES[case["x"]])}
        if op == "combine":
            s |= {"topk_w": torch.softmax(normal(T, k), 1), "out_dtype": DTYPES[case["out"]]}
            if case["backward"]:
                s["grad"] = normal(T, d).to(DTYPES[case["out"]])
        return s
    if op != "gemm":   # skewed loads: k distinct experts per token, grouped stably by expert
        scores = normal(T, E) + normal(E, sd=0.5)
        slots = scores.topk(k, dim=1).indices.reshape(-1)
        order = torch.argsort(slots, stable=True)
        counts = torch.bincount(slots, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
        s["expert"] = slots[order]
        s["place"] = torch.arange(T * k, device=DEV) - s["offsets"][s["expert"]]
        s["most"] = int(counts.max())
        gathers = op == "gate_up" or case["gather"]
        s["perm_tok"] = (order // k).int() if gathers else None
    K = case["d"] if op == "gate_up" else case["K"]
    s["x_q"], s["x_s"] = rows_of(T if op == "gemm" or s["perm_tok"] is not None else T * k, K, spread=0.5)
    s["out_dtype"] = DTYPES[case["out"]]
    for name in ("g", "u") if op == "gate_up" else ("w",):
        N = case["F"] if op == "gate_up" else case["N"]
        q, scale = rows_of(E * N, K, sd=K ** -0.5, spread=0.2)
        s[name + "_q"], s[name + "_s"] = (q, scale) if op == "gemm" else (q.view(E, N, K), scale.view(E, N))
    return s


# ---- one pass

def run(s):
    if not own:
        return plain(s)
    import expert_routed_ffn_selectedsoftmax_gb300 as moe
    op = s["op"]
    if op == "quant":
        return moe.moe_quant_i8(s["x"])
    if op == "dispatch":
        return moe.moe_dispatch_backward(s["x"], s["inv"], s["k"]) if s["backward"] else moe.moe_dispatch(s["x"], s["inv"], s["k"])
    if op == "combine":
        if s["backward"]:
            return moe.moe_combine_backward(s["grad"], s["x"], s["topk_w"], s["inv"])
        return moe.moe_combine(s["x"], s["topk_w"], s["inv"], out_dtype=s["out_dtype"])
    if op == "gemm":
        return moe.moe_gemm_i8(s["x_q"], s["x_s"], s["w_q"], s["w_s"], out_dtype=s["out_dtype"])
    if op == "grouped":
        return moe.moe_grouped_gemm_i8(s["x_q"], s["x_s"], s["w_q"], s["w_s"], s["offsets"], perm_tok=s["perm_tok"], out_dtype=s["out_dtype"])
    return moe.moe_gate_up_i8(s["x_q"], s["x_s"], s["g_q"], s["g_s"], s["u_q"], s["u_s"], offsets=s["offsets"], perm_tok=s["perm_tok"],
                              h_dtype=s["out_dtype"])


# ---- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "quant":
        codes, scales = [], []
        for x in s["x"].split(1024):
            v = x.double()
            top = torch.maximum(v.amax(1), -v.amin(1))
            scales.append(top / 127)
            each = 127 * v / top.clamp(min=1e-300)[:, None]
            low = each.floor()
            up = (each - low > 0.5) | ((each - low == 0.5) & (low % 2 != 0))
            codes.append((low + up).to(torch.int8))
        return torch.cat(codes), torch.cat(scales)
    if op in ("dispatch", "combine"):
        k, rows = s["k"], s["x"].double()
        T = s["inv"].numel() // k
        slot = [s["inv"].view(T, k)[:, j].long() for j in range(k)]
        if op == "combine" and s["backward"]:
            dy, dw = torch.zeros_like(rows), []
            grad = s["grad"].double()
            for j in range(k):
                dy.index_copy_(0, slot[j], grad * s["topk_w"][:, j:j + 1].double())
                dw.append(torch.einsum("td,td->t", grad, rows.index_select(0, slot[j])))
            return dy, torch.stack(dw, 1)
        if op == "dispatch" and not s["backward"]:
            out = rows.new_zeros(T * k, rows.shape[1])
            for j in range(k):
                out.index_copy_(0, slot[j], rows)
            return out
        out = rows.new_zeros(T, rows.shape[1])
        for j in range(k):
            each = rows.index_select(0, slot[j])
            out += each * s["topk_w"][:, j:j + 1].double() if op == "combine" else each
        return out

    def values(name, e=None):
        q, scale = s[name + "_q"], s[name + "_s"]
        if e is not None:
            q, scale = q[e], scale[e]
        return q.double() * scale.double()[:, None]

    x = values("x")
    if op == "gemm":
        return x @ values("w").T
    off = s["offsets"].tolist()
    parts = []
    for e in range(len(off) - 1):
        rows = torch.arange(off[e], off[e + 1], device=DEV)
        xe = x[rows if s["perm_tok"] is None else s["perm_tok"][rows].long()]
        if op == "grouped":
            parts.append(xe @ values("w", e).T)
        else:
            g, u = xe @ values("g", e).T, xe @ values("u", e).T
            parts.append(g * torch.sigmoid(g) * u)
    return torch.cat(parts)
