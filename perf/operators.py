"""Cases of the block-scaled fp8 operators: quantisation, residual + RMS norm, dense and grouped products, SwiGLU product.

`run` computes an operator in its plain form (elementary torch operations in 32 bits), or, where `own` is set, by the
library's call.  Codes are OCP E4M3 (torch.float8_e4m3fn); activations carry one fp32 scale per row and 128 columns,
weights one per 128 x 128 block; a value is code * scale.
"""
import math

import torch

own = False
DEV = "cuda"
B = 128            # columns (and weight rows) that share a scale
FP8_MAX = 448.0    # largest finite E4M3 value
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
MOST_FLOPS, MOST_BYTES = 1.9e11, 4.2e8   # a drawn case's work stays below the largest listed one's


def listed():
    return [
        # residual + norm of one token of a decode step (latency), fp32 residual stream
        {"name": "norm_one_token", "op": "norm", "T": 1, "d": 2048, "k": 0, "x": "f32", "delta": "bf16", "normed": True},
        # a prefill's rows: combine of two expert rows per token, residual, norm
        {"name": "norm_combine_prefill", "op": "norm", "T": 8192, "d": 1024, "k": 2, "x": "f32", "delta": "bf16", "normed": True},
        # an odd batch, width that is no multiple of the block, bf16 residual stream, codes only
        {"name": "norm_odd_width", "op": "norm", "T": 999, "d": 2000, "k": 0, "x": "bf16", "delta": "bf16", "normed": False},
        # activations that no norm precedes, a small odd batch
        {"name": "quant_rows", "op": "quant", "E": 1, "rows": 37, "cols": 2816, "block_rows": 1, "x": "bf16"},
        # a checkpoint's expert weights, 128 x 128 blocks
        {"name": "quant_experts", "op": "quant", "E": 16, "rows": 2816, "cols": 2048, "block_rows": 128, "x": "bf16"},
        # dense projection of one token: the weights are streamed
        {"name": "gemm_one_token", "op": "gemm", "T": 1, "K": 2048, "N": 5632, "out": "bf16"},
        # the same projection over a prefill: bound by the tensor cores
        {"name": "gemm_prefill", "op": "gemm", "T": 8192, "K": 2048, "N": 5632, "out": "bf16"},
        # down projection of a decode batch over 16 experts, ragged groups of about 4 rows
        {"name": "grouped_decode", "op": "grouped", "T": 64, "E": 16, "k": 1, "K": 2816, "N": 2048, "out": "f32", "gather": False},
        # down projection of a prefill over 64 experts, top-2
        {"name": "grouped_prefill", "op": "grouped", "T": 8192, "E": 64, "k": 2, "K": 512, "N": 1024, "out": "bf16", "gather": False},
        # gate/up + SwiGLU of one token, two of 64 experts
        {"name": "gate_up_one_token", "op": "gate_up", "T": 1, "E": 64, "k": 2, "d": 1024, "F": 512},
        # gate/up + SwiGLU of a decode batch (64 streams x a pair): every expert's weights for 4 rows each
        {"name": "gate_up_decode", "op": "gate_up", "T": 128, "E": 64, "k": 2, "d": 1024, "F": 512},
        # gate/up + SwiGLU of a prefill over 16 wide experts, top-1
        {"name": "gate_up_prefill", "op": "gate_up", "T": 4096, "E": 16, "k": 1, "d": 2048, "F": 2816},
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi):   # multiples of 16 (rows of codes are read in 16-byte pieces)
        return 16 * log_int(lo / 16, hi / 16)

    op = rng.choice(["norm", "quant", "gemm", "grouped", "gate_up"])
    if op == "norm":
        case = {"op": op, "T": log_int(1, 8192), "d": width(128, 8192), "k": rng.choice([0, 0, 1, 2, 4, 8]),
                "x": rng.choice(["f32", "bf16"]), "delta": rng.choice(["f32", "bf16"]), "normed": rng.random() < 0.7}
    elif op == "quant":
        case = {"op": op, "E": log_int(1, 16), "rows": log_int(1, 8192), "cols": width(128, 8192),
                "block_rows": rng.choice([1, 128]), "x": rng.choice(["f32", "bf16"])}
    elif op == "gemm":
        case = {"op": op, "T": log_int(1, 8192), "K": width(128, 8192), "N": log_int(128, 8192), "out": rng.choice(["f32", "bf16"])}
    else:
        E = log_int(1, 128)
        case = {"op": op, "T": log_int(1, 8192), "E": E, "k": rng.randint(1, min(E, 8))}
        if op == "grouped":
            case |= {"K": width(128, 4096), "N": log_int(128, 4096), "out": rng.choice(["f32", "bf16"]), "gather": rng.random() < 0.5}
        else:
            case |= {"d": width(128, 4096), "F": width(128, 4096)}
    key = "rows" if op == "quant" else "T"
    while work(case)["flops"] > MOST_FLOPS or work(case)["bytes"] > MOST_BYTES:   # few rows first, then fewer experts
        if case[key] > 256 or case.get("E", 1) == 1:
            case[key] = max(1, case[key] // 2)
        else:
            case["E"] = max(1, case["E"] // 2)
            case["k"] = min(case.get("k", 1), case["E"])
            if op == "quant":
                del case["k"]
    return case


def blocks(n):
    return -(-n // B)


def work(case):
    op = case["op"]
    if op == "quant":
        n = case["E"] * case["rows"] * case["cols"]
        scales = case["E"] * -(-case["rows"] // case["block_rows"]) * blocks(case["cols"])
        return {"bytes": n * (DTYPES[case["x"]].itemsize + 1) + 4 * scales, "flops": 2 * n}
    if op == "norm":
        n, k = case["T"] * case["d"], case["k"]
        size = 2 * DTYPES[case["x"]].itemsize + max(k, 1) * DTYPES[case["delta"]].itemsize + 2 * case["normed"] + 1
        return {"bytes": n * size + 4 * case["T"] * (blocks(case["d"]) + 2 * k) + 4 * case["d"], "flops": n * (6 + 2 * k)}
    T, E, k = case["T"], case.get("E", 1), case.get("k", 1)
    rows = T * k
    K, N = (case["d"], 2 * case["F"]) if op == "gate_up" else (case["K"], case["N"])
    gathers = op == "gate_up" or case.get("gather", False)
    active = E * (1 - (1 - k / E) ** T)   # experts that have rows, of even loads
    x = (T if gathers else rows) * (K + 4 * blocks(K)) + 4 * rows * gathers
    y = rows * (case["F"] + 4 * blocks(case["F"])) if op == "gate_up" else rows * N * DTYPES[case["out"]].itemsize
    return {"bytes": x + active * (N * K + 4 * blocks(N) * blocks(K)) + y, "flops": 2 * rows * N * K}


# ---- the plain forms

def plain_quant(x, block_rows):
    """[..., rows, cols] -> E4M3 codes, fp32 scales [..., rows / block_rows, cols / 128]: s = max|x| / 448, c = e4m3(x / s)."""
    rows, cols = x.shape[-2:]
    nr, nc = -(-rows // block_rows), blocks(cols)
    padded = x.new_zeros(*x.shape[:-2], nr * block_rows, nc * B, dtype=torch.float32)
    padded[..., :rows, :cols] = x
    tiles = padded.view(*x.shape[:-2], nr, block_rows, nc, B)
    scale = tiles.abs().amax(dim=(-3, -1)) / FP8_MAX
    codes = tiles / torch.where(scale == 0, 1.0, scale)[..., :, None, :, None]
    codes = codes.clamp(-FP8_MAX, FP8_MAX).view(padded.shape)[..., :rows, :cols]
    return codes.to(torch.float8_e4m3fn).contiguous(), scale


def values(codes, scales, block_rows):
    """code * scale in 32 bits."""
    rows, cols = codes.shape[-2:]
    r = torch.arange(rows, device=codes.device) // block_rows
    c = torch.arange(cols, device=codes.device) // B
    return codes.float() * scales[..., r, :][..., c]


def plain_grouped(x, w, s):
    """Rows of `x` (in group order) times their expert's `w` [E, N, K]: groups padded to the plan's largest."""
    start, count = s["offsets"][:-1, None], (s["offsets"][1:] - s["offsets"][:-1])[:, None]
    at = torch.arange(s["most"], device=x.device)[None, :]
    inside = at < count
    rows = torch.where(inside, start + at, 0)
    y = torch.bmm(x[rows] * inside[..., None], w.transpose(1, 2))
    return y[s["expert"], s["place"]]


def plain(s):
    op = s["op"]
    if op == "quant":
        return plain_quant(s["x"], s["block_rows"])
    if op == "norm":
        r = s["x"].float()
        if s["k"]:
            r = r + (s["topk_w"][..., None] * s["delta"].float()[s["inv"]].view(*s["topk_w"].shape, -1)).sum(1)
        else:
            r = r + s["delta"].float()
        y = r * torch.rsqrt(r.square().mean(1, keepdim=True) + s["eps"]) * s["weight"].float()
        out = (r.to(s["x"].dtype),) + ((y.bfloat16(),) if s["want_normed"] else ())
        return out + plain_quant(y, 1)
    x = values(s["x_q"], s["x_s"], 1)
    if op == "gemm":
        return (x @ values(s["w_q"], s["w_s"], B).T).to(s["out_dtype"])
    if s["perm_tok"] is not None:
        x = x[s["perm_tok"]]
    if op == "grouped":
        return plain_grouped(x, values(s["w_q"], s["w_s"], B), s).to(s["out_dtype"])
    g = plain_grouped(x, values(s["g_q"], s["g_s"], B), s)
    u = plain_grouped(x, values(s["u_q"], s["u_s"], B), s)
    return plain_quant(g / (1 + torch.exp(-g)) * u, 1)


# ---- inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, sd=1.0):
        return torch.randn(*shape, generator=gen, device=DEV) * sd

    op = case["op"]
    s = {"op": op}
    if op == "quant":
        x = normal(case["E"], case["rows"], case["cols"]) * torch.exp(normal(case["E"], case["rows"], 1, sd=0.5))
        return s | {"x": x.to(DTYPES[case["x"]]), "block_rows": case["block_rows"]}
    T, E, k = case["T"], case.get("E", 1), case.get("k", 1)
    if op == "norm":
        d = case["d"]
        s |= {"x": normal(T, d, sd=2.0).to(DTYPES[case["x"]]), "weight": 1 + normal(d, sd=0.1), "eps": 1e-6, "k": k,
              "want_normed": case["normed"], "delta": normal(T * max(k, 1), d).to(DTYPES[case["delta"]])}
        if k:   # routing weights and the grouped row of each (token, slot)
            s["topk_w"] = torch.softmax(normal(T, k), 1)
            s["inv"] = torch.randperm(T * k, generator=gen, device=DEV).int()
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
    rows = T if op == "gemm" or s["perm_tok"] is not None else T * k
    s["x_q"], s["x_s"] = plain_quant(normal(rows, K) * torch.exp(normal(rows, 1, sd=0.5)), 1)
    if op == "gate_up":
        s["g_q"], s["g_s"] = plain_quant(normal(E, case["F"], K, sd=K ** -0.5), B)
        s["u_q"], s["u_s"] = plain_quant(normal(E, case["F"], K, sd=K ** -0.5), B)
        return s
    shape = (case["N"], K) if op == "gemm" else (E, case["N"], K)
    s["w_q"], s["w_s"] = plain_quant(normal(*shape, sd=K ** -0.5), B)
    s["out_dtype"] = DTYPES[case["out"]]
    return s


# ---- one pass

def run(s):
    if not own:
        return plain(s)
    import expert_routed_ffn_selectedsoftmax_gb300 as moe
    op = s["op"]
    if op == "quant":
        return moe.moe_quant_fp8b(s["x"], block_rows=s["block_rows"])
    if op == "norm":
        combine = {"topk_w": s["topk_w"], "inv": s["inv"]} if s["k"] else {}
        out = moe.moe_norm_fp8b(s["x"], s["weight"], s["eps"], delta=s["delta"], want_normed=s["want_normed"], **combine)
        return out if s["want_normed"] else (out[0], out[2], out[3])
    if op == "gemm":
        return moe.moe_gemm_fp8b(s["x_q"], s["x_s"], s["w_q"], s["w_s"], out_dtype=s["out_dtype"])
    if op == "grouped":
        return moe.moe_grouped_gemm_fp8b(s["x_q"], s["x_s"], s["w_q"], s["w_s"], s["offsets"], perm_tok=s["perm_tok"], out_dtype=s["out_dtype"])
    return moe.moe_gate_up_fp8b(s["x_q"], s["x_s"], s["g_q"], s["g_s"], s["u_q"], s["u_s"], offsets=s["offsets"], perm_tok=s["perm_tok"])


# ---- the definitions in 64 bits

def exact_e4m3(v):
    """The nearest E4M3 value (ties to the even code): steps of 2^(e-3) in [2^e, 2^(e+1)), e >= -6."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -30))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-FP8_MAX, FP8_MAX)


def exact_quant(x, block_rows):
    rows, cols = x.shape
    codes, scales = torch.empty_like(x), x.new_empty(-(-rows // block_rows), blocks(cols))
    for j in range(blocks(cols)):
        col = x[:, j * B:(j + 1) * B]
        top = col.abs().amax(1)
        top = torch.nn.functional.pad(top, (0, scales.shape[0] * block_rows - rows)).view(-1, block_rows).amax(1)
        scales[:, j] = top / FP8_MAX
        each = scales[:, j].repeat_interleave(block_rows)[:rows, None]
        codes[:, j * B:(j + 1) * B] = exact_e4m3(torch.where(each > 0, col / each.clamp(min=1e-300), 0.0))
    return codes, scales


def exact_values(codes, scales, block_rows):
    v = codes.double()
    spread = scales.double().repeat_interleave(block_rows, 0)[:v.shape[0]].repeat_interleave(B, 1)[:, :v.shape[1]]
    return v * spread


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "quant":
        parts = [exact_quant(x.double(), s["block_rows"]) for x in s["x"]]
        return torch.stack([c for c, _ in parts]), torch.stack([t for _, t in parts])
    if op == "norm":
        r = s["x"].double()
        for j in range(max(s["k"], 1)):
            at = s["inv"].view(-1, s["k"])[:, j].long() if s["k"] else slice(None)
            r = r + s["delta"].double()[at] * (s["topk_w"][:, j:j + 1].double() if s["k"] else 1.0)
        y = r / torch.sqrt((r * r).sum(1, keepdim=True) / r.shape[1] + s["eps"]) * s["weight"].double()
        return ((r, y) if s["want_normed"] else (r,)) + exact_quant(y, 1)
    x = exact_values(s["x_q"], s["x_s"], 1)
    if op == "gemm":
        return x @ exact_values(s["w_q"], s["w_s"], B).T
    off = s["offsets"].tolist()
    parts = []
    for e in range(len(off) - 1):
        rows = torch.arange(off[e], off[e + 1], device=DEV)
        xe = x[rows if s["perm_tok"] is None else s["perm_tok"][rows].long()]
        if op == "grouped":
            parts.append(xe @ exact_values(s["w_q"][e], s["w_s"][e], B).T)
        else:
            g, u = (xe @ exact_values(s[n + "_q"][e], s[n + "_s"][e], B).T for n in "gu")
            parts.append(g * torch.sigmoid(g) * u)
    y = torch.cat(parts)
    return exact_quant(y, 1) if op == "gate_up" else y
