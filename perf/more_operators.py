"""The cases on which the operators of experts that a caller trains, and of 8-bit dense products, are measured: the
products grouped by expert with their gradients, the gated activation between them with its gradient, and the product
of e4m3 operands with one fp32 scale for each block of 128, with its quantizers.

`run` computes an operator in plain torch operations (32 bits, one rounding at the end) where `own` is false, and by
the library's calls where it is true, on what `prepare` made. e4m3 codes are returned in torch's type of that name."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK, TOP, LEAST = 128, 448.0, 2.0 ** -100   # a block's side, e4m3's largest value, the least maximum a scale is made for


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode batch's activations on their way into a dense product
        {"name": "quant_b8", "op": "quant", "what": "rows", "T": 8, "H": 4096, "skip": 0},
        # a prefill chunk's activations
        {"name": "quant_prefill", "op": "quant", "what": "rows", "T": 4096, "H": 4096, "skip": 0},
        # a weight after an optimizer step, for the product and, transposed, for its input's gradient
        {"name": "quant_weight", "op": "quant", "what": "weight", "T": 4096, "H": 4096, "skip": 0},
        # one token through a dense projection
        {"name": "fp8_one", "op": "fp8", "T": 1, "N": 4096, "K": 4096},
        # a ragged chunk whose sizes fill no tile, K ending inside a block
        {"name": "fp8_ragged", "op": "fp8", "T": 517, "N": 2085, "K": 4112},
        # a dense projection over a prefill chunk
        {"name": "fp8_prefill", "op": "fp8", "T": 4096, "N": 4096, "K": 4096},
        # the decode batch's rows through the gate and up projections of their experts
        {"name": "grouped_b8", "op": "grouped", "way": "forward", "T": 8, "E": 64, "top": 8, "N": 1536, "D": 2048, "tile": 16,
         "out": "bf16", "zipf": False, "pad": False},
        # a training chunk through the down projections
        {"name": "grouped_chunk", "op": "grouped", "way": "forward", "T": 4096, "E": 128, "top": 8, "N": 4096, "D": 1536, "tile": 128,
         "out": "bf16", "zipf": False, "pad": False},
        # the gradient of those projections' input for a ragged batch under skewed routing
        {"name": "grouped_input_grad_zipf", "op": "grouped", "way": "input", "T": 517, "E": 128, "top": 8, "N": 4096, "D": 1536,
         "tile": 16, "out": "bf16", "zipf": True, "pad": False},
        # the gradient of those projections over the chunk, in the optimizer's type
        {"name": "grouped_weight_grad_chunk", "op": "grouped", "way": "weight", "T": 4096, "E": 128, "top": 8, "N": 4096, "D": 1536,
         "tile": 128, "out": "f32", "zipf": False, "pad": False},
        # the activation of 64 tokens' rows
        {"name": "swiglu_b64", "op": "swiglu", "way": "forward", "T": 64, "E": 128, "top": 8, "I": 1536, "tile": 16, "dtype": "bf16",
         "zipf": True, "pad": False},
        # its gradient over the chunk
        {"name": "swiglu_grad_chunk", "op": "swiglu", "way": "backward", "T": 4096, "E": 128, "top": 8, "I": 1536, "tile": 128,
         "dtype": "bf16", "zipf": False, "pad": False},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["quant", "fp8", "fp8", "grouped", "grouped", "grouped", "swiglu"])
    T = _log(rng, 1, 4096)
    if op == "quant":
        return {"op": op, "what": rng.choice(["rows", "rows", "weight"]), "T": T, "H": 16 * _log(rng, 1, 256), "skip": rng.choice([0, 8, 64])}
    if op == "fp8":
        return {"op": op, "T": T, "N": _log(rng, 1, 4096), "K": 16 * _log(rng, 1, 256)}
    case = {"op": op, "T": T, "E": rng.choice([8, 64, 128]), "top": rng.randint(1, 8), "tile": rng.choice([16, 32, 64, 128]),
            "zipf": rng.random() < 0.4, "pad": rng.random() < 0.3}
    if op == "swiglu":
        return {**case, "way": rng.choice(["forward", "backward"]), "I": 8 * _log(rng, 4, 192), "dtype": rng.choice(["bf16", "bf16", "f32"])}
    return {**case, "way": rng.choice(["forward", "input", "weight"]), "N": 8 * _log(rng, 4, 512), "D": 8 * _log(rng, 4, 192),
            "out": rng.choice(["bf16", "f32"])}


def _rows_max(T, K, E, tile):
    routes = T * K
    filled = min(routes, E)
    return (filled + (routes - filled) // tile) * tile


def _served(c):
    return c["T"] * c["top"] * (0.8 if c["pad"] else 1.0)


def _experts_hit(c):
    """About how many experts hold a row."""
    share = [(e + 1) ** -1.1 if c["zipf"] else 1.0 for e in range(c["E"])]
    total = sum(share)
    return sum(1.0 - (1.0 - min(1.0, p / total)) ** _served(c) for p in share)


def work(case):
    c = case
    if c["op"] == "quant":
        n, blocks = c["T"] * c["H"], -(-c["H"] // BLOCK)
        if c["what"] == "rows":
            return {"bytes": 3 * n + 4 * c["T"] * blocks, "flops": 3 * n}
        return {"bytes": 4 * n + 8 * -(-c["T"] // BLOCK) * blocks, "flops": 3 * n}
    if c["op"] == "fp8":
        T, N, K = c["T"], c["N"], c["K"]
        blocks = -(-K // BLOCK)
        return {"bytes": T * K + N * K + 4 * blocks * (T + -(-N // BLOCK)) + 2 * T * N, "flops": 2 * T * N * K}
    rows = _served(c)
    if c["op"] == "swiglu":
        size = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": rows * c["I"] * size * (3 if c["way"] == "forward" else 5), "flops": rows * c["I"] * (5 if c["way"] == "forward" else 12)}
    size = 2 if c["out"] == "bf16" else 4
    ins, outs = {"forward": (c["D"], c["N"]), "input": (c["N"], c["D"]), "weight": (c["N"] + c["D"], 0)}[c["way"]]
    weights = c["E"] * size if c["way"] == "weight" else _experts_hit(c) * 2
    return {"bytes": rows * (2 * ins + size * outs) + weights * c["N"] * c["D"], "flops": 2 * rows * c["N"] * c["D"]}


# ------------------------------------------------------------------ inputs
def _routing(c, g, dev):
    """The maps of a top-k routing, experts' rows padded to whole tiles: first row of each expert (and the end), its
    rows, the token of each row, the rows in all, and the same as a list of (expert, first, rows, end)."""
    T, E, K = c["T"], c["E"], c["top"]
    score = torch.randn(T, E, generator=g, device=dev)
    if c["zipf"]:
        score = score - 1.1 * torch.log(1.0 + torch.randperm(E, generator=g, device=dev).float())
    expert = score.topk(K, dim=1).indices
    if c["pad"]:
        expert = torch.where((torch.rand(T, generator=g, device=dev) >= 0.2)[:, None], expert, E)
    expert = expert.reshape(-1)
    count = torch.bincount(expert, minlength=E + 1)[:E]
    end = torch.cumsum((count + c["tile"] - 1) // c["tile"] * c["tile"], 0)
    start = torch.cat((end.new_zeros(1), end))
    order = torch.argsort(expert, stable=True)
    held = order[: int(count.sum())]
    rank = torch.arange(held.numel(), device=dev) - (torch.cumsum(count, 0) - count)[expert[held]]
    perm2tok = torch.full((_rows_max(T, K, E, c["tile"]),), -1, dtype=torch.int32, device=dev)
    perm2tok[start[expert[held]] + rank] = (held // K).to(torch.int32)
    first, rows = start.tolist(), count.tolist()
    groups = [(e, first[e], rows[e], first[e + 1]) for e in range(E)]
    return start.to(torch.int32), count.to(torch.int32), perm2tok, end[-1:].to(torch.int32), groups


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*dims):
        return torch.randn(*dims, generator=g, device=dev)

    def activations(rows, cols):  # one in a hundred is an outlier
        x = normal(rows, cols)
        return torch.where(torch.rand(rows, cols, generator=g, device=dev) < 0.01, 20 * x, x)

    s = {"case": dict(c)}
    if c["op"] == "quant":
        T, H = c["T"], c["H"]
        blocks = -(-H // BLOCK)
        s["codes"] = torch.empty(T, H, dtype=torch.uint8, device=dev)
        if c["what"] == "rows":
            s["x"] = activations(T, H + c["skip"]).to(torch.bfloat16)[:, :H]
            s["sf"] = torch.empty(blocks, T, dtype=torch.float32, device=dev)
        else:
            s["x"] = (normal(T, H + c["skip"]) / math.sqrt(H)).to(torch.bfloat16)[:, :H]
            s["sf"] = torch.empty(-(-T // BLOCK), blocks, dtype=torch.float32, device=dev)
            wide = (T + 15) // 16 * 16      # rows of the transposed codes start at multiples of 16 bytes
            s["codes_t"] = torch.zeros(H, wide, dtype=torch.uint8, device=dev)[:, :T]
            s["sf_t"] = torch.empty(blocks, -(-T // BLOCK), dtype=torch.float32, device=dev)
        return s
    if c["op"] == "fp8":
        T, N, K = c["T"], c["N"], c["K"]
        q, s["a_sf"] = _quant_rows(activations(T, K).to(torch.bfloat16).float())
        s["a_codes"] = q.to(torch.float8_e4m3fn).view(torch.uint8)
        q, s["w_sf"] = _quant_blocks((normal(N, K) / math.sqrt(K)).to(torch.bfloat16).float())
        s["w_codes"] = q.to(torch.float8_e4m3fn).view(torch.uint8)
        s["out"] = torch.empty(T, N, dtype=torch.bfloat16, device=dev)
        return s
    s["offsets"], s["counts"], s["perm2tok"], s["total"], s["groups"] = _routing(c, g, dev)
    R = s["perm2tok"].numel()
    held = (s["perm2tok"] >= 0)[:, None]

    def rows(cols, dt, scale=1.0):  # padding rows are zeros, as the sort of the tokens leaves them
        return torch.where(held, scale * normal(R, cols), 0.0).to(dt)

    if c["op"] == "swiglu":
        dt = DTYPES[c["dtype"]]
        s["gate_up"] = rows(2 * c["I"], dt, 2.0)
        s["d_inter"] = rows(c["I"], dt) if c["way"] == "backward" else None
        s["out"] = torch.zeros(R, c["I"] * (1 if c["way"] == "forward" else 2), dtype=dt, device=dev)
        return s
    N, D, dt = c["N"], c["D"], DTYPES[c["out"]]
    if c["way"] != "weight":
        s["w"] = torch.empty(c["E"], N, D, dtype=torch.bfloat16, device=dev)
        for e in range(c["E"]):
            s["w"][e] = (normal(N, D) / math.sqrt(D)).to(torch.bfloat16)
    s["x"] = rows(D, torch.bfloat16) if c["way"] != "input" else None
    s["d_out"] = rows(N, torch.bfloat16) if c["way"] != "forward" else None
    dims = {"forward": (R, N), "input": (R, D), "weight": (c["E"], N, D)}[c["way"]]
    s["out"] = torch.zeros(*dims, dtype=dt, device=dev)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from nvfp4_block_scaled_route_amd import native as N

    c = s["case"]
    if c["op"] == "quant":
        if c["what"] == "rows":
            N.fp8_quant(s["x"], s["codes"], s["sf"])
            return s["codes"].view(torch.float8_e4m3fn), s["sf"]
        N.fp8_quant_weight(s["x"], s["codes"], s["sf"], s["codes_t"], s["sf_t"])
        return s["codes"].view(torch.float8_e4m3fn), s["sf"], s["codes_t"].view(torch.float8_e4m3fn), s["sf_t"]
    if c["op"] == "fp8":
        N.fp8_gemm(s["a_codes"], s["a_sf"], s["w_codes"], s["w_sf"], s["out"])
    elif c["op"] == "swiglu":
        if c["way"] == "forward":
            N.moe_swiglu(s["gate_up"], s["perm2tok"], s["total"], s["out"])
        else:
            N.moe_swiglu_bwd(s["d_inter"], s["gate_up"], s["perm2tok"], s["total"], s["out"])
    elif c["way"] == "forward":
        N.moe_grouped_gemm(s["x"], s["w"], s["offsets"], s["counts"], s["out"])
    elif c["way"] == "input":
        N.moe_grouped_gemm_dgrad(s["d_out"], s["w"], s["offsets"], s["counts"], s["out"])
    else:
        N.moe_grouped_gemm_wgrad(s["d_out"], s["x"], s["offsets"], s["counts"], s["out"])
    return s["out"]


def _blocks(x, rows):
    """x [T, H] -> [T / rows, rows, H / 128, 128], zeros behind its edges."""
    T, H = x.shape
    up, across = -(-T // rows), -(-H // BLOCK)
    return torch.nn.functional.pad(x, (0, across * BLOCK - H, 0, up * rows - T)).reshape(up, rows, across, BLOCK)


def _quant(x, rows):
    """fp32 values to e4m3 under a scale for each `rows` x 128: the elements' values before scaling, the scales."""
    b = _blocks(x, rows)
    top = b.abs().amax((1, 3)).clamp(min=LEAST)
    q = b * 0.875 / (top * 2.0 ** -9)[:, None, :, None]     # 448 b / top, the division's rounding alone
    q = q.clamp(-TOP, TOP).to(torch.float8_e4m3fn).float()
    return q.reshape(q.shape[0] * rows, -1)[: x.shape[0], : x.shape[1]], top / TOP


def _quant_rows(x):
    q, sf = _quant(x, 1)
    return q, sf.t().contiguous()


def _quant_blocks(x):
    return _quant(x, BLOCK)


def _silu(g):
    return g / (1.0 + torch.exp(-g))


def _run_plain(s):
    c = s["case"]
    if c["op"] == "quant":
        if c["what"] == "rows":
            q, sf = _quant_rows(s["x"].float())
            return q.to(torch.float8_e4m3fn), sf
        q, sf = _quant_blocks(s["x"].float())
        codes = q.to(torch.float8_e4m3fn)
        return codes, sf, codes.t(), sf.t().contiguous()
    if c["op"] == "fp8":
        T, N, K = c["T"], c["N"], c["K"]
        a = s["a_codes"].view(torch.float8_e4m3fn).float() * s["a_sf"].t().repeat_interleave(BLOCK, dim=1)[:, :K]
        w = s["w_sf"].repeat_interleave(BLOCK, dim=0)[:N].repeat_interleave(BLOCK, dim=1)[:, :K]
        w = s["w_codes"].view(torch.float8_e4m3fn).float() * w
        return (a @ w.t()).to(torch.bfloat16)
    if c["op"] == "swiglu":
        gate, up = s["gate_up"].float().chunk(2, dim=1)
        if c["way"] == "forward":
            y = _silu(gate) * up
        else:
            d, sig = s["d_inter"].float(), 1.0 / (1.0 + torch.exp(-gate))
            y = torch.cat((d * up * sig * (1.0 + gate * (1.0 - sig)), d * _silu(gate)), dim=1)
        y = torch.where((s["perm2tok"] >= 0)[:, None], y, 0.0)
        live = torch.arange(y.shape[0], device=y.device) < s["total"]
        return torch.where(live[:, None], y, s["out"].float()).to(s["out"].dtype)
    out = s["out"].clone()      # rows behind the last tile stay
    for e, first, rows, end in s["groups"]:
        if c["way"] == "weight":
            out[e] = (s["d_out"][first : first + rows].float().t() @ s["x"][first : first + rows].float()).to(out.dtype)
            continue
        out[first + rows : end] = 0.0
        if rows:
            w = s["w"][e].float()
            y = s["x"][first : first + rows].float() @ w.t() if c["way"] == "forward" else s["d_out"][first : first + rows].float() @ w
            out[first : first + rows] = y.to(out.dtype)
    return out


# ------------------------------------------------------------------ in 64 bits
def _nearest_e4m3(v):
    """float64 values to e4m3 by a search of its whole grid, ties to the even code."""
    code = torch.arange(127, device=v.device)
    ex, man = (code >> 3).double(), (code & 7).double()
    grid = torch.where(ex == 0, man * 2.0 ** -9, torch.ldexp(1 + man / 8, ex - 7))
    m = v.abs()
    up = torch.searchsorted(grid, m.contiguous()).clamp(max=126)
    down = (up - 1).clamp(min=0)
    below, above = m - grid[down], grid[up] - m
    pick = torch.where((below < above) | ((below == above) & (down % 2 == 0)), down, up)
    return torch.copysign(grid[pick], v)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "quant":
        x, T, H = s["x"].double(), c["T"], c["H"]
        tall = 1 if c["what"] == "rows" else BLOCK
        top = torch.stack([x[:, k : k + BLOCK].abs().amax(1) for k in range(0, H, BLOCK)], dim=1)
        if tall > 1:
            top = torch.stack([top[t : t + BLOCK].amax(0) for t in range(0, T, BLOCK)])
        top = top.clamp(min=LEAST)
        sf = top / 448.0
        row, col = torch.arange(T, device=x.device) // tall, torch.arange(H, device=x.device) // BLOCK
        q = _nearest_e4m3(x * 448.0 / top[row][:, col])
        return (q, sf.t().contiguous()) if tall == 1 else (q, sf, q.t().contiguous(), sf.t().contiguous())
    if c["op"] == "fp8":
        out = torch.zeros(c["T"], c["N"], dtype=torch.float64, device="cuda")
        a, w = (s[n].view(torch.float8_e4m3fn).double() for n in ("a_codes", "w_codes"))
        of_row = torch.arange(c["N"], device="cuda") // BLOCK
        for b in range(-(-c["K"] // BLOCK)):
            k = slice(b * BLOCK, min((b + 1) * BLOCK, c["K"]))
            out += torch.mm(a[:, k].contiguous(), w[:, k].t().contiguous()) * s["a_sf"][b].double()[:, None] * s["w_sf"][:, b].double()[of_row][None]
        return out
    if c["op"] == "swiglu":
        out, total, I = s["out"].double(), int(s["total"]), c["I"]
        held = torch.nonzero(s["perm2tok"] >= 0).reshape(-1)
        out[:total] = 0.0
        gate, up = s["gate_up"][held, :I].double(), s["gate_up"][held, I:].double()
        sig = torch.sigmoid(gate)
        if c["way"] == "forward":
            out[held] = gate * sig * up
        else:
            d = s["d_inter"][held].double()
            out[held, :I] = d * up * (sig + gate * sig * (1.0 - sig))
            out[held, I:] = d * gate * sig
        return out
    out = s["out"].double()
    if c["way"] != "weight":
        out[: int(s["total"])] = 0.0
    for e in range(c["E"]):
        rows = slice(int(s["offsets"][e]), int(s["offsets"][e]) + int(s["counts"][e]))
        if c["way"] == "forward":
            out[rows] = torch.mm(s["x"][rows].double(), s["w"][e].double().t().contiguous())
        elif c["way"] == "input":
            out[rows] = torch.mm(s["d_out"][rows].double(), s["w"][e].double())
        else:
            out[e] = torch.mm(s["d_out"][rows].double().t().contiguous(), s["x"][rows].double())
    return out
