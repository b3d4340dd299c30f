"""Cases, plain forms and 64-bit values of the grouped products by expert and of the microscaled 4-bit floating point
format (MXFP4) that feeds them.

Each case names an operator by its "op":
  mx_round_trip   rows to MXFP4 and back to the values that the codes stand for
  mx_gemm         MXFP4 rows, grouped by expert, times the experts' MXFP4 matrices; with SwiGLU: the gate and up products
  gemm            the same with 16-bit rows and matrices
  gemm_dx         its gradient by the rows
  gemm_dw         its gradient by the matrices

Where `own` is false, run() computes them in elementary torch operations, where it is true with the library's kernels."""
import math

import torch

own = False

_BF16, _F16, _F32 = "bf16", "f16", "f32"
_TORCH = {_BF16: torch.bfloat16, _F16: torch.float16, _F32: torch.float32}
_SIZE = {_BF16: 2, _F16: 2, _F32: 4}


# ---- cases ----------------------------------------------------------------------------------------------------------

def listed():
    """The layer's own shapes: 256 experts of hidden size 2048 and SwiGLU width 512, eight experts a token, and the small
    layer of 64 experts, hidden size 1024 and width 256, four a token."""
    return [
        # the inputs of a 16-request decode batch on their way into the expert products: launch latency
        {"name": "mx rows, decode batch", "op": "mx_round_trip", "rows": 16, "cols": 2048, "type": _BF16, "out": _BF16},
        # the gate matrices of a layer's 256 experts, laid out once when a model is loaded: the largest conversion
        {"name": "mx rows, expert weights", "op": "mx_round_trip", "rows": 131072, "cols": 2048, "type": _F32, "out": _BF16},
        # one token's gate and up products: eight experts with one row each, the weights read once
        {"name": "mx gate/up, one token", "op": "mx_gemm", "rows": 8, "tokens": 1, "active": 8, "experts": 256, "n": 512,
         "k": 2048, "skew": 0.0, "swiglu": True, "gather": True, "weighted": False, "out": _BF16},
        # 16 requests share the popular experts: 29 of 256, the down product scaled by the routing weights
        {"name": "mx down, 16 requests", "op": "mx_gemm", "rows": 128, "tokens": 128, "active": 29, "experts": 256, "n": 2048,
         "k": 512, "skew": 1.1, "swiglu": False, "gather": False, "weighted": True, "out": _F32},
        # a 2048-token prompt chunk: about 64 rows an expert, the tokens' rows gathered
        {"name": "mx gate/up, prompt chunk", "op": "mx_gemm", "rows": 16384, "tokens": 2048, "active": 256, "experts": 256,
         "n": 512, "k": 2048, "skew": 0.3, "swiglu": True, "gather": True, "weighted": False, "out": _BF16},
        # several prompts at once, 16384 tokens: the matrix cores and the output rows
        {"name": "mx down, many prompts", "op": "mx_gemm", "rows": 131072, "tokens": 131072, "active": 256, "experts": 256,
         "n": 2048, "k": 512, "skew": 0.3, "swiglu": False, "gather": False, "weighted": True, "out": _BF16},
        # one token through 16-bit experts: the down product
        {"name": "down, one token", "op": "gemm", "rows": 8, "tokens": 8, "active": 8, "experts": 256, "n": 2048, "k": 512,
         "skew": 0.0, "gather": False, "weighted": True, "type": _BF16, "out": _F32},
        # a prompt chunk or a training batch of 2048 tokens: gate and up rows in one matrix
        {"name": "gate/up, prompt chunk", "op": "gemm", "rows": 16384, "tokens": 2048, "active": 256, "experts": 256, "n": 1024,
         "k": 2048, "skew": 0.3, "gather": True, "weighted": False, "type": _BF16, "out": _BF16},
        # the gradient by the rows of a small training batch on the small layer, float16, some experts without rows
        {"name": "dx, small layer", "op": "gemm_dx", "rows": 1000, "active": 50, "experts": 64, "n": 512, "k": 1024, "skew": 0.7,
         "type": _F16, "out": _F32},
        # the same of a training batch of 4096 tokens on the large layer
        {"name": "dx, training batch", "op": "gemm_dx", "rows": 32768, "active": 256, "experts": 256, "n": 1024, "k": 2048,
         "skew": 0.3, "type": _BF16, "out": _BF16},
        # the gradient by the matrices: odd widths, ragged groups, experts without rows get zeros
        {"name": "dw, odd widths", "op": "gemm_dw", "rows": 4001, "tokens": 1501, "active": 50, "experts": 64, "n": 520,
         "k": 1000, "skew": 0.7, "gather": True, "type": _F16, "out": _F16},
        # the same of a training batch of 4096 tokens on the large layer, held in 32 bits
        {"name": "dw, training batch", "op": "gemm_dw", "rows": 32768, "tokens": 4096, "active": 256, "experts": 256, "n": 1024,
         "k": 2048, "skew": 0.3, "gather": True, "type": _BF16, "out": _F32},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One token to a large training batch, one expert to 256, narrow to wide matrices, odd widths wherever an operator
    takes them (16-bit matrices: multiples of eight)."""
    op = rng.choice(["mx_round_trip", "mx_gemm", "mx_gemm", "gemm", "gemm", "gemm_dx", "gemm_dw"])
    if op == "mx_round_trip":
        cols = _spread(rng, 32, 4096)
        return {"op": op, "rows": _spread(rng, 1, (131072 * 2048) // cols // 2), "cols": cols,
                "type": rng.choice([_BF16, _F16, _F32]), "out": rng.choice([_BF16, _F32])}
    experts = _spread(rng, 1, 256)
    n, k = (_spread(rng, 40, 2048) for _ in range(2))
    if op != "mx_gemm":
        n, k = (max(8, v // 8 * 8) for v in (n, k))
    rows = _spread(rng, 1, 32768)
    active = min(rows, experts, rng.randint(max(1, experts // 4), experts))
    c = {"op": op, "rows": rows, "active": active, "experts": experts, "n": n, "k": k, "skew": rng.choice([0.0, 0.3, 0.7, 1.1])}
    if op == "mx_gemm":
        c |= {"swiglu": rng.random() < 0.5}
        if c["swiglu"]:
            c["n"] = max(20, n // 2)
    if op in ("mx_gemm", "gemm", "gemm_dw"):
        c["gather"] = rng.random() < 0.5
        c["tokens"] = max(1, rows // rng.randint(1, 8)) if c["gather"] else rows
    if op in ("mx_gemm", "gemm"):
        c["weighted"] = rng.random() < 0.5
    if op == "mx_gemm":
        c["out"] = rng.choice([_BF16, _F16, _F32])
    else:
        c["type"] = rng.choice([_BF16, _F16])
        c["out"] = rng.choice([c["type"], _F32])
    return c


def work(case):
    c = case
    if c["op"] == "mx_round_trip":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (_SIZE[c["type"]] + 2 * 17 / 32 + _SIZE[c["out"]]), "flops": n}
    rows, n, k = c["rows"], c["n"], c["k"]
    if c["op"] == "mx_gemm":
        mats = 2 if c["swiglu"] else 1
        return {"bytes": (mats * c["active"] * n + min(rows, c["tokens"])) * k * 17 / 32 + rows * n * _SIZE[c["out"]],
                "flops": 2.0 * mats * rows * n * k}
    flops = 2.0 * rows * n * k
    if c["op"] == "gemm":
        return {"bytes": 2 * (c["active"] * n + min(rows, c["tokens"])) * k + rows * n * _SIZE[c["out"]], "flops": flops}
    if c["op"] == "gemm_dx":
        return {"bytes": 2 * (c["active"] * n * k + rows * n) + rows * k * _SIZE[c["out"]], "flops": flops}
    return {"bytes": 2 * (rows * n + min(rows, c["tokens"]) * k) + c["experts"] * n * k * _SIZE[c["out"]], "flops": flops}


# ---- inputs ---------------------------------------------------------------------------------------------------------

def _pad_cols(cols):
    return -(-cols // 128) * 128


def _codes(x):
    """MXFP4 codes (two a byte, the earlier element in the low bits) and scale bytes of finite rows, the rows padded with
    zeros to a multiple of 128 elements."""
    rows, cols = x.shape
    v = torch.zeros((rows, _pad_cols(cols)), dtype=torch.float64, device=x.device)
    v[:, :cols] = x
    v = v.reshape(rows, -1, 32)
    amax = v.abs().amax(dim=2, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -127).clamp(-127, 127)
    y = torch.ldexp(v, -e)
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6.0)
    code = torch.bucketize(a.float(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device))
    code = (code | torch.where(y < 0, 8, 0)).reshape(rows, -1, 2)
    return (code[..., 0] | (code[..., 1] << 4)).to(torch.uint8), (e + 127).reshape(rows, -1).to(torch.uint8)


def _many_codes(gen, dev, rows, cols, scale):
    """Codes of rows of normal values, made in parts so that their 64-bit values stay small."""
    q = torch.empty((rows, _pad_cols(cols) // 2), dtype=torch.uint8, device=dev)
    s = torch.empty((rows, _pad_cols(cols) // 32), dtype=torch.uint8, device=dev)
    part = max(1, (64 << 20) // cols)
    for r in range(0, rows, part):
        x = torch.randn((min(part, rows - r), cols), generator=gen, device=dev) * scale
        q[r:r + part], s[r:r + part] = _codes(x)
    return q, s


def _groups(case, gen, dev):
    """Group sizes with exactly case["active"] experts in use, popular ones larger with the skew, and the row order's token
    of each row: every expert's rows in the order of their tokens, as a permutation by expert leaves them."""
    rows, experts, active = case["rows"], case["experts"], case["active"]
    used = torch.randperm(experts, generator=gen, device=dev)[:active]
    p = torch.arange(1, active + 1, device=dev, dtype=torch.float32) ** -case["skew"]
    counts = torch.zeros(experts, dtype=torch.int64, device=dev)
    counts[used] = 1
    more = torch.multinomial(p, rows - active, replacement=True, generator=gen) if rows > active else used[:0]
    counts += torch.bincount(used[more], minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=dev)
    offsets[1:] = torch.cumsum(counts, 0)
    most = int(counts.max())
    tok = None
    if case.get("gather"):
        t = torch.randperm(rows, generator=gen, device=dev) % case["tokens"]
        of = torch.repeat_interleave(torch.arange(experts, device=dev), counts)
        tok = (torch.sort(of * case["tokens"] + t)[0] % case["tokens"]).to(torch.int32)
    return {"offsets": offsets, "row_tok": tok, "most": most, "active": torch.sort(used)[0]}


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    c = case
    if c["op"] == "mx_round_trip":
        # rows with a spread of magnitudes from row to row and a few large channels, as activations and weights have
        x = torch.randn((c["rows"], c["cols"]), generator=gen, device=dev)
        x *= torch.exp(torch.randn((c["rows"], 1), generator=gen, device=dev))
        x *= torch.where(torch.rand(c["cols"], generator=gen, device=dev) < 0.01, 20.0, 1.0)
        rows, cols = x.shape
        return {"op": c["op"], "x": x.clamp(-6e4, 6e4).to(_TORCH[c["type"]]), "out_type": _TORCH[c["out"]],
                "q": torch.empty((rows, _pad_cols(cols) // 2), dtype=torch.uint8, device=dev),
                "s": torch.empty((rows, _pad_cols(cols) // 32), dtype=torch.uint8, device=dev),
                "out": torch.empty((rows, cols), dtype=_TORCH[c["out"]], device=dev)}
    rows, n, k, experts = c["rows"], c["n"], c["k"], c["experts"]
    st = {"op": c["op"], "rows": rows, "n": n, "k": k, "experts": experts, "out_type": _TORCH[c["out"]], **_groups(c, gen, dev)}
    weighted = c.get("weighted", False)
    st["row_w"] = torch.rand(rows, generator=gen, device=dev) * 0.5 if weighted else None
    if c["op"] == "mx_gemm":
        st["x"] = _many_codes(gen, dev, c["tokens"], k, 1.0)
        st["w"] = _many_codes(gen, dev, experts * n, k, 1 / math.sqrt(k))
        st["up"] = _many_codes(gen, dev, experts * n, k, 1 / math.sqrt(k)) if c["swiglu"] else None
        shape = (rows, n)
    else:
        t = _TORCH[c["type"]]

        def normal(*shape, scale=1.0):
            return (torch.randn(shape, generator=gen, device=dev) * scale).to(t)

        if c["op"] != "gemm_dw":
            st["w"] = normal(experts, n, k, scale=1 / math.sqrt(k))
        if c["op"] != "gemm_dx":
            st["x"] = normal(c["tokens"], k)
        if c["op"] != "gemm":
            st["dy"] = normal(rows, n)
        shape = {"gemm": (rows, n), "gemm_dx": (rows, k), "gemm_dw": (experts, n, k)}[c["op"]]
    st["out"] = torch.empty(shape, dtype=st["out_type"], device=dev)
    return st


# ---- one pass -------------------------------------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    from mixture_experts_decode_moe_amd import binding as mb
    op, out = st["op"], st["out"]
    if op == "mx_round_trip":
        mb.mx_quantize(st["x"], st["q"], st["s"])
        mb.mx_dequantize(st["q"], st["s"], out)
    elif op == "mx_gemm":
        mb.mx_grouped_gemm(st["x"], st["w"], st["experts"], st["k"], st["offsets"], out, up=st["up"], row_tok=st["row_tok"],
                           row_w=st["row_w"])
    elif op == "gemm":
        mb.grouped_gemm(st["x"], st["w"], st["offsets"], out, row_tok=st["row_tok"], row_w=st["row_w"])
    elif op == "gemm_dx":
        mb.grouped_gemm_dx(st["dy"], st["w"], st["offsets"], out)
    else:
        mb.grouped_gemm_dw(st["dy"], st["x"], st["offsets"], out, row_tok=st["row_tok"])
    return out


def _values(codes, cols):
    """The values that MXFP4 codes and scales stand for, in 32 bits."""
    q, s = codes
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=q.device)
    v = torch.stack([table[(q & 15).int()], table[(q >> 4).int()]], dim=-1).reshape(q.shape[0], -1, 32)
    return (v * torch.exp2(s.float() - 127)[..., None]).reshape(q.shape[0], -1)[:, :cols]


def _places(st):
    """Of each row: its group among the groups in use, and its place in that group."""
    r = torch.arange(st["rows"], device=st["offsets"].device, dtype=torch.int32)
    e = torch.searchsorted(st["offsets"][1:], r, right=True)
    return torch.searchsorted(st["active"], e), r - st["offsets"][e]


def _padded(st, rows, places):
    """Rows in 32 bits laid out [groups in use][longest group][width], the rest zero."""
    out = torch.zeros((st["active"].numel(), st["most"], rows.shape[1]), device=rows.device)
    out[places] = rows.float()
    return out


def _run_plain(st):
    op = st["op"]
    if op == "mx_round_trip":
        x = st["x"]
        return _values(_codes(x), x.shape[1]).to(st["out_type"])
    places = _places(st)
    if op in ("mx_gemm", "gemm"):
        x = _values(st["x"], st["k"]) if op == "mx_gemm" else st["x"]
        x = _padded(st, x if st["row_tok"] is None else x[st["row_tok"].long()], places)

        def product(w):
            if op == "mx_gemm":
                q, s = (v.reshape(st["experts"], st["n"], -1)[st["active"]] for v in w)
                w = _values((q.reshape(-1, q.shape[2]), s.reshape(-1, s.shape[2])), st["k"]).reshape(-1, st["n"], st["k"])
            else:
                w = w[st["active"]].float()
            return torch.bmm(x, w.transpose(1, 2))[places]

        y = product(st["w"])
        if st.get("up") is not None:
            y = y / (1 + torch.exp(-y)) * product(st["up"])
        if st["row_w"] is not None:
            y = y * st["row_w"][:, None]
        return y.to(st["out_type"])
    dy = _padded(st, st["dy"], places)
    if op == "gemm_dx":
        return torch.bmm(dy, st["w"][st["active"]].float())[places].to(st["out_type"])
    x = st["x"] if st["row_tok"] is None else st["x"][st["row_tok"].long()]
    dw = torch.zeros((st["experts"], st["n"], st["k"]), dtype=st["out_type"], device=dy.device)
    dw[st["active"]] = torch.bmm(dy.transpose(1, 2), _padded(st, x, places)).to(st["out_type"])
    return dw


# ---- in 64 bits -----------------------------------------------------------------------------------------------------

def _exact_codes(x):
    """The values of the nearest codes, by the distance to each of the eight magnitudes (ties to the even code)."""
    rows, cols = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -cols % 32)).reshape(-1, 32)
    amax = v.abs().amax(dim=1, keepdim=True)
    e = ((amax.view(torch.int64) >> 52) - 1023 - 2).clamp(-127, 127)
    scale = ((e + 1023) << 52).view(torch.float64)
    best, value = torch.full_like(v, math.inf), torch.zeros_like(v)
    for code in (0, 2, 4, 6, 1, 3, 5, 7):  # the even codes first: an odd one has to be nearer
        m = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)[code]
        d = (v.abs() - m * scale).abs()
        value = torch.where(d < best, m * scale, value)
        best = torch.minimum(d, best)
    return (value * torch.sign(v)).reshape(rows, -1)[:, :cols]


def _exact_values(codes, cols):
    q, s = codes
    n = torch.stack([q & 15, q >> 4], dim=-1).reshape(q.shape[0], -1).long()
    e, m = (n >> 1) & 3, (n & 1).double() / 2
    v = torch.where(e == 0, m, (1 + m) * 2.0 ** (e - 1).double()) * (1 - 2 * (n >> 3)).double()
    return (v * torch.repeat_interleave(2.0 ** (s.double() - 127), 32, dim=1))[:, :cols]


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "mx_round_trip":
        part = max(1, (64 << 20) // case["cols"])
        return torch.cat([_exact_codes(p) for p in torch.split(st["x"], part)])
    off, n, k = st["offsets"].tolist(), case["n"], case["k"]
    wide = case["k"] if op == "gemm_dx" else case["n"]
    out = torch.zeros((case["experts"], n, k) if op == "gemm_dw" else (case["rows"], wide), dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        if op != "gemm_dx":
            at = st["row_tok"][a:b].long() if case["gather"] else torch.arange(a, b, device="cuda")
        if op == "mx_gemm":
            x = _exact_values((st["x"][0][at], st["x"][1][at]), k)

            def matrix(w):
                return _exact_values((w[0][e * n:(e + 1) * n], w[1][e * n:(e + 1) * n]), k)

            y = x @ matrix(st["w"]).T.contiguous()
            if case["swiglu"]:
                y = y * torch.sigmoid(y) * (x @ matrix(st["up"]).T.contiguous())
        elif op == "gemm":
            y = st["x"][at].double() @ st["w"][e].double().T.contiguous()
        elif op == "gemm_dx":
            y = st["dy"][a:b].double() @ st["w"][e].double()
        else:
            out[e] = st["dy"][a:b].double().T.contiguous() @ st["x"][at].double()
            continue
        out[a:b] = y * st["row_w"][a:b, None].double() if st.get("row_w") is not None else y
    return out
