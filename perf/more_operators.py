"""Cases of the operators between the 8-bit GEMMs: the root-mean-square norm with the residual's addition and an output
in 8 bits, its backward pass, tokens sorted by expert and back with their gradients, and the INT8 linear layer.

`run` computes a case in its plain form (elementary torch operations in 32 bits, rounded once at the end) or, where
`own` is true, through moe_grouped_gemm_x128_amd."""
import math

import numpy as np
import torch

own = False
_dg = None

DEV = "cuda"
BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
EPS = 1e-6
SEGMENT = 128  # rows that an expert's segment of the contiguous layout is a multiple of


def _lib():
    global _dg
    if _dg is None:
        import moe_grouped_gemm_x128_amd
        _dg = moe_grouped_gemm_x128_amd
    return _dg


def listed():
    return [
        # one token of a generation step before its FP8 experts: latency
        dict(name="norm fp8 one token", op="norm", out="fp8", t=1, h=7168, residual=True, weight="bf16", keep=False),
        # a prefill chunk before its FP8 experts
        dict(name="norm fp8 prefill", op="norm", out="fp8", t=4096, h=7168, residual=True, weight="bf16", keep=False),
        # a training step's forward over rows of an odd width: 1/rms is kept for the backward pass
        dict(name="norm bf16 odd training", op="norm", out="bf16", t=333, h=2111, residual=True, weight="f32",
             keep=True),
        # a training step's backward: the residual stream brings a gradient of its own
        dict(name="norm backward training", op="norm_backward", t=4096, h=4096, stream=True, weight="f32"),
        # a fine-tuning micro-batch of odd length and width, no residual stream
        dict(name="norm backward odd", op="norm_backward", t=517, h=1161, stream=False, weight="bf16"),
        # a decode batch through an INT8 layer
        dict(name="int8 decode batch", op="int8", m=16, n=4096, k=7168, act="gelu_tanh", bias=True, residual=False,
             out="bf16"),
        # a prompt of odd length through an INT8 layer whose width is odd too
        dict(name="int8 odd prompt", op="int8", m=333, n=2111, k=1536, act="silu", bias=True, residual=True,
             out="bf16"),
        # a prefill chunk: the norm writes the INT8 layer's operand
        dict(name="norm int8 prefill", op="norm_int8", t=4096, h=4096, n=7168, residual=True, weight="bf16",
             act="none", bias=True),
        # a decode batch spread over the experts' slots; a part of the tokens' experts is on other devices
        dict(name="dispatch masked decode", op="dispatch", layout="masked", out="fp8", t=64, e=32, experts=64, top_k=8,
             h=7168, m_max=64),
        # a prefill chunk spread over the experts' segments
        dict(name="dispatch contiguous prefill", op="dispatch", layout="contiguous", out="fp8", t=8192, e=64,
             experts=64, top_k=8, h=7168, m_max=0),
        # the experts' outputs of a short odd prompt back in token order, added to the residual stream
        dict(name="combine odd prompt", op="combine", t=777, e=24, experts=32, top_k=6, h=2048, weights=True,
             residual=True),
        # a training step's gradients through combine and dispatch
        dict(name="moe backward training", op="moe_backward", t=4096, e=64, experts=64, top_k=8, h=4096),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "int8", "int8", "norm_int8", "dispatch", "dispatch", "combine",
                     "moe_backward"])
    weight = rng.choice(["bf16", "f32"])
    if op == "norm":
        out = rng.choice(["bf16", "fp8", "fp8_ue8m0"])
        t = _log_int(rng, 1, 8192)
        h = _log_int(rng, 64, 8192) if out == "bf16" else 128 * _log_int(rng, 1, 64)
        return dict(op=op, out=out, t=t, h=h, residual=rng.random() < 0.7, weight=weight, keep=rng.random() < 0.3)
    if op == "norm_backward":
        h = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            h = -(-h // 8) * 8
        return dict(op=op, t=_log_int(rng, 8, 8192), h=h, stream=rng.random() < 0.6, weight=weight)
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
    if op == "int8":
        return dict(op=op, m=_log_int(rng, 1, 4096), n=_log_int(rng, 64, 8192), k=16 * _log_int(rng, 16, 512), act=act,
                    bias=rng.random() < 0.7, residual=rng.random() < 0.5, out="f32" if rng.random() < 0.2 else "bf16")
    if op == "norm_int8":
        return dict(op=op, t=_log_int(rng, 1, 4096), h=16 * _log_int(rng, 16, 448), n=_log_int(rng, 64, 7168),
                    residual=rng.random() < 0.7, weight=weight, act=act, bias=rng.random() < 0.5)
    experts = rng.choice([8, 16, 64, 128, 256])
    c = dict(op=op, t=_log_int(rng, 1, 4096), e=experts // rng.choice([1, 1, 2, 4]), experts=experts,
             top_k=rng.randint(1, 8), h=128 * _log_int(rng, 4, 56))
    if op == "dispatch":
        masked = c["t"] <= 256 and rng.random() < 0.6
        c.update(layout="masked" if masked else "contiguous", out=rng.choice(["fp8", "fp8", "bf16"]),
                 m_max=rng.choice([16, 64, 128]) if masked else 0)
    elif op == "combine":
        c.update(weights=rng.random() < 0.7, residual=rng.random() < 0.6)
    return c


# ---- inputs -------------------------------------------------------------------------------------------------------

def _codes(x):
    """INT8 codes and fp32 scales of x [M, K]: one scale per row, absmax / 127."""
    s = x.abs().amax(1) / 127
    s = torch.where(s == 0, torch.ones_like(s), s)
    return torch.round(x / s[:, None]).clamp(-127, 127).to(torch.int8), s


def _fp8_codes(x):
    """FP8 codes and fp32 scales of x [T, H]: one scale per row and 128 columns, absmax / 448."""
    t, h = x.shape
    g = x.view(t, h // 128, 128)
    s = g.abs().amax(2) / 448
    s = torch.where(s == 0, torch.ones_like(s), s)
    return (g / s[:, :, None]).clamp(-448, 448).view(t, h).to(FP8), s


def _capacity(c):
    """Rows of the contiguous layout that hold any routing: every expert's last segment may be nearly empty."""
    slots = c["t"] * c["top_k"]
    return max(SEGMENT, (slots + min(c["e"], slots) * (SEGMENT - 1)) // SEGMENT * SEGMENT)


def _routing(gen, c):
    """ids int32 [T, k]: distinct experts of a token, some of them liked better than others, in the local numbering
    (0 <= id < e; the others are on other devices)."""
    logits = torch.randn((c["t"], c["experts"]), generator=gen, device=DEV)
    logits += 0.5 * torch.randn((1, c["experts"]), generator=gen, device=DEV)
    top, ids = torch.sort(logits, dim=1, descending=True)
    w = torch.softmax(top[:, :c["top_k"]], 1)
    return (ids[:, :c["top_k"]] - (c["experts"] - c["e"]) // 2).to(torch.int32).contiguous(), w.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 7919 + 29)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    def new(*shape, dtype=BF16):
        return torch.empty(shape, dtype=dtype, device=DEV)

    c = case
    s = dict(case=case)
    op = c["op"]
    if op in ("norm", "norm_int8"):
        t, h = c["t"], c["h"]
        # a residual stream: some channels are much larger than the others
        s["x"] = randn(t, h).to(BF16)
        s["residual"] = (randn(t, h) * torch.exp(1.2 * randn(1, h))).to(BF16) if c["residual"] else None
        s["w"] = (1 + 0.2 * randn(h)).to(BF16 if c["weight"] == "bf16" else F32)
        s["sum"] = new(t, h) if c["residual"] else None
    if op == "norm":
        s["rstd"] = new(t, dtype=F32) if c["keep"] else None
        if c["out"] == "bf16":
            s["y"] = new(t, h)
        else:
            s["q"] = new(t, h, dtype=FP8)
            s["s"] = new(t, h // 128, dtype=F32) if c["out"] == "fp8" else new(t, -(-h // 512), dtype=torch.int32)
        return s
    if op == "norm_backward":
        t, h = c["t"], c["h"]
        x = (randn(t, h) * torch.exp(0.5 * randn(1, h))).to(BF16)
        s["x"], s["dy"] = x, randn(t, h).to(BF16)
        s["w"] = (1 + 0.2 * randn(h)).to(BF16 if c["weight"] == "bf16" else F32)
        s["rstd"] = torch.rsqrt(x.float().square().mean(1) + EPS)
        s["dsum"] = randn(t, h).to(BF16) if c["stream"] else None
        s["dx"], s["dw"] = new(t, h), new(h, dtype=F32)
        return s
    if op in ("int8", "norm_int8"):
        m, n, k = (c["m"], c["n"], c["k"]) if op == "int8" else (c["t"], c["n"], c["h"])
        if op == "int8":
            s["a"] = _codes(randn(m, k) * torch.exp(0.5 * randn(1, k)))
            s["residual"] = randn(m, n).to(BF16) if c["residual"] else None
        else:
            s["a"] = new(m, k, dtype=torch.int8), new(m, dtype=F32)
        s["b"] = _codes(randn(n, k) / math.sqrt(k))
        s["bias"] = 0.2 * randn(n) if c["bias"] else None
        s["out"] = new(m, n, dtype=F32 if c.get("out") == "f32" else BF16)
        return s
    t, h, k = c["t"], c["h"], c["top_k"]
    s["ids"], s["weights"] = _routing(gen, c)
    if op == "dispatch":
        masked = c["layout"] == "masked"
        m = c["e"] * c["m_max"] if masked else _capacity(c)
        x = randn(t, h)
        s["rows"] = new(t, k, dtype=torch.int32)
        if masked:
            s["masked_m"] = new(c["e"], dtype=torch.int32)
        else:
            s["m_indices"] = new(m, dtype=torch.int32)
        # (rows that no token takes keep what they hold: zeros here)
        if c["out"] == "fp8":
            s["x"] = _fp8_codes(x)
            s["a"] = torch.zeros((m, h), dtype=torch.uint8, device=DEV).view(FP8)
            s["sa"] = torch.zeros((m, h // 128), dtype=F32, device=DEV)
        else:
            s["x"] = x.to(BF16)
            s["a"] = torch.zeros((m, h), dtype=BF16, device=DEV)
        return s
    s["m"] = m = _capacity(c)
    rows, m_indices, _ = _sorted(s["ids"], c["e"], m)
    s["rows"], s["m_indices"] = rows, m_indices
    s["o"] = randn(m, h).to(BF16)
    if op == "combine":
        if not c["weights"]:
            s["weights"] = None
        s["residual"] = randn(t, h).to(BF16) if c["residual"] else None
        s["y"] = new(t, h)
        return s
    s["dy"], s["da"] = randn(t, h).to(BF16), randn(m, h).to(BF16)
    s["do"] = torch.zeros((m, h), dtype=BF16, device=DEV)
    s["dweights"], s["dx"] = new(t, k, dtype=F32), new(t, h)
    return s


# ---- one pass -----------------------------------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    dg, c = _lib(), s["case"]
    op = c["op"]
    if op == "norm":
        if c["out"] == "bf16":
            dg.rmsnorm_bf16(s["x"], s["w"], s["y"], EPS, residual=s["residual"], sum_out=s["sum"], rstd=s["rstd"])
            return [s["sum"], s["rstd"], s["y"]]
        dg.rmsnorm_quantize_fp8_1x128(s["x"], s["w"], s["q"], s["s"], EPS, residual=s["residual"], sum_out=s["sum"],
                                      rstd=s["rstd"])
        return [s["sum"], s["rstd"], s["q"], _scale_values(s["s"])]
    if op == "norm_backward":
        dg.rmsnorm_bf16_backward(s["dy"], s["x"], s["w"], s["rstd"], s["dx"], s["dw"], dsum=s["dsum"])
        return [s["dx"], s["dw"]]
    if op == "int8":
        return dg.gemm_int8_nt_epilogue(s["a"], s["b"], s["out"], s["bias"], c["act"], s["residual"])
    if op == "norm_int8":
        dg.rmsnorm_quantize_int8(s["x"], s["w"], *s["a"], EPS, residual=s["residual"], sum_out=s["sum"])
        dg.gemm_int8_nt_epilogue(s["a"], s["b"], s["out"], s["bias"], c["act"])
        return [s["sum"], s["out"]]
    if op == "dispatch":
        if c["layout"] == "masked":
            first = s["masked_m"]
            dg.moe_sort_masked(s["ids"], c["m_max"], first, s["rows"])
        else:
            first = s["m_indices"]
            dg.moe_sort_contiguous(s["ids"], c["e"], first, s["rows"])
        if c["out"] == "fp8":
            dg.moe_dispatch_fp8(s["x"], s["rows"], (s["a"], s["sa"]))
            return [first, s["rows"], s["a"], s["sa"]]
        dg.moe_dispatch_bf16(s["x"], s["rows"], s["a"])
        return [first, s["rows"], s["a"]]
    if op == "combine":
        return dg.moe_combine_bf16(s["o"], s["rows"], s["y"], s["weights"], s["residual"])
    dg.moe_combine_bf16_backward(s["dy"], s["o"], s["rows"], s["weights"], s["do"], s["dweights"], s["m_indices"])
    dg.moe_dispatch_bf16_backward(s["da"], s["rows"], s["dx"])
    return [s["do"], s["dweights"], s["dx"]]


def _scale_values(s):
    """Packed power-of-two scales as the values of their bytes."""
    return s if s.dtype == F32 else s.view(torch.float8_e8m0fnu)


def _act(x, act):
    if act == "relu":
        return torch.clamp(x, min=0)
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    if act == "silu":
        return x * torch.sigmoid(x)
    return x


def _norm(s):
    """x + residual rounded (None without a residual), 1 / rms and the normed rows, in 32 bits."""
    z = s["x"].float()
    if s["residual"] is not None:
        z = z + s["residual"].float()
    r = torch.rsqrt((z * z).mean(1) + EPS)
    return z.to(BF16) if s["residual"] is not None else None, r, z * r[:, None] * s["w"].float()


def _power_codes(s):
    """Bytes of the least powers of two not below the fp32 scales s [T, G], each row padded with zeros to whole words."""
    bits = s.view(torch.int32)
    e = (bits >> 23) + ((bits & 0x7fffff) != 0)
    pad = torch.zeros((s.shape[0], -s.shape[1] % 4), dtype=e.dtype, device=DEV)
    return torch.cat([e, pad], 1).to(torch.uint8)


def _sorted(ids, experts, limit, m_max=None):
    """Destination row of every slot (-1: none), the expert of every row of the contiguous layout, rows per expert."""
    key = ids.reshape(-1).long()
    key = torch.where((key >= 0) & (key < experts), key, torch.full_like(key, experts))
    ordered, order = torch.sort(key, stable=True)
    first = torch.searchsorted(ordered, torch.arange(experts + 1, device=DEV))
    count = first[1:] - first[:-1]
    if m_max is None:
        padded = (count + SEGMENT - 1) // SEGMENT * SEGMENT
        start = torch.cumsum(padded, 0) - padded
    else:
        start = torch.arange(experts, device=DEV) * m_max
    rank = torch.arange(key.numel(), device=DEV) - first[ordered]
    row = torch.cat([start, start.new_zeros(1)])[ordered] + rank
    kept = (ordered < experts) & (row < limit if m_max is None else rank < m_max)
    rows = torch.empty_like(key)
    rows[order] = torch.where(kept, row, torch.full_like(row, -1))
    m_indices = torch.full((limit + 1,), -1, dtype=torch.int32, device=DEV)
    m_indices[torch.where(kept, row, torch.full_like(row, limit))] = ordered.to(torch.int32)
    if m_max is not None:
        count = torch.clamp(count, max=m_max)
    return rows.view(ids.shape).to(torch.int32), m_indices[:limit].contiguous(), count.to(torch.int32)


def _spread(x, rows, m):
    """x [T, ...] at the rows of its slots, zeros elsewhere."""
    out = torch.zeros((m + 1, x.shape[1]), dtype=x.dtype, device=DEV)
    at = torch.where(rows < 0, torch.full_like(rows, m), rows).reshape(-1).long()
    out[at] = x.repeat_interleave(rows.shape[1], 0)
    return out[:m]


def _gathered(o, rows):
    """o's rows of every slot [T, k, H], zeros where a slot has none, in 32 bits."""
    return torch.where((rows >= 0)[:, :, None], o[rows.clamp(min=0).long()].float(), torch.zeros((), device=DEV))


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm":
        total, r, y = _norm(s)
        r = r if c["keep"] else None
        if c["out"] == "bf16":
            return [total, r, y.to(BF16)]
        if c["out"] == "fp8":
            return [total, r, *_fp8_codes(y)]
        t, h = y.shape
        g = y.view(t, h // 128, 128)
        amax = g.abs().amax(2) / 448
        e = _power_codes(torch.where(amax == 0, torch.ones_like(amax), amax))
        scale = torch.exp2(e[:, :h // 128].float() - 127)
        return [total, r, (g / scale[:, :, None]).clamp(-448, 448).view(t, h).to(FP8),
                e.view(torch.float8_e8m0fnu)]
    if op == "norm_backward":
        x, dy, r = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
        n = x * r
        g = dy * s["w"].float()
        dx = r * (g - n * (g * n).mean(1, keepdim=True))
        if c["stream"]:
            dx = dx + s["dsum"].float()
        return [dx.to(BF16), (dy * n).sum(0)]
    if op in ("int8", "norm_int8"):
        if op == "int8":
            (qa, sa), total = s["a"], None
        else:
            total, _, y = _norm(s)
            qa, sa = _codes(y)
        qb, sb = s["b"]
        y = (qa.float() @ qb.float().t()) * sa[:, None] * sb
        if c["bias"]:
            y = y + s["bias"]
        y = _act(y, c["act"])
        if op == "norm_int8":
            return [total, y.to(BF16)]
        if c["residual"]:
            y = y + s["residual"].float()
        return y.to(s["out"].dtype)
    if op == "dispatch":
        m = s["a"].shape[0]
        rows, m_indices, count = _sorted(s["ids"], c["e"], m, c["m_max"] if c["layout"] == "masked" else None)
        first = count if c["layout"] == "masked" else m_indices
        if c["out"] == "fp8":
            q, scale = s["x"]
            return [first, rows, _spread(q.view(torch.uint8), rows, m).view(FP8), _spread(scale, rows, m)]
        return [first, rows, _spread(s["x"], rows, m)]
    rows = s["rows"]
    o = _gathered(s["o"], rows)
    if op == "combine":
        y = (o * s["weights"][:, :, None]).sum(1) if c["weights"] else o.sum(1)
        if c["residual"]:
            y = y + s["residual"].float()
        return y.to(BF16)
    dy = s["dy"].float()
    w = s["weights"].reshape(-1, 1) * dy.repeat_interleave(c["top_k"], 0)
    do = torch.zeros((s["m"] + 1, c["h"]), dtype=BF16, device=DEV)
    do[torch.where(rows < 0, torch.full_like(rows, s["m"]), rows).reshape(-1).long()] = w.to(BF16)
    return [do[:s["m"]], (o * dy[:, None, :]).sum(2), _gathered(s["da"], rows).sum(1).to(BF16)]


# ---- 64 bits ------------------------------------------------------------------------------------------------------

def _rows_by_hand(ids, c, m):
    """Rows, experts of rows and rows per expert by walking the experts in order, on the host."""
    flat = ids.cpu().numpy().reshape(-1)
    rows, of, counts, start = np.full(flat.size, -1, np.int64), np.full(m, -1, np.int64), [], 0
    for e in range(c["e"]):
        at = np.nonzero(flat == e)[0]
        if c.get("layout") == "masked":
            at = at[:c["m_max"]]
            rows[at] = e * c["m_max"] + np.arange(at.size)
        else:
            rows[at] = start + np.arange(at.size)
            start += (at.size + SEGMENT - 1) // SEGMENT * SEGMENT
            of[rows[at]] = e
        counts.append(at.size)
    to = lambda v: torch.from_numpy(np.asarray(v, np.int32)).to(DEV)  # noqa: E731
    return to(rows).view(ids.shape), to(of), to(counts)


def _act64(x, act):
    return {"none": lambda v: v, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
            "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[act](x)


def _norm64(s):
    z = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
    r = 1 / torch.sqrt(torch.linalg.vector_norm(z, dim=1) ** 2 / z.shape[1] + EPS)
    return (None if s["residual"] is None else z), r, s["w"].double() * (z * r[:, None])


def exact(case, seed):
    c, s = case, prepare(case, seed)
    op = c["op"]
    if op == "norm":
        total, r, y = _norm64(s)
        r = r if c["keep"] else None
        if c["out"] == "bf16":
            return [total, r, y]
        groups = y.unflatten(1, (-1, 128))
        scale = torch.linalg.vector_norm(groups, ord=math.inf, dim=2) / 448
        scale[scale == 0] = 1
        if c["out"] == "fp8_ue8m0":
            scale = 2.0 ** torch.ceil(torch.log2(scale))
        y = (groups / scale[..., None]).flatten(1)
        if c["out"] == "fp8_ue8m0":  # (padding bytes of a row's last word stand for 2^-127)
            scale = torch.nn.functional.pad(scale, (0, -scale.shape[1] % 4), value=2.0 ** -127)
        return [total, r, y, scale]
    if op == "norm_backward":
        x, r = s["x"].double(), s["rstd"].double()
        g = s["w"].double() * s["dy"].double()
        dx = r[:, None] * g - x * (r ** 3 * torch.sum(x * g, 1) / x.shape[1])[:, None]
        if c["stream"]:
            dx += s["dsum"].double()
        return [dx, torch.mv((s["dy"].double() * x).t(), r)]
    if op in ("int8", "norm_int8"):
        if op == "int8":
            a, total = s["a"][0].double() * s["a"][1].double()[:, None], None
        else:
            total, _, y = _norm64(s)
            step = y.abs().max(1, keepdim=True).values / 127
            a = torch.round(y / step) * step
        y = a @ (s["b"][0].double() * s["b"][1].double()[:, None]).t()
        if c["bias"]:
            y += s["bias"].double()
        y = _act64(y, c["act"])
        if op == "norm_int8":
            return [total, y]
        return y + s["residual"].double() if c["residual"] else y
    if op == "dispatch":
        m = s["a"].shape[0]
        rows, of, counts = _rows_by_hand(s["ids"], c, m)
        token = torch.zeros(m, dtype=torch.long, device=DEV)
        used = torch.zeros(m, dtype=torch.bool, device=DEV)
        t, j = torch.nonzero(rows >= 0, as_tuple=True)
        token[rows[t, j].long()] = t
        used[rows[t, j].long()] = True
        first = counts if c["layout"] == "masked" else of

        def at(x):
            return x[token] * used[:, None].to(x.dtype)

        if c["out"] == "fp8":
            return [first, rows, at(s["x"][0].view(torch.uint8)).view(FP8), at(s["x"][1].double())]
        return [first, rows, at(s["x"])]
    rows, _, _ = _rows_by_hand(s["ids"], c, s["m"])
    t, j = torch.nonzero(rows >= 0, as_tuple=True)
    at = rows[t, j].long()

    def back(o, w):
        y = torch.zeros((c["t"], c["h"]), dtype=torch.float64, device=DEV)
        v = o[at].double()
        return y.index_add_(0, t, v if w is None else v * w[t, j].double()[:, None])

    if op == "combine":
        y = back(s["o"], s["weights"])
        return y + s["residual"].double() if c["residual"] else y
    do = torch.zeros((s["m"], c["h"]), dtype=torch.float64, device=DEV)
    do[at] = s["dy"][t].double() * s["weights"][t, j].double()[:, None]
    dw = torch.zeros(rows.shape, dtype=torch.float64, device=DEV)
    dw[t, j] = (s["dy"][t].double() * s["o"][at].double()).sum(1)
    return [do, dw, back(s["da"], None)]


# ---- what a pass cannot do without --------------------------------------------------------------------------------

def work(case):
    c = case
    op = c["op"]
    if op == "norm":
        v = c["t"] * c["h"]
        out = 2 * v if c["out"] == "bf16" else v + (v // 128 * 4 if c["out"] == "fp8" else 4 * c["t"] * -(-c["h"] // 512))
        return {"bytes": v * (6 if c["residual"] else 2) + out + c["h"] * (2 if c["weight"] == "bf16" else 4)
                + 4 * c["t"] * c["keep"], "flops": 8 * v}
    if op == "norm_backward":
        v = c["t"] * c["h"]
        return {"bytes": v * (8 if c["stream"] else 6) + 4 * c["t"] + c["h"] * (6 if c["weight"] == "bf16" else 8),
                "flops": 12 * v}
    if op in ("int8", "norm_int8"):
        m, n, k = (c["m"], c["n"], c["k"]) if op == "int8" else (c["t"], c["n"], c["h"])
        size = n * k + 4 * n + 4 * n * c["bias"]
        if op == "int8":
            size += m * k + 4 * m + m * n * ((4 if c["out"] == "f32" else 2) + 2 * c["residual"])
        else:  # (the 8-bit rows between the two calls stay on the chip at best)
            size += m * k * (6 if c["residual"] else 2) + k * (2 if c["weight"] == "bf16" else 4) + 2 * m * n
        return {"bytes": size, "flops": 2 * m * n * k}
    t, h, k = c["t"], c["h"], c["top_k"]
    kept = t * k * c["e"] / c["experts"]  # slots whose expert is here, were the choices even
    if op == "dispatch":
        if c["layout"] == "masked":
            kept = min(kept, c["e"] * c["m_max"])
        each = h + h // 128 * 4 if c["out"] == "fp8" else 2 * h
        return {"bytes": 8 * t * k + (4 * c["e"] if c["layout"] == "masked" else 4 * _capacity(c))
                + min(t, kept) * each + kept * each, "flops": 0}
    if op == "combine":
        return {"bytes": kept * 2 * h + t * h * (2 + 2 * c["residual"]) + t * k * (4 + 4 * c["weights"]),
                "flops": 2 * kept * h}
    return {"bytes": t * h * 4 + kept * 6 * h + t * k * 12 + 4 * _capacity(c), "flops": 4 * kept * h}
