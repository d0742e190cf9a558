"""Cases of the operators around the GEMMs: a linear layer with its epilogue (forward in BF16 and FP8, backward in
BF16) and a whole mixture-of-experts layer for a few tokens.

`run` computes a case in its plain form (elementary torch operations in 32 bits, rounded once at the end) or, where
`own` is true, through moe_grouped_gemm_x128_amd."""
import math

import torch

own = False
_dg = None

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def _lib():
    global _dg
    if _dg is None:
        import moe_grouped_gemm_x128_amd
        _dg = moe_grouped_gemm_x128_amd
    return _dg


def listed():
    return [
        # one token of a generation step through a projection with its residual
        dict(name="linear bf16 one token", op="linear", dtype="bf16", m=1, n=7168, k=2048, act="none", bias=True,
             residual=True, out="bf16", save=False),
        # the logits of a router over 256 experts for a small decode batch: few columns, long rows, fp32 result
        dict(name="linear bf16 router logits", op="linear", dtype="bf16", m=16, n=256, k=7168, act="none", bias=True,
             residual=False, out="f32", save=False),
        # a prompt of odd length through a layer whose width is odd too
        dict(name="linear bf16 odd prompt", op="linear", dtype="bf16", m=333, n=2111, k=1536, act="silu", bias=True,
             residual=True, out="bf16", save=False),
        # a training step's forward: the pre-activation is kept for the backward pass
        dict(name="linear bf16 training", op="linear", dtype="bf16", m=4096, n=7168, k=2048, act="gelu", bias=True,
             residual=False, out="bf16", save=True),
        # a decode batch on FP8 weights
        dict(name="linear fp8 decode batch", op="linear", dtype="fp8", m=64, n=4096, k=7168, act="gelu_tanh",
             bias=True, residual=False, out="bf16", save=False),
        # a prefill chunk on FP8 weights, added to the residual stream
        dict(name="linear fp8 prefill", op="linear", dtype="fp8", m=4096, n=4096, k=7168, act="none", bias=True,
             residual=True, out="bf16", save=False),
        # the backward pass of the training step above
        dict(name="linear backward training", op="backward", m=4096, n=7168, k=2048, act="gelu", bias=True),
        # a fine-tuning micro-batch of odd length on narrow layers
        dict(name="linear backward odd", op="backward", m=517, n=1161, k=1096, act="silu", bias=True),
        # one token through a small layer: latency
        dict(name="moe fp8 small one token", op="moe", dtype="fp8", t=1, e=8, top_k=2, h=1024, i=512, scoring="softmax",
             residual=False, routing="logits"),
        # one token of a generation step through a large layer
        dict(name="moe fp8 one token", op="moe", dtype="fp8", t=1, e=16, top_k=8, h=7168, i=2048, scoring="softmax",
             residual=True, routing="logits"),
        # a decode batch, routed by the caller, on BF16 weights
        dict(name="moe bf16 batch", op="moe", dtype="bf16", t=13, e=16, top_k=4, h=4096, i=1536, scoring="sigmoid",
             residual=False, routing="ids"),
        # the largest decode batch over many experts
        dict(name="moe fp8 large batch", op="moe", dtype="fp8", t=64, e=64, top_k=8, h=7168, i=2048, scoring="sigmoid",
             residual=True, routing="logits"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
    op = rng.choice(["linear", "linear", "backward", "moe", "moe"])
    if op == "linear":
        dtype = rng.choice(["bf16", "fp8"])
        step = 8 if dtype == "bf16" else 128
        m = _log_int(rng, 1, 4096)
        n = _log_int(rng, 64, 8192)
        k = step * max(1, _log_int(rng, 256, 8192) // step)
        return dict(op="linear", dtype=dtype, m=m, n=n, k=k, act=act, bias=rng.random() < 0.7,
                    residual=rng.random() < 0.5, out="f32" if rng.random() < 0.2 else "bf16",
                    save=dtype == "bf16" and act != "none" and rng.random() < 0.5)
    if op == "backward":
        return dict(op="backward", m=_log_int(rng, 16, 4096), n=_log_int(rng, 64, 7168),
                    k=8 * (_log_int(rng, 128, 4096) // 8), act=act, bias=rng.random() < 0.7)
    dtype = rng.choice(["bf16", "fp8"])
    e = rng.choice([4, 8, 16, 32])
    return dict(op="moe", dtype=dtype, t=_log_int(rng, 1, 64), e=e, top_k=rng.randint(1, min(8, e)),
                h=128 * _log_int(rng, 4, 56), i=128 * _log_int(rng, 2, 16), scoring=rng.choice(["softmax", "sigmoid"]),
                residual=rng.random() < 0.5, routing=rng.choice(["logits", "ids"]))


# ---- inputs -------------------------------------------------------------------------------------------------------

FP8_MAX = 448.0


def _quantise(x, rows):
    """FP8 codes and fp32 scales of x [N, K]: one scale per `rows` rows (1 or 128) and 128 columns, absmax / 448."""
    n, k = x.shape
    pad = (-n) % rows
    blocks = torch.nn.functional.pad(x, (0, 0, 0, pad)).view((n + pad) // rows, rows, k // 128, 128)
    s = blocks.abs().amax(dim=(1, 3)) / FP8_MAX
    s = torch.where(s == 0, torch.ones_like(s), s)
    q = (blocks / s[:, None, :, None]).clamp(-FP8_MAX, FP8_MAX).view(n + pad, k)[:n]
    return q.to(torch.float8_e4m3fn).contiguous(), s


def _expert_weights(gen, dtype, e, n, k):
    """The stacked weights of e experts, [e, n, k], made one expert at a time (n a multiple of 128)."""
    if dtype == "bf16":
        w = torch.empty((e, n, k), dtype=BF16, device=DEV)
        for j in range(e):
            w[j] = torch.randn((n, k), generator=gen, device=DEV) / math.sqrt(k)
        return w
    q = torch.empty((e, n, k), dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty((e, n // 128, k // 128), dtype=F32, device=DEV)
    for j in range(e):
        qj, sj = _quantise(torch.randn((n, k), generator=gen, device=DEV) / math.sqrt(k), 128)
        q.view(torch.uint8)[j] = qj.view(torch.uint8)
        s[j] = sj
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 7919 + 17)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    c = case
    s = dict(case=case)
    if c["op"] == "moe":
        t, e, h, i, top_k = c["t"], c["e"], c["h"], c["i"], c["top_k"]
        s["x"] = randn(t, h).to(BF16)
        # some experts are liked better than others, as trained routers like them
        s["logits"] = randn(t, e) + 0.5 * randn(1, e)
        s["w13"] = _expert_weights(gen, c["dtype"], e, 2 * i, h)
        s["w2"] = _expert_weights(gen, c["dtype"], e, h, i)
        s["residual"] = randn(t, h).to(BF16) if c["residual"] else None
        s["ids"] = torch.empty((t, top_k), dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty((t, top_k), dtype=F32, device=DEV)
        if c["routing"] == "ids":
            ids, w = _route(s["logits"], top_k, c["scoring"])
            s["ids"].copy_(ids)
            s["weights"].copy_(w)
            s["logits"] = None
        s["out"] = torch.empty((t, h), dtype=BF16, device=DEV)
        s["workspace"] = torch.empty(t * top_k * i, dtype=BF16, device=DEV)
        return s
    m, n, k = c["m"], c["n"], c["k"]
    a, b = randn(m, k), randn(n, k) / math.sqrt(k)
    if c["op"] == "linear" and c["dtype"] == "fp8":
        s["a"], s["b"] = _quantise(a, 1), _quantise(b, 128)
    else:
        s["a"], s["b"] = a.to(BF16), b.to(BF16)
    if c["op"] == "linear":
        s["bias"] = 0.2 * randn(n) if c["bias"] else None
        s["residual"] = randn(m, n).to(BF16) if c["residual"] else None
        s["out"] = torch.empty((m, n), dtype=F32 if c["out"] == "f32" else BF16, device=DEV)
        s["pre"] = torch.empty((m, n), dtype=BF16, device=DEV) if c["save"] else None
        return s
    s["dout"] = randn(m, n).to(BF16)
    s["pre"] = randn(m, n).to(BF16) if c["act"] != "none" else None
    s["da"] = torch.empty((m, k), dtype=BF16, device=DEV)
    s["db"] = torch.empty((n, k), dtype=BF16, device=DEV)
    s["dbias"] = torch.empty(n, dtype=F32, device=DEV) if c["bias"] else None
    return s


# ---- one pass -----------------------------------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    dg, c = _lib(), s["case"]
    if c["op"] == "linear":
        if c["dtype"] == "fp8":
            dg.gemm_fp8_nt_epilogue(s["a"], s["b"], s["out"], s["bias"], c["act"], s["residual"])
            return s["out"]
        dg.gemm_bf16_nt_epilogue(s["a"], s["b"], s["out"], s["bias"], c["act"], s["residual"], s["pre"])
        return [s["out"], s["pre"]] if c["save"] else s["out"]
    if c["op"] == "backward":
        dg.gemm_bf16_nt_epilogue_backward(s["dout"], s["a"], s["b"], s["pre"], c["act"], s["da"], s["db"], s["dbias"])
        return [s["da"], s["db"], s["dbias"]]
    moe = dg.moe_few_tokens_fp8 if c["dtype"] == "fp8" else dg.moe_few_tokens_bf16
    moe(s["x"], s["w13"], s["w2"], s["out"], s["ids"], s["weights"], logits=s["logits"], scoring=c["scoring"],
        residual=s["residual"], workspace=s["workspace"])
    return [s["out"], s["ids"], s["weights"]]


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


def _act_grad(x, act):
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (x + 0.044715 * x * x * x))
        return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)
    if act == "silu":
        g = torch.sigmoid(x)
        return g * (1 + x * (1 - g))
    return torch.ones_like(x)


def _values(q, s, rows):
    """fp32 values of FP8 codes [.., N, K] with a scale per `rows` rows and 128 columns."""
    k = q.shape[-1]
    return q.float() * s.repeat_interleave(rows, -2)[..., :q.shape[-2], :].repeat_interleave(128, -1)[..., :k]


def _route(logits, top_k, scoring):
    top, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    top, ids = top[:, :top_k], ids[:, :top_k]
    w = torch.exp(top - top[:, :1]) if scoring == "softmax" else torch.sigmoid(top)
    return ids.to(torch.int32), w / w.sum(-1, keepdim=True)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "moe":
        return _plain_moe(s)
    if c["op"] == "linear":
        if c["dtype"] == "fp8":
            a, b = _values(*s["a"], 1), _values(*s["b"], 128)
        else:
            a, b = s["a"].float(), s["b"].float()
        pre = a @ b.t()
        if c["bias"]:
            pre = pre + s["bias"]
        y = _act(pre, c["act"])
        if c["residual"]:
            y = y + s["residual"].float()
        y = y.to(s["out"].dtype)
        return [y, pre.to(BF16)] if c["save"] else y
    d = s["dout"].float()
    if c["act"] != "none":
        d = d * _act_grad(s["pre"].float(), c["act"])
    da = d @ s["b"].float()
    db = d.t() @ s["a"].float()
    return [da.to(BF16), db.to(BF16), d.sum(0) if c["bias"] else None]


def _pick(w, sel, dtype):
    """fp32 weights [S, N, K] of the experts `sel`."""
    if dtype == "bf16":
        return w[sel].float()
    q, sc = w
    return _values(q.view(torch.uint8)[sel].view(torch.float8_e4m3fn), sc[sel], 128)


def _plain_moe(s):
    c = s["case"]
    t, e, top_k = c["t"], c["e"], c["top_k"]
    x = s["x"].float()
    ids, w = (s["ids"], s["weights"]) if c["routing"] == "ids" else _route(s["logits"], top_k, c["scoring"])
    # the weights of every expert, or of the chosen ones where those are fewer
    if t * top_k >= e:
        sel = torch.arange(e, device=DEV)
        mix = torch.zeros((t, e), device=DEV).scatter_(1, ids.long(), w)
    else:
        sel = ids.reshape(-1).long()
        mix = (torch.eye(t, device=DEV)[:, :, None] * w[:, None, :]).transpose(0, 1).reshape(t, t * top_k)
    gate, up = torch.matmul(x, _pick(s["w13"], sel, c["dtype"]).transpose(1, 2)).chunk(2, -1)
    hid = gate * torch.sigmoid(gate) * up * mix.t()[:, :, None]
    y = torch.matmul(hid, _pick(s["w2"], sel, c["dtype"]).transpose(1, 2)).sum(0)
    if c["residual"]:
        y = y + s["residual"].float()
    return [y.to(BF16), ids, w]


# ---- 64 bits ------------------------------------------------------------------------------------------------------

def _f64(operand, rows):
    if isinstance(operand, torch.Tensor):
        return operand.double()
    q, s = operand
    v = q.to(torch.float32).double()
    for r in range(s.shape[0]):
        scale = torch.repeat_interleave(s[r].double(), 128)
        v[r * rows:(r + 1) * rows] *= scale
    return v


def _one_f64(operand, j):
    return _f64(operand[j] if isinstance(operand, torch.Tensor) else (operand[0][j], operand[1][j]), 128)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "moe":
        t, top_k = c["t"], c["top_k"]
        if c["routing"] == "ids":
            ids, w = s["ids"].long(), s["weights"].double()
        else:
            logits = s["logits"].double()
            ids = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :top_k]
            picked = torch.gather(logits, 1, ids)
            w = torch.softmax(picked, 1) if c["scoring"] == "softmax" else 1 / (1 + torch.exp(-picked))
            w = w / w.sum(1, keepdim=True)
        y = s["residual"].double() if c["residual"] else torch.zeros((t, c["h"]), dtype=torch.float64, device=DEV)
        for j in range(c["e"]):
            rows, slot = torch.nonzero(ids == j, as_tuple=True)
            if rows.numel() == 0:
                continue
            z = s["x"][rows].double() @ _one_f64(s["w13"], j).t()
            g, u = z[:, :c["i"]], z[:, c["i"]:]
            z = (g / (1 + torch.exp(-g)) * u) @ _one_f64(s["w2"], j).t()
            y[rows] += w[rows, slot][:, None] * z
        return [y, ids.to(torch.int32), w if c["routing"] == "logits" else None]
    if c["op"] == "linear":
        pre = _f64(s["a"], 1) @ _f64(s["b"], 128).t()
        if c["bias"]:
            pre += s["bias"].double()
        y = {"none": lambda v: v, "relu": torch.relu, "silu": torch.nn.functional.silu,
             "gelu": torch.nn.functional.gelu,
             "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[c["act"]](pre)
        if c["residual"]:
            y = y + s["residual"].double()
        return [y, pre] if c["save"] else y
    d = s["dout"].double()
    if c["act"] != "none":
        p = s["pre"].double()
        if c["act"] == "relu":
            d = torch.where(p > 0, d, torch.zeros_like(d))
        elif c["act"] == "silu":
            g = 1 / (1 + torch.exp(-p))
            d = d * (g + p * g * (1 - g))
        elif c["act"] == "gelu":
            d = d * (torch.special.ndtr(p) + p * torch.exp(-p * p / 2) / (2 * math.pi) ** 0.5)
        else:
            r = math.sqrt(2 / math.pi)
            u = r * (p + 0.044715 * p ** 3)
            sech2 = 1 / torch.cosh(u) ** 2
            d = d * (0.5 * (1 + torch.tanh(u)) + 0.5 * p * sech2 * r * (1 + 0.134145 * p ** 2))
    return [d @ s["b"].double(), d.t() @ s["a"].double(), d.sum(0) if c["bias"] else None]


# ---- what a pass cannot do without --------------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "moe":
        t, e, k, h, i = c["t"], c["e"], c["top_k"], c["h"], c["i"]
        each = 3 * i * h
        each = each * 2 if c["dtype"] == "bf16" else each + each // (128 * 128) * 4
        # experts that at least one token chooses, were the choices even
        chosen = e * (1 - (1 - k / e) ** t)
        return {"bytes": chosen * each + 2 * t * h * (2 + c["residual"]) + 8 * t * k
                + (4 * t * e if c["routing"] == "logits" else 0), "flops": 6 * t * k * h * i}
    m, n, k = c["m"], c["n"], c["k"]
    if c["op"] == "linear":
        if c["dtype"] == "fp8":
            size = m * k + n * k + 4 * (m * (k // 128) + -(-n // 128) * (k // 128))
        else:
            size = 2 * (m * k + n * k)
        size += m * n * ((4 if c["out"] == "f32" else 2) + 2 * c["residual"] + 2 * c["save"]) + 4 * n * c["bias"]
        return {"bytes": size, "flops": 2 * m * n * k}
    return {"bytes": 2 * (m * n * (1 if c["act"] == "none" else 2) + 2 * m * k + 2 * n * k) + 4 * n * c["bias"],
            "flops": 4 * m * n * k}
