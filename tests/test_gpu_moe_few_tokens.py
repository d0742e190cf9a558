"""The few-token MoE layer on the GPU against the formula in 64 bits.

Tolerance (before the first run).  x and the weights are exact in the
products; the kernel rounds each weighted hidden value to bf16 (relative 2^-9)
and the output once more (2^-9 of itself).  Per output, with
c = |w2| . |w h| the sum of absolute products,
    |y - ref| <= 2^-9 c + 2^-8 |ref| + (fp32 sums and silu) 2^-16 c' ,
where c' also takes the absolute products of the first layer through the
second; 2^-16 covers sums of up to 2^7 blocks with MFMA rounding.  The worst
case of 2^-9 c is never met by random roundings, so wrong columns, experts or
weights stand far outside it (they are O(c))."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.parity import say

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_x128_amd as m
    return m


def make(t, e, k, h, i, fp8, seed):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)
    d = dict(x=rn(t, h).to(BF16), logits=rn(t, e), residual=rn(t, h).to(BF16))
    for name, n, kk in (("w13", 2 * i, h), ("w2", h, i)):
        w = rn(e, n, kk) / kk ** 0.5
        if fp8:
            s = 2.0 ** torch.randint(-10, -6, (e, n // 128, kk // 128), generator=g).float() * (1 + 0.3 * torch.rand(
                (e, n // 128, kk // 128), generator=g))
            sc = s.repeat_interleave(128, 1).repeat_interleave(128, 2)
            q = (w / sc).clamp(-448, 448).to(torch.float8_e4m3fn)
            d[name] = (q.cuda(), s.cuda())
            d[name + "_64"] = q.float().double() * sc.double()
        else:
            d[name] = w.to(BF16).cuda()
            d[name + "_64"] = d[name].cpu().double()
    return d


def reference(d, ids, w, residual):
    """(y, bound) in 64 bits; ids outside the experts drop out."""
    x = d["x"].double()
    t, h = x.shape
    w13, w2 = d["w13_64"], d["w2_64"]
    i = w2.shape[2]
    y = torch.zeros(t, h, dtype=torch.float64)
    c = torch.zeros_like(y)
    for r in range(t):
        for j in range(ids.shape[1]):
            e = int(ids[r, j])
            if not 0 <= e < w13.shape[0]:
                continue
            z = w13[e] @ x[r]
            za = w13[e].abs() @ x[r].abs()
            g, u = z[:i], z[i:]
            hid = g / (1 + torch.exp(-g)) * u * float(w[r, j])
            # the first layer's fp32 sums: |d(silu(g) u)| <= 1.1 |dg| |u| + |g| |du|
            err = 2.0 ** -16 * abs(float(w[r, j])) * (1.1 * za[:i] * u.abs() + g.abs() * za[i:])
            y[r] += w2[e] @ hid
            c[r] += w2[e].abs() @ (2.0 ** -9 * hid.abs() + 2.0 ** -16 * hid.abs() + err)
    if residual:
        y = y + d["residual"].double()
    return y, c + 2.0 ** -8 * y.abs() + 1e-30


def topk_reference(logits, k, scoring, renormalize, scale):
    """Top-k with ties to the lowest index, -inf never chosen, in 64 bits."""
    t, e = logits.shape
    ids = np.full((t, k), -1, np.int64)
    w = np.zeros((t, k))
    for r in range(t):
        l = logits[r].double().numpy()
        order = sorted((j for j in range(e) if l[j] != -np.inf), key=lambda j: (-l[j], j))[:k]
        if not order:
            continue
        v = l[order]
        p = np.exp(v - v[0]) if scoring == "softmax" else 1 / (1 + np.exp(-v))
        if renormalize:
            p = p / p.sum()
        elif scoring == "softmax":
            p = p / np.exp(l - v[0]).sum()
        ids[r, :len(order)] = order
        w[r, :len(order)] = p * scale
    return ids, w


def call(dg, d, fp8, t, k, ids=None, weights=None, residual=True, **kw):
    h = d["x"].shape[1]
    out = torch.full((t, h), -1, dtype=torch.int16, device="cuda").view(BF16)
    routed = ids is None
    ids = torch.full((t, k), -7, dtype=torch.int32, device="cuda") if routed else ids.cuda()
    weights = torch.full((t, k), float("nan"), device="cuda") if routed else weights.cuda()
    fn = dg.moe_few_tokens_fp8 if fp8 else dg.moe_few_tokens_bf16
    fn(d["x"].cuda(), d["w13"], d["w2"], out, ids, weights, logits=d["logits"].cuda() if routed else None,
       residual=d["residual"].cuda() if residual else None, **kw)
    torch.cuda.synchronize()
    return out, ids, weights


def check(y, ref, bound, what):
    err = (y.double().cpu() - ref).abs()
    assert torch.isfinite(err).all(), what
    worst = (err / bound).max().item()
    assert worst <= 1, f"{what}: {worst:.3g} times the bound"
    rel = (err.norm() / ref.norm()).item()
    # 2^-9 per rounding, two of them, at most uniform: 2^-9 * sqrt(2) / sqrt(3) of the norm is what is expected
    assert rel <= 2.0 ** -8, f"{what}: relative error {rel:.3g}"


SHAPES = [(1, 4, 1, 128, 128), (1, 8, 2, 1024, 512), (3, 5, 5, 640, 256), (16, 7, 3, 384, 384), (17, 16, 4, 256, 128),
          (64, 3, 2, 512, 256), (33, 40, 16, 128, 256), (64, 512, 16, 128, 128), (50, 1, 1, 1152, 128),
          (2, 65, 8, 256, 1152)]


@pytest.mark.parametrize("t,e,k,h,i", SHAPES)
@pytest.mark.parametrize("fp8", [True, False])
def test_routed(dg, t, e, k, h, i, fp8):
    say(f"moe t={t} e={e} k={k} h={h} i={i} fp8={fp8}")
    d = make(t, e, k, h, i, fp8, 100 * t + e)
    scoring = "softmax" if (t + e) % 2 else "sigmoid"
    out, ids, w = call(dg, d, fp8, t, k, scoring=scoring, renormalize=t % 3 != 0, scale=1.5)
    rid, rw = topk_reference(d["logits"], k, scoring, t % 3 != 0, 1.5)
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert np.abs(w.cpu().numpy() - rw).max() <= 2.0 ** -20 * 1.5  # a few fp32 roundings of values up to 1.5
    ref, bound = reference(d, rid, w.cpu(), True)
    check(out, ref, bound, f"routed {t} {e} {k} {h} {i} {fp8}")
    again = call(dg, d, fp8, t, k, scoring=scoring, renormalize=t % 3 != 0, scale=1.5)[0]
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)), "not deterministic"


@pytest.mark.parametrize("fp8", [True, False])
def test_given_ids_out_of_range_and_repeated(dg, fp8):
    t, e, k, h, i = 20, 6, 4, 256, 256
    say("moe given ids")
    d = make(t, e, k, h, i, fp8, 5)
    g = torch.Generator().manual_seed(9)
    ids = torch.randint(-1, e + 2, (t, k), generator=g).to(torch.int32)
    ids[0] = -1                                                  # a token without experts
    ids[1] = torch.tensor([2, 2, 2, 2])
    ids[2] = torch.tensor([3, 1, 3, 1])
    ids[3] = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, 5])
    w = torch.randn(t, k, generator=g)
    for residual in (True, False):
        out, ids2, w2 = call(dg, d, fp8, t, k, ids=ids, weights=w, residual=residual)
        assert torch.equal(ids2.cpu(), ids) and torch.equal(w2.cpu(), w)   # inputs stay
        ref, bound = reference(d, ids, w, residual)
        check(out[1:], ref[1:], bound[1:], f"given ids residual={residual}")
        want = d["residual"][0].float() if residual else torch.zeros(h)
        assert torch.equal(out[0].float().cpu(), want)


def test_ties_infinities_and_empty_rows(dg):
    t, e, k, h, i = 6, 130, 4, 128, 128
    say("moe ties")
    d = make(t, e, k, h, i, True, 6)
    l = torch.full((t, e), float("-inf"))
    l[0, :] = 0.25                                # every expert alike: 0, 1, 2, 3
    l[1, [129, 64, 63]] = torch.tensor([1.0, 1.0, 2.0])
    l[2, 77] = -3e38                              # one expert, the type's lowest values
    l[3, :] = float("-inf")                       # nothing left
    l[4, [5, 70]] = torch.tensor([0.0, -0.0])     # equal
    l[4, 100] = -1.0
    l[5, 0], l[5, 128] = torch.finfo(F32).min, torch.finfo(F32).max
    d["logits"] = l
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            out, ids, w = call(dg, d, True, t, k, scoring=scoring, renormalize=renorm)
            rid, rw = topk_reference(l, k, scoring, renorm, 1.0)
            assert np.array_equal(ids.cpu().numpy(), rid)
            got = w.cpu().numpy()
            ok = np.abs(got - rw) <= 2.0 ** -20
            if scoring == "sigmoid" and renorm:
                ok[2] = got[2] == 0               # every sigmoid underflows: defined as 0
                rw[2] = 0
            assert ok.all(), (scoring, renorm, got, rw)
            ref, bound = reference(d, rid, torch.from_numpy(got), True)
            rows = [0, 1, 2, 4, 5]
            check(out[rows], ref[rows], bound[rows], f"{scoring} {renorm}")
            assert torch.equal(out[3].float().cpu(), d["residual"][3].float())


@pytest.mark.parametrize("fp8", [True, False])
def test_nan_stays_in_its_row(dg, fp8):
    """A NaN or infinity in one token, in one token's logits, or in the weights
    of one expert reaches no token that has no part in it."""
    t, e, k, h, i = 18, 8, 2, 256, 256
    say("moe nan")
    d = make(t, e, k, h, i, fp8, 7)
    clean, ids, _ = call(dg, d, fp8, t, k)
    d2 = dict(d, x=d["x"].clone(), logits=d["logits"].clone())
    d2["x"][4, 17] = float("nan")
    d2["x"][9, 3] = float("inf")
    d2["logits"][12, 5] = float("nan")
    out, ids2, w2 = call(dg, d2, fp8, t, k)
    keep = [r for r in range(t) if r not in (4, 9, 12)]
    assert torch.equal(out[keep].view(torch.int16), clean[keep].view(torch.int16))
    assert torch.isnan(out[4].float()).all() and torch.isnan(out[12].float()).all()
    assert ids2[12, 0].item() == 5 and torch.isnan(w2[12]).all()
    # NaN weights of expert 3
    bad = int(ids[0, 0])
    if fp8:
        q, s = d["w2"]
        q = q.clone()
        q.view(torch.uint8)[bad, 5] = 0x7F
        d3 = dict(d, w2=(q, s))
    else:
        w = d["w2"].clone()
        w[bad, 5] = float("nan")
        d3 = dict(d, w2=w)
    out, _, _ = call(dg, d3, fp8, t, k)
    hit = (ids == bad).any(1).cpu()
    assert torch.isnan(out[:, 5].float().cpu()[hit]).all()
    assert torch.equal(out[~hit.to(out.device)].view(torch.int16), clean[~hit.to(out.device)].view(torch.int16))


def test_row_does_not_depend_on_the_others(dg):
    t, e, k, h, i = 40, 12, 3, 512, 256
    say("moe independence")
    d = make(t, e, k, h, i, True, 8)
    out, _, _ = call(dg, d, True, t, k)
    for r in (0, 17, 39):
        one = dict(d, x=d["x"][r:r + 1], logits=d["logits"][r:r + 1], residual=d["residual"][r:r + 1])
        got, _, _ = call(dg, one, True, 1, k)
        # the waves meet in another order when the units are dealt out differently: fp32 roundings only
        ref = out[r].double().cpu()
        assert ((got[0].double().cpu() - ref).abs() <= 2.0 ** -7 * ref.abs() + 2.0 ** -14 * ref.abs().max()).all()


def test_side_stream_and_graph(dg):
    t, e, k, h, i = 5, 8, 2, 512, 256
    say("moe graph")
    d = make(t, e, k, h, i, True, 11)
    x, lg = d["x"].cuda(), d["logits"].cuda()
    out = torch.empty((t, h), dtype=BF16, device="cuda")
    ids = torch.empty((t, k), dtype=torch.int32, device="cuda")
    w = torch.empty((t, k), device="cuda")
    ws = torch.empty(t * k * i, dtype=BF16, device="cuda")
    run = lambda: dg.moe_few_tokens_fp8(x, d["w13"], d["w2"], out, ids, w, logits=lg, workspace=ws)
    run()
    torch.cuda.synchronize()
    want = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    gen = torch.Generator().manual_seed(3)
    for _ in range(4):
        x.copy_(torch.randn(t, h, generator=gen))
        lg.copy_(torch.randn(t, e, generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        run()
        torch.cuda.synchronize()
        assert torch.equal(got, out)


def test_refusals(dg):
    d = make(2, 4, 2, 256, 128, True, 1)
    x = d["x"].cuda()
    out = torch.empty_like(x)
    ids = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    w = torch.zeros((2, 2), device="cuda")
    ok = dict(x=x, w13=d["w13"], w2=d["w2"], out=out, ids=ids, weights=w)

    def bad(exc, **kw):
        with pytest.raises(exc):
            dg.moe_few_tokens_fp8(**{**ok, **kw})

    bad(TypeError, x=x.float())
    bad(TypeError, ids=ids.long())
    bad(TypeError, w2=(d["w2"][0], d["w2"][1].double()))
    bad(ValueError, out=out[:1])
    bad(ValueError, w2=(d["w2"][0][:3], d["w2"][1]))
    bad(ValueError, x=x.cpu())
    bad(ValueError, x=torch.empty((256, 2), dtype=BF16, device="cuda").t())
    bad(ValueError, scoring="top")
    bad(ValueError, workspace=torch.empty(8, dtype=BF16, device="cuda"))
    bad(ValueError, logits=torch.zeros((2, 5), device="cuda"))
    big = torch.zeros((65, 256), dtype=BF16, device="cuda")
    with pytest.raises(dg.DGError):
        dg.moe_few_tokens_fp8(big, d["w13"], d["w2"], torch.empty_like(big),
                              torch.zeros((65, 2), dtype=torch.int32, device="cuda"), torch.zeros((65, 2), device="cuda"))
