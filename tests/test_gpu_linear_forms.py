"""The forms of the linear layer's kernels that large shapes use, each by itself:
the 32-column form of the few-row kernel (N above 16 columns per compute unit),
every FP8 tile with every epilogue, several tiles per workgroup, the backward
pair of products with several tiles per workgroup, and the single products with
K split.  The launch log names the form that ran.

Tolerances as in tests/test_gpu_linear.py."""
from __future__ import annotations

import os
import re

import pytest
import torch

from tests.parity import say
from tests.test_gpu_linear import ACTS, BF16, F32, backward_case, forward_case

pytestmark = pytest.mark.gpu

FP8_TILES = ["256x256x2x4", "192x256x2x4", "256x128x2x2", "128x128x2x2", "128x64x2x2", "64x128x1x4", "64x64x1x4",
             "64x32x2x2"]
FP8_TILES_F32 = ["128x128x2x2", "128x64x2x2", "64x128x1x4", "64x64x1x4", "64x32x2x2"]
BF16_TILES = ["256x256x2x4x1", "256x128x4x2x1", *(f"{t}x{w}" for t in ("128x128x2x2", "64x128x2x2", "64x64x2x2") for w in (1, 2))]
# tiles of the backward pair, and the workgroups that share a compute unit
PAIR_TILES = {"256x256x2x4": 1, "256x128x4x2": 1, "128x128x2x2": 2, "64x128x2x2": 2, "64x64x2x2": 2}


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_x128_amd as m
    return m


@pytest.fixture
def log(capfd):
    """Switches of the library, and what it logged since the last look."""
    def switches(tile=None, splits=None):
        for k, v in (("DG_FORCE_TILE", tile), ("DG_FORCE_SPLITS", splits), ("DG_LOG", 1)):
            os.environ.pop(k, None)
            if v is not None:
                os.environ[k] = str(v)
        capfd.readouterr()
    switches.read = lambda: capfd.readouterr().err
    yield switches
    for k in ("DG_FORCE_TILE", "DG_FORCE_SPLITS", "DG_LOG"):
        os.environ.pop(k, None)


def cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


def fields(line):
    return {k: int(v) for k, v in re.findall(r"(\w+)=(\d+)", line)}


@pytest.mark.parametrize("m", [1, 5, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("n,k", [(5001, 72), (7168, 1032), (4352, 264)])
def test_few_rows_wide_bf16(dg, log, m, n, k):
    say(f"few rows wide bf16 {m}x{n}x{k}")
    assert n > 16 * cus(), "not the 32-column form"
    for v in range(2):
        log()
        forward_case(dg, m, n, k, ACTS[(m + v) % 5], bias=(F32, BF16)[v], residual=v == 1, pre=v == 0,
                     out=F32 if (m + v) % 3 == 0 else BF16, pad=8 * v)
        assert "linear layout" not in log.read(), "ran on tiles"


@pytest.mark.parametrize("m", [1, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("n,k", [(5001, 128), (7168, 1152), (4352, 384)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_few_rows_wide_fp8(dg, log, m, n, k, out):
    say(f"few rows wide fp8 {m}x{n}x{k} {out}")
    assert n > 16 * cus(), "not the 32-column form"
    log()
    forward_case(dg, m, n, k, ACTS[m % 5], bias=F32, residual=m % 2 == 1, pre=m % 2 == 0, out=out, fp8=True)
    assert "kind=" not in log.read(), "ran on tiles"


# aligned rows, odd ones, rows of 4 and of 8 columns with a stride that is neither
SIZES = [(300, 520, 256), (257, 391, 384), (130, 132, 640), (70, 264, 1152)]


@pytest.mark.parametrize("tile", FP8_TILES)
@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("residual,pre", [(False, False), (True, False), (False, True), (True, True)])
def test_fp8_tiles(dg, log, tile, m, n, k, residual, pre):
    say(f"fp8 tile {tile} {m}x{n}x{k} res={residual} pre={pre}")
    bm, bn = (int(x) for x in tile.split("x")[:2])
    for splits in (1, 3):
        for pad in (0, 8, 3):
            log(tile, splits)
            forward_case(dg, m, n, k, ACTS[(m + pad + splits) % 5], bias=F32 if pad else BF16, residual=residual, pre=pre,
                         fp8=True, pad=pad)
            err = log.read()
            assert f"tile {bm}x{bn} " in err and f"splits={min(splits, k // 128)}" in err, err


@pytest.mark.parametrize("tile", FP8_TILES_F32)
@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("residual,pre", [(False, False), (True, True)])
def test_fp8_tiles_with_fp32_result(dg, log, tile, m, n, k, residual, pre):
    say(f"fp8 tile {tile} fp32 {m}x{n}x{k} res={residual} pre={pre}")
    bm, bn = (int(x) for x in tile.split("x")[:2])
    for splits in (1, 3):
        for pad in (0, 8, 3):
            log(tile, splits)
            forward_case(dg, m, n, k, ACTS[(m + pad + splits) % 5], bias=F32, residual=residual, pre=pre, out=F32,
                         fp8=True, pad=pad)
            err = log.read()
            assert f"tile {bm}x{bn} " in err and f"splits={min(splits, k // 128)}" in err, err


def exact_case(dg, m, n, k, residual, pre, out, pad=0):
    """Small integers with power-of-two scales: every product, sum and rounding
    before the results' own is exact whatever the order, so the results are the
    formula's bit for bit."""
    g = torch.Generator(device="cuda").manual_seed(3 * m + n + k)
    ints = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g, device="cuda").float()
    a, b = ints(-2, 2, m, k), ints(-2, 2, n, k)
    sa, sb = torch.exp2(ints(-1, 1, m, k // 128)), torch.exp2(ints(-1, 1, (n + 127) // 128, k // 128))
    bias, res = ints(-40, 40, n) / 4, (ints(-200, 200, m, n) / 4).to(BF16) if residual else None
    o = torch.full((m, n + pad), float("nan"), dtype=out, device="cuda")
    p = torch.full((m, n + pad), float("nan"), dtype=BF16, device="cuda") if pre else None
    dg.gemm_fp8_nt_epilogue((a.to(torch.float8_e4m3fn), sa), (b.to(torch.float8_e4m3fn), sb), o[:, :n], bias, "relu", res,
                            p[:, :n] if pre else None)
    # (fp32 products of these values are exact too: below 2^24 quarters)
    z = (a * sa.repeat_interleave(128, 1)) @ (b * sb.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)).t() + bias
    want = torch.relu(z) + (res.float() if residual else 0)
    assert torch.equal(o[:, :n], want.to(out)), f"{(o[:, :n] != want.to(out)).sum().item()} outputs differ"
    assert not pre or torch.equal(p[:, :n], z.to(BF16)), "pre differs"
    assert torch.isnan(o[:, n:].float()).all() and (not pre or torch.isnan(p[:, n:].float()).all())


@pytest.mark.parametrize("tile", FP8_TILES)
@pytest.mark.parametrize("odd", [0, 5])
@pytest.mark.parametrize("residual,pre", [(False, False), (True, False), (False, True), (True, True)])
def test_fp8_many_tiles_per_workgroup(dg, log, tile, odd, residual, pre):
    """More tiles than workgroups, with K of one block (shorter than the ring) and of several."""
    say(f"fp8 many tiles {tile} odd={odd} res={residual} pre={pre}")
    bm, bn = (int(x) for x in tile.split("x")[:2])
    for k in (128, 640):
        log(tile)
        exact_case(dg, 24 * bm - 7, 24 * bn - odd, k, residual, pre, BF16, pad=8 if k == 640 else 0)
        f = fields(log.read())
        assert f["tiles"] == 24 * 24 and f["grid"] < f["tiles"] and f["splits"] == 1, f


@pytest.mark.parametrize("tile", FP8_TILES_F32)
@pytest.mark.parametrize("odd", [0, 5])
def test_fp8_with_fp32_result_many_tiles_per_workgroup(dg, log, tile, odd):
    say(f"fp8 fp32 many tiles {tile} odd={odd}")
    bm, bn = (int(x) for x in tile.split("x")[:2])
    log(tile)
    exact_case(dg, 24 * bm - 7, 24 * bn - odd, 384, True, odd == 0, F32)
    f = fields(log.read())
    assert f["grid"] < f["tiles"], f


def exact_bf16(dg, m, n, k, residual, pre, out, pad):
    g = torch.Generator(device="cuda").manual_seed(5 * m + n + k)
    ints = lambda lim, *s: torch.randint(-lim, lim + 1, s, generator=g, device="cuda").float()
    a, b, bias = ints(2, m, k), ints(2, n, k), ints(40, n) / 4
    res = (ints(200, m, n + pad) / 4).to(BF16)[:, :n] if residual else None
    o = torch.full((m, n + pad), float("nan"), dtype=out, device="cuda")
    p = torch.full((m, n + pad), float("nan"), dtype=BF16, device="cuda") if pre else None
    dg.gemm_bf16_nt_epilogue(a.to(BF16), b.to(BF16), o[:, :n], bias, "relu", res, p[:, :n] if pre else None)
    z = a @ b.t() + bias
    want = torch.relu(z) + (res.float() if residual else 0)
    assert torch.equal(o[:, :n], want.to(out)), f"{(o[:, :n] != want.to(out)).sum().item()} outputs differ"
    assert not pre or torch.equal(p[:, :n], z.to(BF16)), "pre differs"
    assert torch.isnan(o[:, n:].float()).all() and (not pre or torch.isnan(p[:, n:].float()).all())


@pytest.mark.parametrize("tile", BF16_TILES)
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("residual,pre", [(False, False), (True, False), (False, True), (True, True)])
def test_bf16_many_tiles_per_workgroup(dg, log, tile, out, residual, pre):
    """From K of a part of one block (shorter than the ring) to several blocks."""
    say(f"bf16 many tiles {tile} {out} res={residual} pre={pre}")
    bm, bn = (int(x) for x in tile.split("x")[:2])
    for k in (8, 136, 520):
        for odd, pad in ((0, 8), (5, 0)):
            log(tile)
            exact_bf16(dg, 24 * bm - 7, 24 * bn - odd, k, residual, pre, out, pad)
            f = fields(log.read())
            assert f["grid"] < 24 * 24 and f["splits"] == 1, f


@pytest.mark.parametrize("tile", BF16_TILES)
def test_backward_products_many_tiles_per_workgroup(dg, log, tile):
    """Either product by itself: small integers, so that the gradients are the formula's bit for bit."""
    bm, bn = (int(x) for x in tile.split("x")[:2])
    g = torch.Generator(device="cuda").manual_seed(6)
    ints = lambda lim, *s: torch.randint(-lim, lim + 1, s, generator=g, device="cuda").float()
    for odd in (0, 5):
        say(f"backward products many tiles {tile} odd={odd}")
        k = 24 * bn - 8
        for m, n in ((24 * bm - 3, 72 - odd), (72 - odd, 24 * bm - odd)):
            dc, a, b, pre = ints(2, m, n), ints(2, m, k), ints(2, n, k), ints(1, m, n)
            d = torch.where(pre > 0, dc, torch.zeros_like(dc))
            log(tile, 1)
            if n < m:
                got, want = torch.full((m, k), float("nan"), dtype=BF16, device="cuda"), d @ b
                dg.gemm_bf16_nt_epilogue_backward(dc.to(BF16), a.to(BF16), b.to(BF16), pre.to(BF16), "relu", da=got)
            else:
                got, want = torch.full((n, k), float("nan"), dtype=BF16, device="cuda"), d.t() @ a
                dg.gemm_bf16_nt_epilogue_backward(dc.to(BF16), a.to(BF16), b.to(BF16), pre.to(BF16), "relu", db=got)
            assert torch.equal(got, want.to(BF16)), (got != want.to(BF16)).sum().item()
            f = fields(log.read())
            assert f["grid"] < 24 * 24, f


@pytest.mark.parametrize("tile", PAIR_TILES)
@pytest.mark.parametrize("odd", [0, 5])
def test_backward_pair_many_tiles_per_workgroup(dg, log, tile, odd):
    bm, bn = (int(x) for x in tile.split("x")[:2])
    # more tiles in either product than workgroups of the whole launch (256 compute units)
    across = 12 * PAIR_TILES[tile]
    m, n, k = 24 * bm - 3, 24 * bm - odd, across * bn - 8
    say(f"backward pair {tile} {m}x{n}x{k}")
    log(tile)
    backward_case(dg, m, n, k, "gelu")
    err = log.read()
    assert "linear backward" in err, err
    f = fields(err)
    assert f["first"] < 24 * across and f["grid"] - f["first"] < 24 * across, err


@pytest.mark.parametrize("tile", PAIR_TILES)
@pytest.mark.parametrize("splits", [2, 3])
def test_backward_single_products_with_k_split(dg, log, tile, splits):
    say(f"backward single products {tile} splits={splits}")
    for which, layout in (((True, False, True), 1), ((False, True, False), 2)):
        for m, n, k in ((300, 260, 392), (713, 333, 264)):
            log(tile, splits)
            backward_case(dg, m, n, k, "silu", which=which)
            f = fields(log.read())
            assert f["layout"] == layout and f["splits"] == splits, f


@pytest.mark.parametrize("tile", PAIR_TILES)
def test_backward_both_products_with_k_split(dg, log, tile):
    """Forced splits hold for a call that computes both gradients too."""
    say(f"backward both products split {tile}")
    for m, n, k in ((300, 260, 392), (713, 333, 264)):
        log(tile, 3)
        backward_case(dg, m, n, k, "silu")
        lines = [fields(x) for x in log.read().splitlines() if "linear layout" in x]
        assert [x["layout"] for x in lines] == [1, 2] and all(x["splits"] == 3 for x in lines), lines


def test_backward_two_launches_by_choice(dg, log):
    """Few rows and long K: da's K split over workgroups, without a switch."""
    say("backward 45x6920x2520")
    log()
    backward_case(dg, 45, 6920, 2520, "gelu")
    lines = [fields(x) for x in log.read().splitlines() if "linear layout" in x]
    assert [x["layout"] for x in lines] == [1, 2] and lines[0]["splits"] > 1, lines


@pytest.mark.parametrize("n", [4096, 4097])
def test_backward_in_chunks_of_64_rows(dg, n):
    say(f"backward chunks of 64 rows n={n}")
    backward_case(dg, 2051, n, 64, "gelu_tanh")


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("side", ["a", "b"])
def test_every_fp8_code(dg, out, side):
    """Each of the 256 codes by itself times one: its value, and NaN for the two
    NaN codes, whichever operand holds it, by the few-row kernel and on tiles."""
    say(f"fp8 every code in {side} {out}")
    k = 256
    codes = torch.zeros((256, k), dtype=torch.uint8, device="cuda")
    i = torch.arange(256, device="cuda")
    codes[i, (7 * i) % k] = i.to(torch.uint8)
    codes = codes.view(torch.float8_e4m3fn)
    value = i.to(torch.uint8).view(torch.float8_e4m3fn).float()
    assert torch.isnan(value).sum() == 2
    one = lambda r: torch.ones((r, k), device="cuda").to(torch.float8_e4m3fn)
    ones = lambda r: torch.ones((r, k // 128), device="cuda")
    for m in ((16, 64, 256) if side == "a" else (3, 40, 100)):
        for first in range(0, 256 if side == "a" else 1, m if side == "a" else 256):
            n = 70 if side == "a" else 256
            a, b = (codes[first:first + m], one(n)) if side == "a" else (one(m), codes)
            o = torch.empty((m, n), dtype=out, device="cuda")
            dg.gemm_fp8_nt_epilogue((a, ones(m)), (b, ones((n + 127) // 128)), o)
            want = (value[first:first + m, None].expand(m, n) if side == "a" else value[None].expand(m, n)).to(out)
            nan = torch.isnan(want)
            assert torch.equal(torch.isnan(o), nan) and torch.equal(o[~nan], want[~nan]), (m, first)
