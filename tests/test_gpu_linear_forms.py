"""The forms of the linear layer's kernels that large shapes use, each by itself:
the backward products with K split.  The launch log names the form that ran.

Tolerances as in tests/test_gpu_linear.py."""
from __future__ import annotations

import os
import re

import pytest

from tests.parity import say
from tests.test_gpu_linear import backward_case

pytestmark = pytest.mark.gpu

# tiles of the two products in one launch, and the workgroups that share a compute unit
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


def fields(line):
    return {k: int(v) for k, v in re.findall(r"(\w+)=(\d+)", line)}


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
