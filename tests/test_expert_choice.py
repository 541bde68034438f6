"""The calls of tests/expert_kernels.py run the kernels they name, and
together every kernel of the expert products that a call can reach: the rules
that choose are the library's, compiled for the host."""
import shutil

import pytest

from expert_kernels import GROUPED, WGRAD, Chooser, large_positions

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ needed")

TILES = ["any layout", "large", "128 x 128", "64 x 256", "64 x 64", "16 rows"]


@pytest.fixture(scope="module")
def chooser(tmp_path_factory):
    return Chooser(str(tmp_path_factory.mktemp("choice")))


def run_by(chooser, c, K):
    got = {chooser.grouped(t, o, c["counts"], K, c["N"], trans)
           for t in ("f16", "bf16") for o in (t, "f32") for trans in (False, True)}
    return got | {chooser.fp8(o, c["counts"], K, c["N"]) for o in ("f32", "bf16", "f16")}


@pytest.mark.parametrize("name", list(GROUPED))
def test_a_call_runs_the_kernel_it_names(chooser, name):
    c = GROUPED[name]
    for K in c["K"]:
        for got in run_by(chooser, c, K):
            want = c["kernel"]
            if "exact" in got and want == "large":
                want = "128 x 128"
            assert want in got, (K, got)
    if c["kernel"] == "large":
        whole, cut, half = large_positions(c["counts"], c["N"])
        assert (cut > 0) == c["cut"], (whole, cut, half)
        assert -(-(whole + 2 * cut + half) // 256) == c["rounds"], (whole, cut, half)


@pytest.mark.parametrize("name", list(WGRAD))
def test_a_weight_gradient_runs_the_kernel_it_names(chooser, name):
    c = WGRAD[name]
    for t in ("f16", "bf16"):
        for out in (t, "f32"):
            got = chooser.wgrad(t, out, c["counts"], c["K"], c["N"])
            assert got == f"{t} weight gradient {c['kernel']}", got


def test_every_kernel_is_run_by_a_call(chooser):
    got = set()
    for c in GROUPED.values():
        for K in c["K"]:
            got |= run_by(chooser, c, K)
    for c in WGRAD.values():
        got |= {chooser.wgrad(t, o, c["counts"], c["K"], c["N"]) for t in ("f16", "bf16") for o in (t, "f32")}
    want = {f"{t} [K, N] {v}" for t in ("f16", "bf16") for v in TILES + ["32 rows"]}
    want |= {f"{t} [N, K] {v}" for t in ("f16", "bf16") for v in TILES + ["32 rows narrow", "32 rows wide"]}
    for how in ("native", "exact"):
        want |= {f"fp8 {how} {v}" for v in TILES[:-1] if (how, v) != ("exact", "large")}
        want |= {f"fp8 {how} {v} {s}" for v in ("16 rows", "32 rows") for s in ("narrow", "wide")}
    want |= {f"{t} weight gradient {v}" for t in ("f16", "bf16")
             for v in ("any layout", "large", "large past the cache", "128 x 128")}
    assert got == want


def test_large_tiles_of_one_matrix_are_counted(chooser):
    """The count by hand: 600 rows are two whole tiles of 256 and a half one,
    8200 columns 33 tiles; all in one round, so the whole ones are cut."""
    assert large_positions([600], 8200) == (0, 66, 33)
    assert large_positions([1024], 4096) == (0, 64, 0)
    assert large_positions([4900], 8200) == (627, 0, 33)
