"""The gated block's cuts: the host's form of them against the library's
workspaces, and the GPU tests' sizes against the kinds of launch there are."""
import math
import random

import pytest

import mlp_tiles
import vision_image_preprocessing_amd as V

pytest.importorskip("torch")


def _sizes():
    """Every (rows, d, h) of a GPU test that checks all outputs and gradients."""
    import test_gpu_mlp as gpu

    for test in (gpu.test_sizes, gpu.test_large, gpu.test_tiles_of_256, gpu.test_whole_tiles_next_to_parts):
        (sizes,) = [m.args[1] for m in test.pytestmark if m.name == "parametrize" and m.args[0] == "rows,d,h"]
        yield from sizes


def test_workspaces_are_those_of_the_cuts():
    rng = random.Random(1)
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    for size in [*_sizes(), *((log(1, 200000), log(1, 6000), log(1, 8000)) for _ in range(2000))]:
        got = V.gated_mlp_workspace_bytes(*size), V.gated_mlp_backward_workspace_bytes(*size)
        assert got == mlp_tiles.workspaces(*size), size


def test_gpu_sizes_reach_every_kind_of_launch():
    """Each kernel's tiles of 64, 128 and 256: whole, all in parts, and both in
    one launch (gate, up and dh are never in parts)."""
    reached = {(name, cut[0], mlp_tiles.kind(cut)) for size in _sizes() for name, cut in mlp_tiles.cuts(*size).items()}
    whole = {(name, tile, "whole") for name in ("gate", "gate saved", "dhidden") for tile in (64, 128, 256)}
    every = {(name, tile, kind) for name in ("down", "dx", "dweights") for tile in (64, 128, 256) for kind in ("whole", "parts", "mixed")}
    assert reached == whole | every
