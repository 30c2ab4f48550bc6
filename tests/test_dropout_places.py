"""Masks of several places over several steps. A mask depends on seed and offset + subsequence: a step
of n places has to count the offset up by n."""
import os

import numpy as np
import pytest
import torch

from tests import _block64 as blk

N, P, SEED = 1 << 12, 0.5, 2026


def masks(steps, places, stride):
    return [[blk.kept(0, N, P, SEED, 7 + stride * t, i).tobytes() for i in range(places)] for t in range(steps)]


@pytest.mark.parametrize("places", [1, 2, 3, 7])
def test_offsets_that_pass_over_the_places_draw_new_masks(places):
    every = [m for step in masks(4, places, places) for m in step]
    assert len(set(every)) == len(every)


def test_offsets_counted_by_one_repeat_a_neighbours_mask():
    a = masks(3, 3, 1)
    for t in (0, 1):
        for i in (0, 1):
            assert a[t + 1][i] == a[t][i + 1]


def test_the_documentation_says_so():
    import fp8_block_scaled_dg_amd as m
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    header = open(os.path.join(root, "include", "dg.h")).read()
    assert "other offsets or subsequences draw independent" not in header
    assert "at least n further on" in header and "by n or more" in m.dropout_add.__doc__


@pytest.mark.gpu
def test_the_example_draws_new_masks_at_every_place():
    import fp8_block_scaled_dg_amd as dg
    from tests.test_gpu_block import example
    model = example().PreNormGated(128, 128, 3, "silu", P, seed=SEED)
    ones, seen = torch.ones(N, device="cuda"), set()
    for t in range(3):
        for i in range(4):  # three layers and the end
            got = dg.dropout_add(ones, P, model.rng, i).cpu().numpy() != 0
            assert np.array_equal(got, blk.kept(0, N, P, SEED, 4 * t, i))
            seen.add(got.tobytes())
        model.advance()
    assert len(seen) == 12


@pytest.mark.gpu
def test_a_captured_step_advances():
    import fp8_block_scaled_dg_amd as dg
    from tests.test_gpu_block import example
    model = example().PreNormGated(128, 128, 2, "silu", P, seed=SEED)
    ones = torch.ones(N, device="cuda")
    out = [torch.empty_like(ones) for _ in range(3)]

    def step():
        for i in range(3):
            dg.dropout_add(ones, P, model.rng, i, out=out[i])
        model.advance()

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for t in range(1, 4):
        graph.replay()
        torch.cuda.synchronize()
        for i in range(3):
            assert np.array_equal(out[i].cpu().numpy() != 0, blk.kept(0, N, P, SEED, 3 * t, i)), (t, i)
