"""Sorts at the borders between their ways: one workgroup takes up to 8192 slots in
up to eight runs of its 16 waves, or 4096 in eight runs of 8 waves with more than
512 experts; more slots take a counting and a placing launch."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from tests.gpu_util import say
from tests.test_gpu_moe import _check_table, _experts, _table

pytestmark = pytest.mark.gpu


# (tokens, topk): five to eight runs, whole and partial waves, the last slot of one
# workgroup and the first beyond
@pytest.mark.parametrize("experts", [1, 16, 60, 511, 512])
@pytest.mark.parametrize("tokens, topk", [(4097, 1), (5120, 1), (777, 7), (6145, 1), (1024, 7), (7169, 1), (8191, 1), (4096, 2),
                                          (128, 64), (8193, 1), (4097, 2)])
def test_up_to_512_experts(gpu, tokens, topk, experts):
    one = tokens * topk <= 8192
    assert (fp8.load_library().fp8bw_moe_sort_ws_bytes(tokens, topk, experts) == 0) == one
    for seed, (align, dropped, skew) in enumerate([(1, 0.0, 0.0), (128, 0.2, 0.7)]):
        expert = _experts(tokens, topk, experts, seed, dropped, skew)
        say("moe_sort", tokens, topk, experts, align, dropped, skew)
        _check_table(_table(gpu, expert, experts, align, seed == 0), expert, experts, align)


@pytest.mark.parametrize("experts", [513, 1000, 1024])
@pytest.mark.parametrize("tokens, topk", [(513, 1), (2049, 1), (3000, 1), (3585, 1), (4095, 1), (2048, 2), (64, 64), (4097, 1),
                                          (2049, 2), (8193, 1)])
def test_more_than_512_experts(gpu, tokens, topk, experts):
    one = tokens * topk <= 4096
    assert (fp8.load_library().fp8bw_moe_sort_ws_bytes(tokens, topk, experts) == 0) == one
    for seed, (align, dropped, skew) in enumerate([(1, 0.0, 0.0), (16, 0.2, 0.7)]):
        expert = _experts(tokens, topk, experts, seed, dropped, skew)
        say("moe_sort", tokens, topk, experts, align, dropped, skew)
        _check_table(_table(gpu, expert, experts, align, seed == 1), expert, experts, align)


@pytest.mark.parametrize("experts", [512, 1024])
def test_every_slot_at_the_last_expert(gpu, experts):
    for tokens in (4096, 8192, 8193):
        expert = np.full((tokens, 1), experts - 1)
        say("moe_sort, one expert", tokens, experts)
        _check_table(_table(gpu, expert, experts, 128), expert, experts, 128)


@pytest.mark.parametrize("tokens, experts", [(8192, 512), (4096, 1024)])
def test_a_graph_of_the_largest_single_launch(gpu, tokens, experts):
    e = torch.from_numpy(_experts(tokens, 1, experts, 1)).to(gpu)
    fp8.moe_sort(e, experts, 128)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t = fp8.moe_sort(e, experts, 128)
    for seed in (2, 3, 4):
        expert = _experts(tokens, 1, experts, seed, 0.1, 0.5)
        e.copy_(torch.from_numpy(expert))
        torch.cuda.synchronize()
        say("moe_sort graph", tokens, experts, seed)
        graph.replay()
        torch.cuda.synchronize()
        _check_table(t, expert, experts, 128)
