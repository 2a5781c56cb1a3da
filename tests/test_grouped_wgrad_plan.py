"""The plan of a grouped weight gradient as a host query: refusals, and that it
agrees with the workspace query and with the sizes alone (no GPU)."""

import ctypes

import pytest
import torch

import blockwise_scaled_fp8_amd as fp8

OK, NULL, SHAPE, UNSUP = 0, 1, 2, 5
TILE = {0: 128, 1: 64, 3: 256}


@pytest.mark.parametrize("want, args", [
    (SHAPE, (0, 64, 128, 1, 0)), (SHAPE, (64, -1, 128, 1, 0)), (SHAPE, (64, 64, 0, 1, 0)), (SHAPE, (64, 64, 200, 1, 0)),
    (SHAPE, (64, 64, 128, 0, 0)), (SHAPE, (64, 64, 128, (1 << 20) + 1, 0)), (SHAPE, (1 << 62, 64, 128, 1, 0)),
    (SHAPE, ((1 << 30) + 1, 64, 128, 1, 0)), (UNSUP, (64, 64, 128, 1, 2)), (UNSUP, (1 << 20, 1 << 20, 128, 64, 0)),
    (OK, (64, 64, 128, 1, 1))])
def test_refusals(want, args):
    lib = fp8.load_library()
    assert lib.fp8bw_grouped_wgrad_plan(*args, (ctypes.c_int64 * 4)()) == want
    assert bool(lib.fp8bw_last_error()) == (want != OK)
    assert lib.fp8bw_grouped_wgrad_plan(*args, None) == NULL


@pytest.mark.parametrize("M, N", [(1, 1), (64, 64), (100, 300), (256, 256), (512, 512), (1304, 1032), (2048, 2048), (8192, 5120)])
@pytest.mark.parametrize("blocks", [1, 4, 17, 256])
@pytest.mark.parametrize("groups", [1, 3, 16, 128])
def test_agrees_with_the_workspace(M, N, blocks, groups):
    K = 128 * blocks * groups
    ws = fp8.load_library().fp8bw_grouped_wgrad_ws_bytes(M, N, K, groups)
    for dtype in (torch.bfloat16, torch.float32):
        p = fp8.grouped_wgrad_plan(M, N, K, groups, dtype)
        t = TILE[p["config"]]
        assert p["tiles"] == groups * -(-M // t) * -(-N // t) and 1 <= p["pieces"] <= 32
        need = p["pieces"] * groups * M * N * 4 if p["pieces"] > 1 else 0
        assert ws == -(-need // 256) * 256
        assert not p["stream"] or (p["config"] == 3 and p["pieces"] == 1 and dtype == torch.bfloat16 and N % 8 == 0)


@pytest.mark.parametrize("args", [(1 << 30, 1 << 30, 128, 1 << 20, 0), (1 << 30, 1 << 30, 128, 1 << 16, 0),
                                  (1 << 29, 1 << 30, 1 << 20, 1 << 20, 1), (1 << 30, 1 << 30, 1 << 30, 1, 0)])
def test_tiles_past_64_bits(args):
    lib = fp8.load_library()
    assert lib.fp8bw_grouped_wgrad_plan(*args, (ctypes.c_int64 * 4)()) == UNSUP
    assert lib.fp8bw_grouped_wgrad_ws_bytes(*args[:4]) == 0
