"""Grouped weight gradients on the kernel that each size is meant for: every case
asserts the plan before it runs, so that a change of the plan's constants cannot
move it to another kernel unnoticed.  The stream of 256x256 tiles (ragged
windows, gaps, empty groups, as many groups as it takes), 256x256 and 128x128
tiles one to a workgroup (fp32, few tiles, columns or strides that the stream
does not take), pieces of each configuration, and the fall back to small tiles.
Tolerances are the GEMM's (tests/gpu_util.py)."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from oracle import moe
from tests.gpu_util import check_gemm_output, host_f32, say
from tests.test_gpu_grouped_wgrad import _case, _colmajor, _operands

pytestmark = pytest.mark.gpu

STREAM, LARGE, MIDDLE, SMALL = (3, 1, True), (3, 1, False), (0, 1, False), (1, 1, False)


def _planned(want, M, N, K, groups, od="bf16"):
    p = fp8.grouped_wgrad_plan(M, N, K, groups, torch.bfloat16 if od == "bf16" else torch.float32)
    assert (p["config"], p["pieces"], p["stream"]) == want, p
    return p


def _ends(lengths):
    return [int(e) * 128 for e in np.cumsum(lengths)]


def _edges(M, tile):
    """Rows at the first, inner and last tiles' borders, and the last window's first row."""
    r = {0, 1, tile - 1, tile, M - tile - 1, M - tile, M // tile * tile - 1, M // tile * tile, M - 2, M - 1}
    return sorted(i for i in r if 0 <= i < M)


# odd and even lengths, one, none, one group that is long
LENGTHS = [1, 13, 2, 0, 5, 7, 0, 3, 4, 9, 2, 6, 1, 8, 3, 0]


@pytest.mark.parametrize("M, N, lengths, tail", [
    (1304, 1032, LENGTHS, 0),                       # the last windows move back by 232 rows and 248 columns
    (776, 520, [1] * 20 + [120] + [0, 2] * 9 + [3], 90),
    (1288, 768, [4] * 24, 0), (768, 1048, [5, 6] * 16, 0)])
def test_stream_of_ragged_windows(gpu, M, N, lengths, tail):
    ends = _ends(lengths)
    K = ends[-1] + 128 * tail
    _planned(STREAM, M, N, K, len(ends))
    got = _case(gpu, M, N, K, ends, "bf16", seed=M, rows=_edges(M, 256))
    for g, n in enumerate(lengths):
        assert (not got[g].any()) == (n == 0)


@pytest.mark.parametrize("row_gap, col_gap", [(1, 8), (0, 24), (5, 0)])
def test_stream_leaves_gaps_alone(gpu, row_gap, col_gap):
    M, N, G = 776, 520, 40
    lengths = [(7 * i) % 13 for i in range(G)]
    ends = _ends(lengths)
    K = max(ends[-1], 128 * 6 * G)
    _planned(STREAM, M, N, K, G)
    a, ra, b, rb = _operands(M, N, K, 3)
    out = torch.full((G, M + row_gap, N + col_gap), 7.0, dtype=torch.bfloat16, device=gpu)
    say("wgrad stream, gaps", row_gap, col_gap)
    fp8.fp8_scaled_grouped_gemm_blockwise_wgrad(
        torch.from_numpy(a).to(gpu), _colmajor(ra, gpu), torch.from_numpy(b).to(gpu), _colmajor(rb, gpu),
        torch.tensor(ends, dtype=torch.int32, device=gpu), out=out[:, :M, :N])
    rows = _edges(M, 256)
    ref, size = moe.grouped_wgrad(a[rows], ra[rows], b, rb, ends)
    check_gemm_output(host_f32(out[:, rows, :N]).reshape(-1, N), ref.reshape(-1, N), size.reshape(-1, N), K // 128, "bf16",
                      "stream, gaps")
    assert (out[:, M:] == 7.0).all() and (out[:, :, N:] == 7.0).all()


def test_stream_of_strided_operands(gpu):
    """Codes out of wider buffers, row-major scales."""
    M, N = 1304, 1032
    ends = _ends(LENGTHS)
    K = ends[-1]
    _planned(STREAM, M, N, K, 16)
    a, ra, b, rb = _operands(M, N, K, 4)
    wide = [torch.full((n, K + pad), 0x7F, dtype=torch.uint8, device=gpu) for n, pad in ((M, 128), (N, 16))]
    for t, v in zip(wide, (a, b)):
        t[:, :K] = torch.from_numpy(v).to(gpu)
    out = torch.full((16, M, N), float("nan"), dtype=torch.bfloat16, device=gpu)
    say("wgrad stream, strided operands")
    fp8.fp8_scaled_grouped_gemm_blockwise_wgrad(
        wide[0][:, :K], torch.from_numpy(ra).to(gpu), wide[1][:, :K], torch.from_numpy(rb).to(gpu),
        torch.tensor(ends, dtype=torch.int32, device=gpu), out=out)
    rows = _edges(M, 256)
    ref, size = moe.grouped_wgrad(a[rows], ra[rows], b, rb, ends)
    check_gemm_output(host_f32(out[:, rows]).reshape(-1, N), ref.reshape(-1, N), size.reshape(-1, N), K // 128, "bf16",
                      "stream, strided")


@pytest.mark.parametrize("ends", [[0] * 40, [0] * 39 + [128], [640] + [640] * 39, [128 * 160] * 40])
def test_stream_of_empty_groups(gpu, ends):
    M, N, K = 768, 776, 128 * 160
    _planned(STREAM, M, N, K, 40)
    got = _case(gpu, M, N, K, ends, "bf16", seed=5, rows=[0, 255, 256, 511, 767])
    for g in range(40):
        assert got[g].any() == (ends[g] > (ends[g - 1] if g else 0))


@pytest.mark.parametrize("groups, want", [(1024, STREAM), (1025, LARGE)])
def test_as_many_groups_as_the_stream_takes(gpu, groups, want):
    lengths = [(i * 7) % 3 for i in range(groups)]
    ends = _ends(lengths)
    K = max(ends[-1], 128 * groups)
    _planned(want, 256, 256, K, groups)
    _case(gpu, 256, 256, K, ends, "bf16", seed=6, rows=[0, 130, 255])


@pytest.mark.parametrize("M, N, lengths, od", [
    (1304, 1032, LENGTHS, "f32"), (1304, 1033, LENGTHS, "bf16"), (1304, 1033, LENGTHS, "f32"), (1288, 1030, LENGTHS, "bf16"),
    (1000, 1100, [3, 0, 9, 4, 1, 0, 7, 2, 5, 6, 8, 3], "bf16"),        # 240 tiles
    (1024, 1024, [3, 0, 9, 4, 1, 0, 7, 2, 5, 6, 8, 3], "f32"), (256, 256, [4] * 100 + [0, 8] * 25, "bf16")])
def test_one_large_tile_a_workgroup(gpu, M, N, lengths, od):
    ends = _ends(lengths)
    _planned(LARGE, M, N, ends[-1], len(ends), od)
    got = _case(gpu, M, N, ends[-1], ends, od, seed=M + N, rows=_edges(M, 256))
    for g, n in enumerate(lengths):
        assert (not got[g].any()) == (n == 0)


@pytest.mark.parametrize("row_gap, col_gap, od", [(0, 4, torch.bfloat16), (0, 1, torch.bfloat16), (1, 2, torch.float32)])
def test_outputs_that_the_stream_does_not_take(gpu, row_gap, col_gap, od):
    """Output rows that are no multiples of 16 bytes apart: large tiles, stored in
    smaller pieces."""
    M, N = 1304, 1032
    ends = _ends(LENGTHS)
    K = ends[-1]
    _planned(STREAM, M, N, K, 16)
    a, ra, b, rb = _operands(M, N, K, 7)
    out = torch.full((16, M + row_gap, N + col_gap), 7.0, dtype=od, device=gpu)
    say("wgrad large tiles, output stride", N + col_gap, od)
    fp8.fp8_scaled_grouped_gemm_blockwise_wgrad(
        torch.from_numpy(a).to(gpu), _colmajor(ra, gpu), torch.from_numpy(b).to(gpu), _colmajor(rb, gpu),
        torch.tensor(ends, dtype=torch.int32, device=gpu), out=out[:, :M, :N])
    rows = _edges(M, 256)
    ref, size = moe.grouped_wgrad(a[rows], ra[rows], b, rb, ends)
    check_gemm_output(host_f32(out[:, rows, :N]).reshape(-1, N), ref.reshape(-1, N), size.reshape(-1, N), K // 128,
                      "bf16" if od == torch.bfloat16 else "f32", "large tiles, output stride")
    assert (out[:, M:] == 7.0).all() and (out[:, :, N:] == 7.0).all()


@pytest.mark.parametrize("od", ["bf16", "f32"])
@pytest.mark.parametrize("want, M, N, groups", [(MIDDLE, 1040, 1040, 16), (MIDDLE, 520, 776, 60), (SMALL, 392, 400, 17),
                                                (SMALL, 1040, 144, 64)])
def test_one_smaller_tile_a_workgroup(gpu, want, M, N, groups, od):
    lengths = [(5 * i) % 9 for i in range(groups)]
    ends = _ends(lengths)
    K = max(ends[-1], 128 * 4 * groups)
    _planned(want, M, N, K, groups, od)
    _case(gpu, M, N, K, ends, od, seed=8, rows=_edges(M, 128 if want is MIDDLE else 64))


@pytest.mark.parametrize("od", ["bf16", "f32"])
@pytest.mark.parametrize("config, pieces, M, N, lengths, tail", [
    (3, 4, 2048, 2048, [64], 0), (3, 4, 2040, 2060, [150, 106], 0), (3, 8, 2050, 2049, [254], 2),
    (0, 4, 1100, 900, [64], 3), (1, 4, 1024, 1024, [40], 0), (1, 32, 64, 64, [40], 0)])
def test_pieces(gpu, config, pieces, M, N, lengths, tail, od):
    ends = _ends(lengths)
    K = ends[-1] + 128 * tail
    _planned((config, pieces, False), M, N, K, len(ends), od)
    got = _case(gpu, M, N, K, ends, od, seed=M + N, rows=_edges(M, 256))
    again = _case(gpu, M, N, K, ends, od, seed=M + N, rows=[0])
    assert np.array_equal(got, again)


def test_a_stride_past_the_large_tiles_offsets(gpu):
    """256x256 tiles are planned, but 256 rows of codes 2^23 apart pass their
    32-bit offsets: small tiles run instead."""
    M, N, G, ld = 256, 256, 150, 1 << 23
    lengths = [(3 * i) % 9 for i in range(G)]
    ends = _ends(lengths)
    K = max(ends[-1], 128 * 4 * G)
    _planned(LARGE, M, N, K, G)
    a, ra, b, rb = _operands(M, N, K, 9)
    wide = torch.empty(M * ld, dtype=torch.uint8, device=gpu).view(M, ld)
    wide[:, :K] = torch.from_numpy(a).to(gpu)
    say("wgrad, wide stride")
    out = fp8.fp8_scaled_grouped_gemm_blockwise_wgrad(
        wide[:, :K], _colmajor(ra, gpu), torch.from_numpy(b).to(gpu), _colmajor(rb, gpu),
        torch.tensor(ends, dtype=torch.int32, device=gpu))
    rows = [0, 63, 64, 128, 255]
    ref, size = moe.grouped_wgrad(a[rows], ra[rows], b, rb, ends)
    check_gemm_output(host_f32(out[:, rows]).reshape(-1, N), ref.reshape(-1, N), size.reshape(-1, N), K // 128, "bf16", "wide")
