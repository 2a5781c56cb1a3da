"""Grouped weight gradients on the GPU against the oracle: groups of many
lengths, empty ones, every tile size, fp32 and bf16 outputs, strided operands
and a malformed table.  Tolerances are the GEMM's (tests/gpu_util.py)."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from oracle import moe
from tests.gpu_util import check_gemm_output, host_f32, say

pytestmark = pytest.mark.gpu


def _codes(rng, shape):
    c = rng.integers(0, 256, size=shape).astype(np.uint8)
    c[(c & 0x7F) == 0x7F] = 0x7E
    return c


def _operands(M, N, K, seed):
    rng = np.random.default_rng(seed)
    return (_codes(rng, (M, K)), rng.uniform(1e-3, 2e-3, (M, K // 128)).astype(np.float32),
            _codes(rng, (N, K)), rng.uniform(1e-3, 2e-3, (N, K // 128)).astype(np.float32))


def _colmajor(r, gpu):
    return torch.from_numpy(np.ascontiguousarray(r.T)).to(gpu).t()


def _case(gpu, M, N, K, ends, od="f32", seed=0, rows=None):
    a, ra, b, rb = _operands(M, N, K, seed)
    dt = torch.bfloat16 if od == "bf16" else torch.float32
    out = torch.full((len(ends), M, N), float("nan"), dtype=dt, device=gpu)
    say("grouped wgrad", M, N, K, od, list(ends)[:10])
    got = fp8.fp8_scaled_grouped_gemm_blockwise_wgrad(
        torch.from_numpy(a).to(gpu), _colmajor(ra, gpu), torch.from_numpy(b).to(gpu), _colmajor(rb, gpu),
        torch.tensor(ends, dtype=torch.int32, device=gpu), out=out)
    torch.cuda.synchronize()
    assert got is out
    rows = np.arange(M) if rows is None else np.asarray(rows)
    ref, size = moe.grouped_wgrad(a[rows], ra[rows], b, rb, ends)
    check_gemm_output(host_f32(out)[:, rows].reshape(-1, N), ref.reshape(-1, N), size.reshape(-1, N), K // 128, od,
                      f"wgrad {len(ends)}x{M}x{N}x{K}")
    return host_f32(out)


# small tiles; both 128-row kinds; whole and ragged large tiles; many groups
@pytest.mark.parametrize("od", ["bf16", "f32"])
@pytest.mark.parametrize("M, N, K, ends", [
    (16, 16, 128, [128]), (1, 33, 256, [128, 256]), (64, 64, 640, [0, 128, 128, 512, 640]),
    (200, 136, 512, [256, 512]), (512, 256, 1024, [128, 128, 640, 640, 1024, 1024, 1024, 1024])])
def test_small(gpu, M, N, K, ends, od):
    _case(gpu, M, N, K, ends, od, seed=M + N)


def test_tiles_of_128(gpu):
    # 17 groups x 4 x 4 tiles of 128 x 128, too few for larger ones
    _case(gpu, 392, 400, 512, [128 * (i // 5) for i in range(1, 18)], "bf16", seed=3, rows=np.r_[0:20, 120:140, 380:392])


def test_tiles_of_256_by_128(gpu):
    # N below 256: 256 x 128 tiles, ragged in both directions
    _case(gpu, 1040, 144, 384, [128 * min(3, i % 4) for i in np.sort(np.arange(64) % 4)], "f32", seed=4,
          rows=np.r_[0:8, 250:262, 1030:1040])


@pytest.mark.parametrize("od", ["bf16", "f32"])
def test_large_tiles(gpu, od):
    # 16 groups x 5 x 5 ragged tiles of 256 x 256
    ends = np.cumsum([1, 0, 2, 3, 0, 0, 1, 1, 4, 0, 1, 2, 1, 0, 1, 0]) * 128
    _case(gpu, 1168, 1136, int(ends[-1]) + 256, [int(e) for e in ends], od, seed=5,
          rows=np.r_[0:6, 253:259, 1022:1030, 1160:1168])


def test_codes_behind_the_last_end_are_not_used(gpu):
    a, ra, b, rb = _operands(256, 256, 512, 6)
    a[:, 256:] = 0x7F          # NaN
    rb[:, 2:] = np.inf
    out = fp8.fp8_scaled_grouped_gemm_blockwise_wgrad(
        torch.from_numpy(a).to(gpu), _colmajor(ra, gpu), torch.from_numpy(b).to(gpu), _colmajor(rb, gpu),
        torch.tensor([128, 256], dtype=torch.int32, device=gpu), out_dtype=torch.float32)
    assert out.isfinite().all()


def test_a_malformed_table_stays_inside(gpu):
    """Ends past the last column, negative or falling: clamped, an empty group's
    output is zero."""
    got = _case(gpu, 320, 272, 512, [128, 384, 10 ** 6, 2 ** 31 - 1], seed=7)
    assert not got[3].any()
    a, ra, b, rb = _operands(320, 272, 512, 8)
    out = fp8.fp8_scaled_grouped_gemm_blockwise_wgrad(
        torch.from_numpy(a).to(gpu), _colmajor(ra, gpu), torch.from_numpy(b).to(gpu), _colmajor(rb, gpu),
        torch.tensor([-2 ** 31, 256, 128, -5], dtype=torch.int32, device=gpu), out_dtype=torch.float32)
    assert not out[0].any() and not out[2].any() and not out[3].any()
    ref, size = moe.grouped_wgrad(a, ra, b, rb, [0, 256])
    check_gemm_output(host_f32(out[1]), ref[1], size[1], 4, "f32", "after a negative end")


def test_strides(gpu):
    """Operands out of wider buffers, row-major scales, an output of padded
    rows and groups whose gaps stay as they were."""
    M, N, K = 272, 288, 384
    a, ra, b, rb = _operands(M, N, K, 9)
    wide = torch.zeros(M, K + 64, dtype=torch.uint8, device=gpu)
    wide[:, :K] = torch.from_numpy(a).to(gpu)
    out = torch.full((2, M + 3, N + 5), 7.0, device=gpu)
    fp8.fp8_scaled_grouped_gemm_blockwise_wgrad(
        wide[:, :K], torch.from_numpy(ra).to(gpu), torch.from_numpy(b).to(gpu), torch.from_numpy(rb).to(gpu),
        torch.tensor([256, 384], dtype=torch.int32, device=gpu), out=out[:, :M, :N])
    ref, size = moe.grouped_wgrad(a, ra, b, rb, [256, 384])
    check_gemm_output(host_f32(out[:, :M, :N]).reshape(-1, N), ref.reshape(-1, N), size.reshape(-1, N), 3, "f32", "strided")
    assert (out[:, M:] == 7.0).all() and (out[:, :, N:] == 7.0).all()


def test_no_groups_and_no_columns(gpu):
    a, ra, b, rb = _operands(32, 48, 128, 10)
    t = [torch.from_numpy(a).to(gpu), _colmajor(ra, gpu), torch.from_numpy(b).to(gpu), _colmajor(rb, gpu)]
    assert fp8.fp8_scaled_grouped_gemm_blockwise_wgrad(*t, torch.empty(0, dtype=torch.int32, device=gpu)).shape == (0, 32, 48)
    none = [t[0][:, :0], t[1][:, :0], t[2][:, :0], t[3][:, :0]]
    out = fp8.fp8_scaled_grouped_gemm_blockwise_wgrad(*none, torch.zeros(3, dtype=torch.int32, device=gpu))
    assert out.shape == (3, 32, 48) and not out.any()


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("G, rows, cols", [(1, 128, 128), (3, 256, 384), (5, 144, 272)])
def test_grouped_quantizer_is_the_quantizer(gpu, G, rows, cols, transpose):
    g = torch.Generator().manual_seed(11)
    x = torch.randn(G, rows + 4, cols + 8, generator=g).bfloat16().to(gpu)[:, :rows, :cols]
    say("quant grouped", G, rows, cols, transpose)
    q, recip = fp8.fp8_blockwise_quant_grouped(x, transpose)
    for i in range(G):
        want, want_recip = fp8.fp8_blockwise_quant(x[i], "128x128", transpose)
        assert torch.equal(q[i], want) and torch.equal(recip[i], want_recip)


def _stream_case(gpu, M, N, ends, K, rows, seed):
    """More 256x256 tiles than compute units: workgroups that run several tiles."""
    return _case(gpu, M, N, K, ends, "bf16", seed=seed, rows=rows)


def test_streams_of_whole_tiles(gpu):
    # 64 groups x 2 x 3 tiles; odd and even lengths, equal ones, empty groups
    lengths = [(7 * i) % 6 for i in range(64)]
    ends = [int(e) * 128 for e in np.cumsum(lengths)]
    got = _stream_case(gpu, 512, 768, ends, ends[-1] + 128, np.r_[0:4, 254:258, 508:512], 20)
    for g, n in enumerate(lengths):
        assert (not got[g].any()) == (n == 0)


def test_streams_of_ragged_tiles(gpu):
    # 2 x 2 tiles a group whose windows overlap; one long group among many short
    lengths = [1] * 40 + [37] + [2] * 30 + [0] * 9
    ends = [int(e) * 128 for e in np.cumsum(lengths)]
    _stream_case(gpu, 360, 264, ends, ends[-1], np.r_[0:3, 100:108, 252:260, 356:360], 21)


def test_streams_of_empty_groups_only(gpu):
    out = _case(gpu, 512, 512, 256, [0] * 80, "bf16", seed=22, rows=[0, 511])
    assert not out.any()


def test_stream_leaves_gaps_alone(gpu):
    """Strided outputs: rows and groups with gaps between them."""
    M, N, K, G = 264, 520, 384, 100
    a, ra, b, rb = _operands(M, N, K, 23)
    ends = [min(3, i // 20) * 128 for i in range(1, G + 1)]
    out = torch.full((G, M + 1, N + 8), 7.0, dtype=torch.bfloat16, device=gpu)
    fp8.fp8_scaled_grouped_gemm_blockwise_wgrad(
        torch.from_numpy(a).to(gpu), _colmajor(ra, gpu), torch.from_numpy(b).to(gpu), _colmajor(rb, gpu),
        torch.tensor(ends, dtype=torch.int32, device=gpu), out=out[:, :M, :N])
    ref, size = moe.grouped_wgrad(a[:40], ra[:40], b, rb, ends)
    check_gemm_output(host_f32(out[:, :40, :N]).reshape(-1, N), ref.reshape(-1, N), size.reshape(-1, N), 3, "bf16", "stream")
    assert (out[:, M:] == 7.0).all() and (out[:, :, N:] == 7.0).all()


@pytest.mark.parametrize("od", ["bf16", "f32"])
@pytest.mark.parametrize("M, N, lengths, tail", [
    (64, 64, [40], 0), (130, 70, [33, 0, 5], 2), (512, 512, [64], 0), (48, 1001, [17, 30], 1), (256, 256, [9, 60, 0, 3], 4),
    (1024, 1024, [40], 0), (1100, 900, [64], 3)])
def test_long_contractions_in_pieces(gpu, M, N, lengths, tail, od):
    """Few tiles over long contractions: pieces joined in order, some of them
    empty where a group is short."""
    ends = [int(e) * 128 for e in np.cumsum(lengths)]
    K = ends[-1] + 128 * tail
    assert fp8.load_library().fp8bw_grouped_wgrad_ws_bytes(M, N, K, len(ends)) > 0
    got = _case(gpu, M, N, K, ends, od, seed=M + N, rows=np.r_[0:min(M, 40), M - 1])
    again = _case(gpu, M, N, K, ends, od, seed=M + N, rows=[0])
    assert np.array_equal(got, again)


def test_pieces_into_a_strided_output(gpu):
    M, N, K = 96, 120, 128 * 40
    a, ra, b, rb = _operands(M, N, K, 30)
    for N_, od in ((N, torch.bfloat16), (N - 1, torch.float32), (N - 2, torch.bfloat16)):
        out = torch.full((2, M + 2, N + 3), 7.0, dtype=od, device=gpu)
        ends = [128 * 7, K]
        fp8.fp8_scaled_grouped_gemm_blockwise_wgrad(
            torch.from_numpy(a).to(gpu), _colmajor(ra, gpu), torch.from_numpy(b[:N_].copy()).to(gpu),
            _colmajor(rb[:N_], gpu), torch.tensor(ends, dtype=torch.int32, device=gpu), out=out[:, :M, :N_])
        ref, size = moe.grouped_wgrad(a, ra, b[:N_], rb[:N_], ends)
        check_gemm_output(host_f32(out[:, :M, :N_]).reshape(-1, N_), ref.reshape(-1, N_), size.reshape(-1, N_), 40,
                          "f32" if od == torch.float32 else "bf16", "pieces, strided")
        assert (out[:, M:] == 7.0).all() and (out[:, :, N_:] == 7.0).all()


def test_strides_that_the_large_tiles_do_not_take(gpu):
    """A row stride of 2^23 codes: 256 rows pass 2^31 bytes, so that the large
    tiles' 32-bit offsets do not reach; the small ones run instead."""
    M, N, K, ld = 272, 256, 256, 1 << 23
    a, ra, b, rb = _operands(M, N, K, 31)
    wide = torch.empty(M * ld, dtype=torch.uint8, device=gpu).view(M, ld)
    wide[:, :K] = torch.from_numpy(a).to(gpu)
    say("wide stride")
    out = fp8.fp8_scaled_grouped_gemm_blockwise_wgrad(
        wide[:, :K], _colmajor(ra, gpu), torch.from_numpy(b).to(gpu), _colmajor(rb, gpu),
        torch.tensor([128, 256] + [256] * 300, dtype=torch.int32, device=gpu), out_dtype=torch.float32)
    ref, size = moe.grouped_wgrad(a[-30:], ra[-30:], b, rb, [128, 256])
    check_gemm_output(host_f32(out[:2, -30:]).reshape(-1, N), ref.reshape(-1, N), size.reshape(-1, N), 2, "f32", "wide")
