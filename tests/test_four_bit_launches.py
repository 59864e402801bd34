"""That the calls of test_gpu_four_bit.py take the kernels that they are there for, on the CPU (launch_log_grouped.py)."""
import pytest

import launch_log
import launch_log_grouped
import test_gpu_four_bit as f


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    path = launch_log.build(tmp_path_factory.mktemp("launches"))
    if path is None:
        pytest.skip("g++ not available")
    return path


def _grouped_calls(shapes, wtype):
    return [("linear",) + c + (wtype,) for c in shapes] + [
        ("glu", E, R, N // 2 // 8 * 8, K, wtype) for E, R, N, K in shapes]


def _launched(shim, calls):
    """All kernels of the library, and each call's."""
    kernels, launches = launch_log_grouped.launches(shim, calls)
    assert all(len(c) == 1 for c in launches)
    return kernels, [c[0][0] for c in launches]


def test_every_int4_kernel_is_run(shim):
    calls = [("linear_w4",) + c + ("int4",) for c in f.INT4_LINEAR] + [("glu_w4",) + c + ("int4",) for c in f.INT4_GLU]
    kernels, run = _launched(shim, calls + _grouped_calls(f.INT4_GROUPED, "int4"))
    of_int4 = {k for k in kernels for op in (0, 1) for name in ("quant_tile", "grouped_few")
               if k.startswith("%s_kernel<%d,2," % (name, op))}
    assert len(of_int4) >= 15 and sorted(of_int4 - set(run)) == []


def test_every_mxfp4_tile_is_run_with_k_that_ends_inside_a_step(shim):
    calls = [("linear_w4",) + c + ("mxfp4",) for c in f.MX_LINEAR] + [("glu_w4",) + c + ("mxfp4",) for c in f.MX_GLU]
    calls += _grouped_calls(f.MX_GROUPED, "mxfp4")
    kernels, run = _launched(shim, calls)
    tiles = {k for k in kernels for op in (0, 1) if k.startswith("quant_tile_kernel<%d,4," % op)}
    assert len(tiles) == 10
    for left in (32, 64, 96):
        assert left in {c[-2] % 128 for c in calls}
    for tile in tiles:
        ks = {c[-2] for c, k in zip(calls, run) if k == tile}
        assert ks and all(k % 128 for k in ks) and min(ks) < 192 and max(ks) > 1024, (tile, ks)


def test_codes_and_scales_go_through_every_kernel(shim):
    calls = [("linear_w4",) + c[1:] + c[:1] for c in f.PICKED_LINEAR] + [("glu_w4",) + c[1:] + c[:1] for c in f.PICKED_GLU]
    for wtype in ("int4", "mxfp4"):
        calls += _grouped_calls([c[1:] for c in f.PICKED_GROUPED if c[0] == wtype], wtype)
    kernels, run = _launched(shim, calls)
    assert sorted({k for k in kernels for w in (2, 4) for name in ("quant_tile", "grouped_few")
                   for op in (0, 1) if k.startswith("%s_kernel<%d,%d," % (name, op, w))} - set(run)) == []


def test_calls_of_few_rows_stream_their_weights(shim):
    """A tile of 16 rows and more would be empty but for these: one matrix of many columns, and few experts of some rows
    each.  Wider, or of more rows, they take tiles."""
    streams, tiles = [], []
    for w in ("int4", "mxfp4"):
        streams += [("linear_w4", T, 32768, 4096, w) for T in (1, 4)] + [("glu_w4", T, 14336, 4096, w) for T in (1, 4)]
        streams += [("glu", E, E * r, 768, 2048, w) for E, r in ((1, 16), (4, 4), (8, 8), (8, 16), (16, 4))]
        streams += [("linear", E, E * r, 2048, 768, w) for E, r in ((2, 16), (4, 8), (8, 16))]
        tiles += [("linear_w4", 1, 65536, 2048, w), ("linear_w4", 8, 32768, 4096, w), ("glu_w4", 1, 24576, 2048, w),
                  ("linear_w4", 1, 32768, 1024, w), ("glu", 32, 32 * 4, 768, 2048, w), ("glu", 8, 8 * 17, 768, 2048, w)]
    streams += [("glu", 4, 32, 768, 2048, "bf16"), ("glu", 2, 32, 768, 2048, "bf16"), ("linear", 4, 16, 1536, 2048, "bf16")]
    tiles += [("glu", 4, 96, 768, 2048, "bf16"), ("linear", 12, 48, 1536, 2048, "bf16"), ("linear", 4, 68, 1536, 2048, "bf16")]
    _, run = _launched(shim, streams + tiles)
    for c, k in zip(streams + tiles, run):
        assert k.startswith("grouped_few") == (c in streams), (c, k)
