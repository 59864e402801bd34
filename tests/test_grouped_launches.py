"""Which kernels the 4-bit and the expert-grouped operators' calls launch, on the CPU (launch_log_grouped.py): every kernel
that the library holds for them is one that some call reaches, and every one is run by a GPU test."""
import pytest

import launch_log
import launch_log_grouped
import test_gpu_grouped as g


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    path = launch_log.build(tmp_path_factory.mktemp("launches"))
    if path is None:
        pytest.skip("g++ not available")
    return path


def _params(fn, names):
    return {m.args[0]: m.args[1] for m in fn.pytestmark if m.name == "parametrize"}[names]


def calls_of_the_gpu_tests():
    """The calls of the GPU tests that check the operators' outputs."""
    q = ("int4", "mxfp4")
    calls = [("linear_w4", T, N, g._k(w, K), w) for T, N, K in g.W4 + g.WAYS_LINEAR for w in q]
    calls += [("glu_w4", T, I, g._k(w, H), w) for T, I, H in _params(g.test_glu_w4, "T,I,H") + g.WAYS_GLU for w in q]
    for w in ("bf16",) + q:
        calls += [("linear", len(c), sum(c) + b, N, g._k(w, K), w) for c, b in g.COUNTS
                  for N, K in _params(g.test_grouped_linear, "N,K")]
        calls += [("glu", len(c), sum(c) + b, I, g._k(w, H), w) for c, b in g.COUNTS
                  for I, H in _params(g.test_grouped_glu, "I,H")]
        calls += [("linear", E, R, N, K, w) for E, R, N, K in g.WAYS_GROUPED]
        calls += [("glu", E, R, N // 2 // 8 * 8, K, w) for E, R, N, K in g.WAYS_GROUPED]
    calls += [("backward", len(c), sum(c) + b, H, I, "x12", gather) for c, b in g.COUNTS
              for H, I in _params(g.test_grouped_ffn_backward, "H,I") for gather in (0, 1)]
    calls += [("backward", E, R, H, I, "x12", 1)
              for E, R, H, I in _params(g.test_grouped_ffn_backward_where_its_ways_change, "E,R,H,I")]
    calls += [("rows", T, k, E) for f in (g.test_group_rows, g.test_group_rows_of_many_entries)
              for T, k, E in _params(f, "T,k,E")]
    for T, k, H in _params(g.test_combine_and_its_gradients, "T,k,H"):
        calls += [("combine", T, k, H)] + [("combine_backward", T, k, H, w) for w in ("yw", "y", "w")]
    return calls


def _grouped(names):
    return [n for n in names if n.startswith(("grouped_", "quant_", "group_rows", "combine_"))]


def test_every_kernel_is_reached_and_tested(shim):
    kernels, launches = launch_log_grouped.launches(shim, calls_of_the_gpu_tests())
    run = {l[0] for c in launches for l in c}
    assert len(_grouped(kernels)) > 40 and sorted(set(_grouped(kernels)) - run) == []


def test_launches_are_within_the_device(shim):
    """At most 1024 threads and 160 KB of LDS a workgroup, fewer than 2^32 threads a launch, and at least one workgroup."""
    large = [("linear", 1024, 2 ** 20, 4096, 2048, "bf16"), ("glu", 1024, 3000, 4096, 2048, "int4"),
             ("linear_w4", 2 ** 20, 8000, 1024, "mxfp4"), ("backward", 1024, 2 ** 18, 4096, 2048, "x12", 1),
             ("combine", 2 ** 20, 8, 8192), ("combine_backward", 2 ** 20, 8, 8192, "yw"), ("rows", 2 ** 20, 8, 1024),
             ("linear_w4", 3, 2 ** 21, 2048, "int4"), ("linear_w4", 2 ** 22, 8, 128, "int4"),
             ("linear", 1024, 1024, 2 ** 18, 128, "bf16"), ("glu", 1024, 1024, 2 ** 18, 128, "mxfp4")]
    _, launches = launch_log_grouped.launches(shim, calls_of_the_gpu_tests() + large)
    for call in launches:
        assert 1 <= len(call) <= 4
        for name, grid, threads, lds in call:
            assert 64 <= threads <= 1024 and lds <= 160 * 1024, name
            assert min(grid) >= 1 and grid[0] * grid[1] * threads < 2 ** 32 and max(grid[1:]) < 2 ** 16, name
