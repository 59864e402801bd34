"""Which kernels the dense operators' calls launch, on the CPU (tests/launch_log.py): every kernel that the library
holds for them is one that some call reaches, and every one is run by a GPU test."""
import pytest

import launch_log
import test_gpu_dense as g
import test_gpu_dense_kernels as k


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    path = launch_log.build(tmp_path_factory.mktemp("launches"))
    if path is None:
        pytest.skip("g++ not available")
    return path


def _params(fn, names):
    return {m.args[0]: m.args[1] for m in fn.pytestmark if m.name == "parametrize"}[names]


def _k8(K, fp8):
    return max(128, K // 128 * 128) if fp8 else K


def calls_of_the_gpu_tests():
    """The calls of the GPU tests that check the operators' outputs."""
    calls = [("rmsnorm", T, H, q) for T, H, q in _params(g.test_rmsnorm, "T,H,quant")]
    calls += [("rmsnorm", 5, H, False) for H in _params(g.test_rmsnorm_of_large_values, "H")]
    calls += [("route", T, E, top) for T, E, top in _params(g.test_route, "T,E,k")]
    calls += [("linear", T, N, _k8(K, f), f, y) for T, N, K in g.SHAPES for f in (0, 1) for y in (0, 1)]
    calls += [("linear", T, N, _k8(K, f), f, y) for T, N, K in g.CHANGES for f, y in ((0, 0), (1, 0), (1, 1))]
    calls += [("linear", T, N, K, 0, 0) for T, N, K in _params(g.test_linear_of_many_rows, "T,N,K")]
    calls += [("linear", T, N, K, 0, y) for T, N, K in k.LINEAR for y in (0, 1)]
    for fn in (g.test_glu_where_its_ways_change, g.test_glu):
        calls += [("glu", T, _k8(H, f), max(128, I // 128 * 128) if f or q else I, f, q)
                  for T, H, I in _params(fn, "T,H,I") for f in (0, 1) for q in (0, 1)]
    calls += [("glu", T, H, I, 0, 0) for T, H, I in _params(g.test_glu_of_many_rows, "T,H,I")]
    calls += [("glu", T, H, I, int(f), 0) for T, H, I, f in k.GLU]
    calls += [("backward", 70, 2048, 6144, "12")]
    calls += [("backward", T, H, I, w) for T, H, I in _params(g.test_ffn_backward, "T,H,I") for w in ("x12", "x", "1", "2")]
    calls += [("backward", T, H, I, "x12") for T, H, I in _params(g.test_ffn_backward_where_its_launches_change, "T,H,I")]
    calls += [("backward",) + c for c in k.BACKWARD]
    return calls


def _dense(names):
    return [n for n in names if n.startswith(("dense_", "rmsnorm_", "route_"))]


def test_every_kernel_is_reached_and_tested(shim):
    kernels, launches = launch_log.launches(shim, calls_of_the_gpu_tests())
    run = {l[0] for c in launches for l in c}
    assert len(_dense(kernels)) > 50 and sorted(set(_dense(kernels)) - run) == []


def test_launches_are_within_the_device(shim):
    """At most 1024 threads and 160 KB of LDS a workgroup, fewer than 2^32 threads a launch, one to four launches a
    call, and at least one workgroup in each."""
    _, launches = launch_log.launches(shim, calls_of_the_gpu_tests())
    for call in launches:
        assert 1 <= len(call) <= 4
        for name, grid, threads, lds in call:
            assert 64 <= threads <= 1024 and lds <= 160 * 1024, name
            assert min(grid) >= 1 and grid[0] * threads < 2 ** 32 and max(grid[1:]) < 2 ** 16, name


def test_fp8_tiles_around_one_a_unit(shim):
    """The 64 x 128 tile is chosen over a range of sizes, not at one count of tiles: 256 to 288 of 128 x 128."""
    _, launches = launch_log.launches(shim, [("linear", T, 2048, 256, 1, 0) for T in (1920, 2048, 2049, 2177, 2304, 4096)])
    names = [c[0][0].split("<")[1] for c in launches]
    tile, small, large = "0,1,1,1,2,2,2,4,2,1>", "0,1,1,1,2,2,2,2,2,1>", "0,1,1,1,4,2,2,4,2,1>"
    assert names == [small, tile, tile, tile, tile, large]
