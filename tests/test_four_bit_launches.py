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
