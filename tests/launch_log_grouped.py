"""launch_log.py for the 4-bit and the expert-grouped operators.  A call is one of
    ("linear_w4", T, N, K, wtype)          ("glu_w4", T, inter, hidden, wtype)
    ("linear", E, R, N, K, wtype)          ("glu", E, R, inter, hidden, wtype)
    ("backward", E, R, hidden, inter, gradients, row list)
    ("rows", T, top_k, E)                  ("combine", T, top_k, H)
    ("combine_backward", T, top_k, H, gradients)       gradients: any of "x", "1", "2" and "y", "w"
with made-up addresses.
"""
import json
import os
import subprocess
import sys

import launch_log
from launch_log import A

FORMATS = {"bf16": 0, "int4": 2, "mxfp4": 4}


def _call(pe, c):
    kind, a = c[0], c[1:]
    if kind == "linear_w4":
        T, N, K, w = a
        pe.pe_linear_w4(0, FORMATS[w], A[0], K, A[1], A[2], None, 0, None, 0, T, N, K, A[3], N, 0)
    elif kind == "glu_w4":
        T, I, H, w = a
        pe.pe_glu_w4(0, FORMATS[w], 1, A[0], H, A[1], A[2], T, H, I, A[3], I)
    elif kind == "linear":
        E, R, N, K, w = a
        pe.pe_grouped_linear(0, FORMATS[w], A[0], K, 5, A[1], A[2], A[3], None if w == "bf16" else A[4], None, 0, R, E, N, K,
                             A[5], N, 0)
    elif kind == "glu":
        E, R, I, H, w = a
        pe.pe_grouped_glu(0, FORMATS[w], 1, A[0], H, 5, A[1], A[2], A[3], None if w == "bf16" else A[4], R, E, H, I, A[5], I)
    elif kind == "backward":
        E, R, H, I, which, gather = a
        pe.pe_grouped_ffn_backward(0, 1, A[0], H, A[1], H, 5 if gather else R, A[2] if gather else None, A[3], A[4], A[5],
                                   A[6], R, E, H, I, A[7], A[8], A[9] if "x" in which else None, H,
                                   A[10] if "1" in which else None, A[11] if "2" in which else None)
    elif kind == "rows":
        T, k, E = a
        pe.pe_group_rows(0, A[0], T, k, E, A[1], A[2], A[3])
    elif kind == "combine":
        T, k, H = a
        pe.pe_combine(0, A[0], H, T * k, A[1], A[2], None, 0, T, k, H, A[3], H)
    else:
        T, k, H, which = a
        pe.pe_combine_backward(0, A[0], H, A[1], A[2], A[3], H, T * k, T, k, H, A[4] if "y" in which else None, H,
                               A[5] if "w" in which else None)


def launches(shim, calls):
    """As launch_log.launches."""
    r = subprocess.run([sys.executable, os.path.abspath(__file__), shim], input=json.dumps(calls), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    d = json.loads(r.stdout)

    def parse(line):
        name, x, y, z, threads, lds = line.split()
        return launch_log.readable(name), (int(x), int(y), int(z)), int(threads), int(lds)
    return ([launch_log.readable(k) for k in d["kernels"]], [[parse(x) for x in c] for c in d["calls"]])


if __name__ == "__main__":
    launch_log._call = _call
    launch_log._main()
