"""Which kernels libpe.so launches for a call, found without a GPU.

`launches(calls)` runs this file as a program of its own, in which the HIP
runtime is tests/native/launch_log.cpp: the library's host code runs as it is,
checks, choices of kernel and all, and its launches are written down.  A call is
one of
    ("rmsnorm", T, H, quant)             ("route", T, experts, k)
    ("linear", T, N, K, fp8, fp32 out)   ("glu", T, hidden, inter, fp8, e4m3 out)
    ("backward", T, hidden, inter, gradients)   gradients: any of "x", "1", "2"
with made-up addresses.
"""
import ctypes
import json
import os
import re
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
A = [0x10000000000 * (i + 1) for i in range(12)]      # addresses far apart


def _call(pe, c):
    kind, a = c[0], c[1:]
    if kind == "rmsnorm":
        T, H, quant = a
        pe.pe_rmsnorm(0, A[0], H, None, 0, A[1], 1e-6, T, H, None, 0, A[2], H, A[3] if quant else None)
    elif kind == "route":
        T, E, k = a
        pe.pe_route(0, A[0], E, T, E, k, 0, 1, 1.0, A[1], A[2])
    elif kind == "linear":
        T, N, K, fp8, f32 = a
        s = (A[5], A[6]) if fp8 else (None, None)
        pe.pe_linear(0, int(fp8), A[0], K, s[0], A[1], s[1], None, 0, None, 0, T, N, K, A[2], N, int(f32))
    elif kind == "glu":
        T, H, I, fp8, quant = a
        s = (A[5], A[6]) if fp8 else (None, None)
        pe.pe_glu(0, int(fp8), 1, A[0], H, s[0], A[1], s[1], T, H, I, A[2], I, A[3] if quant else None)
    else:
        T, H, I, which = a
        pe.pe_ffn_backward(0, 1, A[0], H, A[1], H, A[2], A[3], A[4], T, H, I, A[5], A[6], A[7] if "x" in which else None,
                           H, A[8] if "1" in which else None, A[9] if "2" in which else None)


def _main():
    shim = ctypes.CDLL(sys.argv[1], ctypes.RTLD_GLOBAL)
    shim.launch_log_kernels.restype = shim.launch_log_take.restype = ctypes.c_char_p
    sys.path.insert(0, ROOT)
    import host_paged_expert_amd as pe
    pe.lib()
    done = []
    for c in json.load(sys.stdin):
        _call(pe, c)
        done.append(shim.launch_log_take().decode().splitlines())
    json.dump({"kernels": shim.launch_log_kernels().decode().splitlines(), "calls": done}, sys.stdout)


def readable(mangled):
    """dense_tile_kernel<0,1,1,1,2,2,2,4,2,1> from the mangled name: the template's arguments as numbers."""
    m = re.match(r"_ZN2pe\d+([a-z_]+)(I?.*)", mangled)
    args = re.findall(r"L[a-z](\d+)E|DenseOpE(\d+)E", m.group(2).split("EEv")[0] + "E")
    return m.group(1) + "<%s>" % ",".join(a or b for a, b in args)


def build(folder):
    """The recording runtime's path, compiled into `folder`; None without a compiler."""
    gxx = shutil.which("g++")
    if gxx is None:
        return None
    out = os.path.join(str(folder), "launch_log.so")
    subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", os.path.join(HERE, "native", "launch_log.cpp"), "-o",
                    out], check=True, capture_output=True, text=True)
    return out


def launches(shim, calls):
    """(names of all the library's kernels, for each call its launches as (name, grid, threads, lds))."""
    r = subprocess.run([sys.executable, os.path.abspath(__file__), shim], input=json.dumps(calls), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    d = json.loads(r.stdout)

    def parse(line):
        name, x, y, z, threads, lds = line.split()
        return readable(name), (int(x), int(y), int(z)), int(threads), int(lds)
    return ([readable(k) for k in d["kernels"]], [[parse(x) for x in c] for c in d["calls"]])


if __name__ == "__main__":
    _main()
