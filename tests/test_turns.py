"""The turns a position of each pair of columns, from the library's own host code, against 80 decimal digits: within a unit of
2^-64 of a turn, half of it the rounding."""
import ctypes
import os
import shutil
import subprocess
from decimal import Decimal, localcontext

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tree_speculative_verification_gdn_gb300",
                    "csrc")
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534")
PROGRAM = '#include "tv_turns.h"\nextern "C" void turns(double t, int r, unsigned long long* f) { tv::turns_of(t, r, f); }\n'


@pytest.fixture(scope="module")
def turns(tmp_path_factory):
    where = tmp_path_factory.mktemp("turns")
    source, lib = where / "turns.cpp", where / "turns.so"
    source.write_text(PROGRAM)
    compiler = shutil.which("g++") or shutil.which("c++")
    subprocess.run([compiler, "-O3", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", str(lib), str(source)], check=True)
    fn = ctypes.CDLL(str(lib)).turns
    fn.argtypes, fn.restype = [ctypes.c_double, ctypes.c_int, ctypes.POINTER(ctypes.c_uint64)], None

    def call(theta, rotary):
        out = (ctypes.c_uint64 * 128)()
        fn(theta, rotary, out)
        return list(out)[:rotary // 2]
    return call


def single(x):
    return ctypes.c_float(x).value      # what the call's argument holds


@pytest.mark.parametrize("rotary", [0, 16, 48, 64, 112, 128, 176, 240, 256])
@pytest.mark.parametrize("theta", [1.0, single(1 + 2.0 ** -23), 2.0, single(3.7), 1e4, 5e5, 1e6, 1e7, single(1e20), single(3.4e38)])
def test_turns(turns, theta, rotary):
    with localcontext() as ctx:
        ctx.prec = 80
        for c, got in enumerate(turns(theta, rotary)):
            want = Decimal(theta) ** (Decimal(-2 * c) / Decimal(rotary)) / (2 * PI) * 2 ** 64
            assert abs(got - want) <= Decimal("0.5000001"), (c, got, want)
