"""The append's table of rotation frequencies (csrc/turns.h), against decimal arithmetic."""
import ctypes
import pathlib
import shutil
import subprocess
from decimal import Decimal, localcontext

import numpy as np
import pytest

CSRC = pathlib.Path(__file__).resolve().parents[1] / "paged_kv_decode_pagetable_gb300" / "csrc"


@pytest.fixture(scope="module")
def table(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("turns")
    (d / "t.cpp").write_text(
        f'#include "{CSRC / "turns.h"}"\n'
        'extern "C" void table(float theta, int pairs, int D, uint64_t *f) {\n'
        "  pkv::rotation_turns(theta, pairs, D, f);\n}\n")
    subprocess.run([cxx, "-O3", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-o",
                    d / "t.so", d / "t.cpp"], check=True)
    lib = ctypes.CDLL(str(d / "t.so"))

    def f(theta, pairs, D):
        out = (ctypes.c_uint64 * (D // 2))(*[7] * (D // 2))
        lib.table(ctypes.c_float(theta), pairs, D, out)
        return list(out)
    return f


def atan_inverse(n):
    x = Decimal(1) / n
    total, term, k = x, x, 1
    while abs(term) > Decimal(10) ** -100:
        term = -term / (n * n)
        total += term / (k + 2)
        k += 2
    return total


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("theta", [2.0 ** -56, 3e-17, 1e-9, 0.3, 0.5, 0.99999994, 1.0, 1.0000001,
                                   4.0, 500.0, 1e4, 5e5, 1e6, 8e6, 1e9, 2.0 ** 64, 3.4e38])
def test_table(table, D, theta):
    got = table(theta, D // 2, D)
    theta = float(np.float32(theta))
    with localcontext() as c:
        c.prec = 120
        two_pi = 2 * (16 * atan_inverse(5) - 4 * atan_inverse(239))
        ln = Decimal(theta).ln()
        for i, f in enumerate(got):
            x = (-ln * 2 * i / D).exp() / two_pi
            off = abs(Decimal(f) / 2 ** 64 - x % 1)
            # cut off at 64 places, and 2^-114 of the value
            assert min(off, 1 - off) <= Decimal(2) ** -64 + x * Decimal(2) ** -114, (i, f)


def test_pairs_that_do_not_turn_are_left(table):
    assert table(1e4, 5, 64)[5:] == [7] * 27 and table(1e4, 0, 64) == [7] * 32


def test_theta_of_one_turns_all_pairs_alike(table):
    assert len(set(table(1.0, 256, 512))) <= 2      # (a last place)


@pytest.mark.parametrize("theta", [1.3e-17, 1e-38, 1e-45])
def test_the_append_refuses_smaller_ones(theta):
    pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")
    A = 1 << 20        # an address that nothing follows
    assert pkv.load_library().tree_qkv_norm_rope_append(
        A, A, A, 256, 128, 128, A, A, A, A, A, A, theta, 1e-6, 64, 0, 2, 5, 4, 2, 64, A, 3, 2, 16,
        4, A, A, A, None, None) == pkv.PKV_E_BAD_ARG
    assert b"theta" in pkv.load_library().pkv_last_error()
