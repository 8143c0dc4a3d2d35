"""The four further bits of a stored state, there and back on the host, for every lower half of a
float32 and rounding to nearest even."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from linear_rnn_sequence_amd import build as hbuild

SOURCE = """
#include "gated_delta_kept.h"
extern "C" void round_trip(const unsigned *x, const unsigned *hi, unsigned *out, int n) {
    for (int i = 0; i < n; ++i) {
        const int at = i & 7;  // its place in a word, between others
        unsigned word = 0x5a5a5a5au & ~(15u << 4 * at);
        word |= gdr::kept_code(x[i]) << 4 * at;
        out[i] = gdr::kept_bits(hi[i], word, at);
    }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    at = tmp_path_factory.mktemp("kept")
    (at / "kept.hip").write_text(SOURCE)
    out = at / "kept.so"
    subprocess.run(["hipcc", "--offload-host-only", "-O1", "-std=c++17", "-fPIC", "-shared", "-I", hbuild.CSRC,
                    str(at / "kept.hip"), "-o", str(out)], check=True, capture_output=True)
    L = ctypes.CDLL(str(out))
    L.round_trip.argtypes = [ctypes.c_void_p] * 3 + [ctypes.c_int]
    L.round_trip.restype = None
    return L


def nearest_even(x):
    """bf16 bits, in the upper half, of float32 bits."""
    x = x.astype(np.uint64)
    return ((x + 0x7fff + (x >> 16 & 1)) & 0xffff0000).astype(np.uint32)


def there_and_back(lib, x):
    hi, out = nearest_even(x), np.empty_like(x)
    lib.round_trip(x.ctypes.data, hi.ctypes.data, out.ctypes.data, len(x))
    return out


# upper halves: even and odd, both signs, next to a power of two, the smallest and largest normal numbers
@pytest.mark.parametrize("upper", [0x3f80, 0x3f81, 0xbf80, 0xbf81, 0x3fff, 0x407e, 0x0080, 0x8081, 0x7f7e, 0xff7d])
def test_every_lower_half(lib, upper):
    x = np.arange(1 << 16, dtype=np.uint32) | np.uint32(upper << 16)
    a, b = (y.view(np.float32).astype(np.float64) for y in (there_and_back(lib, x), x))
    assert np.isfinite(a).all()
    assert (np.abs(a - b) <= 2.0 ** -12 * np.abs(b)).all()


@pytest.mark.parametrize("upper", [0x0000, 0x8000, 0x0001, 0x807f])
def test_numbers_below_the_smallest_normal_one(lib, upper):
    """Their last bits are 2^-149: off by 2^11 of those."""
    x = np.arange(1 << 16, dtype=np.uint32) | np.uint32(upper << 16)
    a, b = (y.view(np.float32).astype(np.float64) for y in (there_and_back(lib, x), x))
    assert np.isfinite(a).all()
    assert (np.abs(a - b) <= 2.0 ** (11 - 149)).all()


def test_what_is_no_number_stays_none(lib):
    x = np.array([0x7f800000, 0xff800000, 0x7fc00000, 0xffc00001, 0x7fc0ffff, 0x7fff8000 - 1], np.uint32)
    assert not np.isfinite(there_and_back(lib, x).view(np.float32)).any()


def test_numbers_that_round_to_infinity_do_not_become_it(lib):
    x = np.arange(0x7f7f8000, 0x7f800000, 17, dtype=np.uint32)
    a, b = (y.view(np.float32).astype(np.float64) for y in (there_and_back(lib, x), x))
    assert (np.abs(a - b) <= 2.0 ** -12 * b).all()


def test_float16_values(lib):
    x = np.arange(0x0400, 0x7c00, dtype=np.uint16).view(np.float16).astype(np.float32)
    a = there_and_back(lib, x.view(np.uint32)).view(np.float32).astype(np.float64)
    assert (np.abs(a - x) <= 2.0 ** -12 * x).all()
