"""A result in a momentum buffer would replace the momentum that the next step goes on from: it is
refused on the host, whichever of the call's matrices it is. (The library goes on to the
workspace's size, here too small, where nothing is shared.)"""
import ctypes
import os

import pytest

import activation_sparse_feedforward_gb300 as tw
from activation_sparse_feedforward_gb300 import _lib

BIG = 1 << 40  # far between the fake matrices


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tw.lib_path()):
        from activation_sparse_feedforward_gb300.build import build
        build()
    return tw.load()


def _call(lib, out, buffers, otype=_lib.TW_F32, ldo=64, ldb=64, m=64, n=64):
    at = lambda p: (ctypes.c_void_p * len(p))(*p)  # noqa: E731
    coef = (ctypes.c_float * 15)(*[3.4445, -4.775, 2.0315] * 5)
    grads = [BIG * (9 + i) for i in range(len(out))]
    return lib.tw_orthogonalize(at(grads), 64, _lib.TW_F32, at(buffers), ldb, 0.9, 1, len(out), m, n, 5, coef, 1.0, 0.0,
                                at(out), ldo, otype, 4096, 1, 4096, None)


def test_a_result_in_a_buffer_is_refused(lib):
    ok, bad = _lib.TW_EWORKSPACE, _lib.TW_EINVAL
    size = 4 * 64 * 64
    assert _call(lib, [BIG], [2 * BIG]) == ok
    assert _call(lib, [BIG], [BIG]) == bad
    assert _call(lib, [BIG, 2 * BIG], [3 * BIG, BIG]) == bad and _call(lib, [BIG, 2 * BIG], [2 * BIG, 3 * BIG]) == bad
    assert _call(lib, [BIG + size - 4], [BIG]) == bad and _call(lib, [BIG + size], [BIG]) == ok
    assert _call(lib, [BIG - size // 2], [BIG], otype=_lib.TW_BF16) == ok       # 16 bits: half as long
    assert _call(lib, [BIG - size // 2 + 2], [BIG], otype=_lib.TW_BF16) == bad
    assert _call(lib, [BIG + 256], [BIG], ldo=128, ldb=128) == ok               # columns of one larger matrix
    assert _call(lib, [BIG + 252], [BIG], ldo=128, ldb=128) == bad
