"""Which kernel form a product's sizes take (csrc/matmul_plan.hpp): the sizes that the GPU tests run by form are of the
forms they are named for, and every form that some size takes has one."""
import ctypes
import itertools

import pytest

import product_forms as pf


@pytest.fixture(scope="module")
def lib():
    return pf.plans()


def test_sizes_take_the_forms_they_are_named_for(lib):
    for kind, M, K, N, dtype, pad, name in pf.FORMS:
        assert pf.form(lib, kind, M, K, N, dtype, pad) == name, (kind, M, K, N, dtype, pad)


def test_no_form_is_without_a_size(lib):
    lengths = [1, 24, 77, 264, 520, 1032, 1037, 2049, 2056, 4100, 4101, 8200, 16384]
    for kind, dtype in itertools.product(("forward", "dx", "dw"), ("bf16", "f32")):
        named = {f[-1] for f in pf.FORMS if f[0] == kind and f[4] == dtype}
        for M, K, N, pad in itertools.product(lengths, lengths, lengths, (0, 1)):
            name = pf.form(lib, kind, M, K, N, dtype, pad)
            assert name in named, (kind, M, K, N, dtype, pad, name)


def test_timed_sizes(lib):
    """Sizes whose times the documentation has, and the forms that those were measured of."""
    for M, K, N, dtype, name in [(1, 4096, 16384, "bf16", "few 1x1 long aligned"), (203, 1001, 517, "f32", "64 any parts"),
                                 (8192, 8192, 8192, "bf16", "256 aligned"), (4096, 4095, 4096, "bf16", "256 aligned copied"),
                                 (64, 4096, 16384, "bf16", "64 aligned parts"), (100352, 256, 256, "bf16", "128 aligned")]:
        assert pf.form(lib, "forward", M, K, N, dtype) == name
    for kind, M, K, N, name in [("dx", 8192, 4096, 4096, "256 aligned"), ("dw", 8192, 4096, 4096, "256 aligned"),
                                ("dx", 100352, 256, 64, "128 aligned"), ("dw", 100352, 256, 64, "64 aligned parts")]:
        assert pf.form(lib, kind, M, K, N, "bf16") == name


def test_tiles_of_256_are_never_split(lib):
    """No kernel is built that would write their parts."""
    out = (ctypes.c_int * 3)()
    sizes = [129, 256, 257, 1024, 4096, 4097, 16384, 65536, 1 << 20, 1 << 24]
    seen = 0
    for rows, cols, K, es in itertools.product(sizes, sizes, [513, 1025, 4096, 1 << 20, 1 << 24], (2, 4)):
        lib.plan_tiles(rows, cols, K, es, 1, out)
        seen += out[0] == 256
        assert out[0] != 256 or out[1] == 1, (rows, cols, K, es)
    assert seen
