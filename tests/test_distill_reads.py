"""The distillation gradient's vector loads stay inside a row's logits, by a host walk of the
kernel's own index arithmetic (the last row of a tensor may end where its memory ends)."""
import ctypes

import pytest

import deterministic_gradient_reduction_gb300 as dgr


@pytest.fixture(scope="module")
def L():
    dgr.build()
    return dgr.lib()


def reads(L, dtype, V, z_at, dz_at, ctas):
    end = ctypes.c_int64(-1)
    assert L.dgr_diag_distill_reads(dtype, V, z_at, dz_at, ctas, ctypes.byref(end)) == 0
    return end.value


@pytest.mark.parametrize("ctas", [1, 2, 4, 8])
@pytest.mark.parametrize("V", [1, 3, 7, 8, 9, 15, 16, 17, 33, 100, 1023, 4097, 20000, 20001, 32768, 50001, 65536])
@pytest.mark.parametrize("dtype", [0, 1])
def test_no_load_passes_the_row(L, dtype, V, ctas):
    vec = 8 if dtype else 4
    for z_at in range(vec):
        for dz_at in range(vec):
            end = reads(L, dtype, V, z_at, dz_at, ctas)
            assert end <= V, (z_at, dz_at, end)


@pytest.mark.parametrize("dtype,vec", [(0, 4), (1, 8)])
def test_every_whole_vector_is_read(L, dtype, vec):
    assert reads(L, dtype, 1024, 0, 0, 1) == 1024
    assert reads(L, dtype, 1024, 0, 1, 4) == 1024      # made of two neighbours
    assert reads(L, dtype, vec - 1, 0, 0, 1) == 0      # single elements only


def test_refusals(L):
    end = ctypes.c_int64(-1)
    for args in ((2, 100, 0, 0, 1), (1, 0, 0, 0, 1), (1, (1 << 20) + 1, 0, 0, 1), (1, 100, 8, 0, 1), (0, 100, 0, 4, 1),
                 (1, 100, -1, 0, 1), (1, 100, 0, 0, 0), (1, 100, 0, 0, 9)):
        assert L.dgr_diag_distill_reads(*args, ctypes.byref(end)) == 1
    assert L.dgr_diag_distill_reads(1, 100, 0, 0, 1, None) == 1
    assert end.value == -1
