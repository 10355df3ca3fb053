"""The product's choice of tile and split, on the host."""
import ctypes

import pytest


def choice(lib, M, N, K, sms=152):
    tile, split = ctypes.c_int(), ctypes.c_int()
    st = lib.sgemm_mx4_choose_check(M, N, K, sms, ctypes.byref(tile), ctypes.byref(split))
    return (tile.value, split.value) if st == 0 else st


@pytest.mark.parametrize("sms", [152, 148, 64])
def test_choices_fit(lib, sms):
    """Tiles hold the rows they are for, parts keep four slabs of 256 columns and fit the SMs,
    and every kind is chosen somewhere."""
    seen = set()
    sizes = [1, 15, 16, 17, 32, 33, 64, 65, 128, 129, 500, 1280, 4096, 16384, 100000]
    for M in sizes:
        for N in sizes:
            for K in (1, 64, 1000, 2048, 4097, 7937, 16384, 65536):
                tile, split = choice(lib, M, N, K, sms)
                seen.add((tile, split))
                rows = tile if tile != 256 else 256
                tiles = -(-N // (128 if tile != 256 else 256)) * -(-M // rows)
                assert tile >= min(M, 16) and (M > 32 or tile == (16 if M <= 16 else 32))
                assert split == 1 or (tile <= 64 and tiles * split <= sms and
                                      -(-K // 256) >= 4 * split)
                assert tile != 256 or (M > 128 and N > 128)
    assert {t for t, _ in seen} == {16, 32, 64, 128, 256}
    assert {s for t, s in seen if t == 64} == {1, 2, 4, 8}


def test_refusals(lib):
    t = ctypes.c_int()
    for args in ((0, 1, 1, 152), (1, 0, 1, 152), (1, 1, 0, 152), (1, 1, 1, 0)):
        assert choice(lib, *args) == -1
    assert lib.sgemm_mx4_choose_check(1, 1, 1, 152, None, ctypes.byref(t)) == -1
    assert choice(lib, 2**30 + 1, 1, 1) == -4
