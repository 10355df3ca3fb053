"""Layer norm's choice of kernel, on the host: on a GPU and on parts of one."""
import ctypes

import pytest

F32, BF16, F16 = 0, 1, 2
WHOLE, SHIFTED, SINGLE, STREAM = range(4)


def choice(lib, rows, cols, dtype, backward, keep, begin, ld, sms, clusters):
    out = [ctypes.c_int(-1) for _ in range(4)]
    st = lib.sgemm_layer_norm_choose_check(rows, cols, dtype, backward, keep, begin, ld, sms, clusters,
                                           *map(ctypes.byref, out))
    return tuple(v.value for v in out) if st == 0 else st


SIZES = [1, 64, 255, 1000, 2047, 4096, 4097, 5001, 8184, 8191, 9001, 12001, 16384, 16393, 20003, 33000, 65537, 100001]


@pytest.mark.parametrize("sms", [1, 2, 7, 8, 9, 18, 19, 38, 76, 152])
def test_every_call_has_a_kernel(lib, sms):
    """Each of a call's sets of blocks has rows that begin at one place, there is a set at least, and no
    more clusters than there is room for."""
    for dtype, elem in ((F32, 4), (BF16, 2), (F16, 2)):
        for cols in SIZES:
            for rows in (1, 5, 300, 1000, 20000):
                for begin, pad in ((0, 0), (elem, 0), (0, 1), (elem, 3), (2 * elem, 8)):
                    for backward, keep in ((0, 0), (0, 1), (1, 0)):
                        for clusters in {0, 1, 3, sms // 8, sms // 4, sms // 2}:
                            ld = cols + pad
                            access, places, blocks, sets = choice(lib, rows, cols, dtype, backward, keep, begin, ld,
                                                                  sms, clusters)
                            at = (rows, cols, dtype, backward, begin, ld, clusters)
                            assert sets >= 1, at
                            if access == SHIFTED:
                                n = next(n for n in (1, 2, 4, 8) if ld * elem * n % 16 == 0)
                                assert places == n and (sets % n == 0 or rows <= sets), at
                            if access == WHOLE:
                                assert begin == 0 and (rows == 1 or ld * elem % 16 == 0), at
                            if blocks > 1:
                                assert backward and blocks in (2, 4, 8) and sets <= min(clusters, sms // blocks), at
                            if access != STREAM and backward:
                                assert sets <= 2 * sms, at          # the workspace's rows


def test_choices_of_the_whole_gpu(lib):
    """152 SMs: what the GPU tests run."""
    whole = lambda *a: choice(lib, *a, 152, 76)
    assert whole(1000, 5001, BF16, 0, 0, 2, 5001) == (SHIFTED, 8, 1, 152)
    assert whole(1000, 5001, BF16, 1, 0, 2, 5001) == (SHIFTED, 8, 1, 152)
    assert whole(1000, 20003, BF16, 1, 0, 2, 20003)[:3] == (SHIFTED, 8, 4)
    assert whole(1000, 9001, F32, 1, 0, 4, 9001)[:3] == (SINGLE, 1, 4)
    assert whole(1000, 16384, BF16, 1, 0, 0, 16384) == (WHOLE, 1, 2, 76)
    assert whole(1000, 100001, BF16, 1, 0, 0, 100001)[0] == STREAM
    assert whole(1000, 20003, BF16, 0, 0, 2, 20003)[0] == STREAM


def test_few_clusters(lib):
    """Shifted rows with room for fewer clusters than their eight places, and for none."""
    few = lambda sms, clusters: choice(lib, 1000, 20003, BF16, 1, 0, 2, 20003, sms, clusters)
    assert few(76, 9) == (SHIFTED, 8, 4, 8)
    assert few(18, 4) == (SINGLE, 1, 8, 2)           # of eight blocks: two fit on 18 SMs
    assert few(18, 0)[0] == STREAM and few(2, 0)[0] == STREAM
    assert choice(lib, 1000, 5001, BF16, 0, 0, 2, 5001, 7, 3)[0] == SINGLE


@pytest.mark.parametrize("args", [(0, 8, 0, 0, 0, 0, 8, 152, 76), (8, 0, 0, 0, 0, 0, 8, 152, 76), (8, 8, 5, 0, 0, 0, 8, 152, 76),
                                  (8, 8, 0, 0, 0, 16, 8, 152, 76), (8, 8, 0, 0, 0, 2, 8, 152, 76), (8, 8, 0, 0, 0, 0, 7, 152, 76),
                                  (8, 8, 0, 0, 0, 0, 8, 0, 76), (8, 8, 0, 0, 0, 0, 8, 152, -1), (-1, 8, 0, 0, 0, 0, 8, 152, 76)])
def test_refusals(lib, args):
    assert choice(lib, *args) == -1
    assert lib.sgemm_layer_norm_choose_check(8, 8, 0, 0, 0, 0, 8, 152, 76, None, None, None, None) == -1
