"""Which tiles take a prompt call: the choice is made on the host from the sizes, without the lengths (no
GPU)."""
import ctypes

import pytest

import dequant_gemv_q4_amd as q


@pytest.fixture(scope="module")
def in_16s():
    q.lib()
    fn = ctypes.CDLL(q.LIB_PATH)["_ZN2qg13prompt_in_16sEliiiil"]
    fn.restype = ctypes.c_bool
    fn.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int64]
    return fn


@pytest.mark.parametrize("rows,nq,nkv,hd,table", [
    (585, 12, 2, 128, 30600), (177, 24, 2, 128, 30200), (369, 12, 2, 128, 30400), (177, 24, 2, 128, 12200),
    (180, 32, 8, 128, 30200), (177, 16, 1, 64, 30200)])
def test_idle_and_one_row_sequences_do_not_move_a_chunk_to_the_small_tiles(in_16s, rows, nq, nkv, hd, table):
    """A chunk behind a long cache: alone it takes the 128-row tiles, and so it does beside any number of
    sequences with one row or none."""
    assert not in_16s(rows, 1, nq, nkv, hd, table)
    for idle in range(1, 1024):
        assert not in_16s(rows, 1 + idle, nq, nkv, hd, table)
        assert not in_16s(rows + idle, 1 + idle, nq, nkv, hd, table)


@pytest.mark.parametrize("rows,n_seq,nq,nkv,hd,table,small", [
    (93, 3, 12, 2, 128, 80, True), (64, 16, 32, 8, 128, 4032, True), (32, 1, 12, 2, 128, 20000, True),
    (128, 1, 12, 2, 128, 20000, False), (128, 1, 32, 8, 128, 144, True), (512, 16, 32, 8, 128, 64, False),
    (4, 1, 128, 8, 128, 1 << 24, True), (128, 4, 12, 2, 128, 2064, True), (203, 1, 12, 2, 128, 30240, False),
    (8192, 1, 32, 8, 128, 8320, False), (1 << 20, 1024, 1024, 1, 256, 1 << 24, False)])
def test_choice(in_16s, rows, n_seq, nq, nkv, hd, table, small):
    assert in_16s(rows, n_seq, nq, nkv, hd, table) == small
