"""Which outputs overlap an input, on the CPU: every pair of small matrices in
one buffer against the sets of their bytes.  A pair that shares none may be
refused only where the two have more than one row each and different strides."""
from __future__ import annotations

import copy_reduce_snac_amd as snac

BASE = 0x100000


def cells(at, rows, width, ld):
    return {at + r * ld + c for r in range(rows) for c in range(width)}


def refused(src, dst, rows_src, rows_dst, width, ld_src, ld_dst) -> bool:
    """Whether snac_combine_backward refuses dy over y (f32 elements; of no token, so nothing is launched)."""
    far = 1 << 44
    try:
        snac.snac_combine_backward(far, width, BASE + 4 * src, ld_src, rows_src, 2 * far, 3 * far, 0, 1, width, "f32",
                                   BASE + 4 * dst, ld_dst, 4 * far)
    except snac.SnacError as e:
        assert e.status == snac.SNAC_E_ARG and "overlaps" in str(e), str(e)
        return True
    return False


def test_every_small_pair():
    shared = apart = 0
    for width in (1, 2, 3):
        for rows in (1, 2, 4):
            for ld_src in {width, width + 1, 2 * width, 7}:
                for ld_dst in {ld_src, width, 7}:
                    for dst in range(0, 40):
                        src = 16
                        if src == dst and ld_src == ld_dst:
                            continue  # in place
                        a, b = cells(src, rows, width, ld_src), cells(dst, rows, width, ld_dst)
                        got = refused(src, dst, rows, rows, width, ld_src, ld_dst)
                        if a & b:
                            shared += 1
                            assert got, (width, rows, ld_src, ld_dst, dst)
                        elif rows == 1 or ld_src == ld_dst:
                            apart += 1
                            assert not got, (width, rows, ld_src, ld_dst, dst)
    assert shared > 500 and apart > 500


def one_row(at_x, at_out, rows_x, rows_out, width, ld_x, ld_out) -> bool:
    """Whether snac_dispatch refuses x over out; topk 1, slots far away."""
    far = 1 << 44
    try:
        snac.snac_dispatch(BASE + 4 * at_x, ld_x, far, rows_x, 1, width, "f32", BASE + 4 * at_out, ld_out, rows_out)
    except snac.SnacError as e:
        if e.status == snac.SNAC_E_ARG:
            assert "overlaps" in str(e), str(e)
            return True
    return False


def test_one_row_of_a_wider_matrix():
    """A decode step's one row beside the columns that are written: rows of 16 in a buffer of rows of 40."""
    import torch

    if torch.cuda.is_available():
        return  # the addresses are no memory: checks only, where nothing can be launched
    for row in (0, 3, 7):
        for ld_x in (16, 40, 999):
            assert not one_row(40 * row, 20, 1, 8, 16, ld_x, 40)
            assert not one_row(40 * row + 20, 0, 1, 8, 16, ld_x, 40)
            assert one_row(40 * row + 10, 20, 1, 8, 16, ld_x, 40)
            assert one_row(40 * row + 30, 0, 1, 9, 16, ld_x, 40) == (row < 8)  # it runs on into the next row's columns
            assert not one_row(20, 40 * row, 8, 1, 16, 40, ld_x)
            assert one_row(20, 40 * row + 5, 8, 1, 16, 40, ld_x)
