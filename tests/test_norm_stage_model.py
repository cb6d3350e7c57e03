"""CPU model of the norm's rows in stages of shared memory (rmsnorm.cuh, rows that are
on no boundary).

The threads that share a row copy it in 16-byte chunks, chunk by thread, and read it
element by element, so that a chunk's writer and its readers are different threads in
different warps; only block barriers order them.  The model runs the warps one
barrier's stretch at a time, in every order that the barriers allow at the extremes
(each warp in turn as far ahead, and as far behind, as it can get), and checks that
each row's elements are its own.
"""
import pytest

LANES, ELEMENTS, STAGES = 32, 8, 3   # elements of a part and of a 16-byte chunk


def program(warp, threads, dim, phase, rows, stages, read_before_sum, memory, out):
    """One warp: a generator that yields at block barriers."""
    chunks = -(-(phase + dim) // ELEMENTS)
    span = LANES * ELEMENTS           # columns of a warp's part
    mine = [c for c in range(dim) if c // span % (threads // LANES) == warp]

    def copy(row):
        if row < rows:
            for chunk in range(chunks):
                if chunk % threads // LANES == warp:
                    for e in range(ELEMENTS):
                        memory[row % stages][chunk * ELEMENTS + e] = (row, chunk * ELEMENTS + e - phase)

    def read(row):
        return [memory[row % stages][phase + c] for c in mine]

    for row in range(stages - 1):
        copy(row)
    for row in range(rows):
        copy(row + stages - 1)
        yield                         # sync_row: the copies are there
        got = read(row) if read_before_sum else None
        yield                         # row_sum
        out[row] += zip(mine, read(row) if got is None else got)


def run(threads, dim, phase, rows, read_before_sum, order):
    memory = [dict() for _ in range(STAGES)]
    out = [[] for _ in range(rows)]
    warps = [program(w, threads, dim, phase, rows, STAGES, read_before_sum, memory, out)
             for w in range(threads // LANES)]
    alive = True
    while alive:                      # every warp to its next barrier, in this order
        alive = False
        for w in order(len(warps)):
            alive = next(warps[w], "end") != "end" or alive
    return all(sorted(got) == [(c, (row, c)) for c in range(dim)] for row, got in enumerate(out))


ORDERS = [lambda n: range(n), lambda n: reversed(range(n)),
          lambda n: [*range(1, n), 0], lambda n: [n - 1, *range(n - 1)]]


@pytest.mark.parametrize("threads,dim", [(64, 513), (64, 1001), (128, 2047), (256, 4095)])
@pytest.mark.parametrize("phase", [1, 3, 7])
def test_what_is_read_before_the_sum_is_the_rows_own(threads, dim, phase):
    assert all(run(threads, dim, phase, 9, True, order) for order in ORDERS)


@pytest.mark.parametrize("threads,dim", [(64, 1001), (128, 2047)])
def test_what_is_read_behind_it_may_be_another_rows(threads, dim):
    """The model sees the difference."""
    assert not all(run(threads, dim, 1, 9, False, order) for order in ORDERS)
