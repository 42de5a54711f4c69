"""dspark_block_attention refuses an out that overlaps q: a row tile's queries may
be read by several workers, of which one may have written its rows already (no
compute calls here)."""
import pytest

from speculative_decoding_draft_head_gb300 import binding

P = 1 << 20
ROWS, HEADS, D = 5, 4, 64
ROW = HEADS * D * 2      # bytes of a packed row


def _attend(q, out, q_stride=HEADS * D, rows=ROWS):
    c = binding._CacheStruct(P, P, P, P, P, 8, 2, 32, D, 0)
    lib = binding.load()
    st = lib.dspark_block_attention(c, q, q_stride, 0, HEADS, P, rows, 2, P, 4, P, None, 0, 0, 0, None, 0.125, out, None,
                                    P, 1 << 30, None)
    return st, lib.dspark_last_error().decode()


@pytest.mark.parametrize("out", [P, P + 16, P + (ROWS - 1) * ROW, P - 16, P - (ROWS - 1) * ROW])
def test_an_overlapping_out_is_refused(out):
    st, err = _attend(P, out)
    assert st == 1 and "overlap" in err


def test_a_strided_q_reaches_to_its_last_row():
    st, err = _attend(P, P + 3 * 2 * ROW, q_stride=2 * HEADS * D)
    assert st == 1 and "overlap" in err
