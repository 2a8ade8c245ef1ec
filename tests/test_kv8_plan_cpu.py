"""The page plan's reference at the rule that no request overtakes an earlier one that found no room."""
import numpy as np

import kv8_reference as ref


def test_a_later_request_does_not_overtake():
    """Requests of 2, 20 and 1 rows, two free pages, six rows: the second needs two pages and one is left (2); the sum
    of rows over it and the third is 23 > 6, so the third, which needs no page, finds no rows either (3)."""
    table, off, kl, pos, slot, used, st = ref.plan([15, 0, 3], [2, 20, 1], [7, 8], np.array([[1, -1], [-1, -1], [2, -1]]),
                                                   16, 6)
    assert st.tolist() == [0, 2, 3]
    assert kl.tolist() == [17, 0, 3] and off.tolist() == [0, 2, 2, 2]
    assert pos.tolist() == [15, 16, -1, -1, -1, -1] and slot.tolist() == [31, 112, -1, -1, -1, -1]
    assert used.tolist() == [1] and table.tolist() == [[1, 7], [-1, -1], [2, -1]]


def test_a_request_that_needs_neither_page_nor_row_is_admitted():
    _, off, kl, _, _, used, st = ref.plan([15, 0, 3, 4], [2, 20, 0, 13], [7, 8], np.full((4, 2), 5), 16, 40)
    assert st.tolist() == [0, 2, 0, 2] and kl.tolist() == [17, 0, 3, 4] and used.tolist() == [1] and off[-1] == 2
