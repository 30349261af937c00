"""The oracle of shared blocks, by hand."""
import numpy as np

from oracle import prompts as oracle


def test_a_fork_of_an_empty_row_holds_nothing():
    table = np.array([[0, -1], [5, 6], [7, 8]])                # rows 1 and 2 hold no tokens: their entries are of no use
    r = oracle.block_fork(4, table, [3, 0, 0], [0] * 9, [3, 2, 1, -1, -1, -1, -1, -1, -1], 3, [1], [2])
    assert r["table"].tolist() == [[0, -1], [5, 6], [-1, -1]] and r["length"].tolist() == [3, 0, 0]
    assert r["n_free"] == 3 and r["copies"] == [] and not r["bad"] and not r["short"]
