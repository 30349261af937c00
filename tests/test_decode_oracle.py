"""Pins of the decoding oracle (oracle/decode.py) on hand-worked cases (CPU)."""
import math

import numpy as np
import torch

from oracle import decode as o


def test_block_tables_by_hand():
    # blocks of 4: request 0 grows 3 -> 9 (one block -> three), request 1 ends, request 2 asks for too much
    r = o.block_tables(4, 10, [3, 5, 0], [9, 0, 30], [[7, -1, -1, -1, -1, -1, -1, -1], [2, 5] + [-1] * 6, [-1] * 8], [0, 1, 3], 3, 40)
    # pool 0 1 3 | 2 5: taken from the top 5, 2; then request 2 needs 8 of the 3 left
    assert r["table"][0].tolist() == [7, 5, 2, -1, -1, -1, -1, -1] and (r["table"][1:] == -1).all()
    assert r["free"].tolist() == [0, 1, 3] + [-1] * 7 and r["n_free"] == 3 and r["short"]
    assert r["length"].tolist() == [9, 0, 0] and r["cu"].tolist() == [0, 6, 6, 36]
    assert r["slots"][:6].tolist() == [7 * 4 + 3, 20, 21, 22, 23, 8] and (r["slots"][6:] == -1).all()
    assert r["pos"][:8].tolist() == [3, 4, 5, 6, 7, 8, 0, 1]


def test_e4m3_rounding_is_torchs():
    x = np.concatenate([np.random.default_rng(0).standard_normal(2000) * 10.0 ** np.arange(-4, 4).repeat(250),
                        o.e4m3_values()[:127], [0.0, -0.0, 17.0, 19.0, 1e9, -1e9, 448, 464, 2 ** -10, 3 * 2.0 ** -10]])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(o.e4m3_round(x), want)


def test_attention_of_equal_keys_is_the_mean_and_an_empty_row_is_zero():
    v = np.arange(8.0).reshape(4, 1, 2)
    out, lse = o.paged_attention(np.ones((2, 1, 2)), np.zeros((4, 1, 2)), v, [[1, 0], [-1, -1]], 2, [3, 0])
    assert np.allclose(out[0, 0], (v[2, 0] + v[3, 0] + v[0, 0]) / 3) and math.isclose(lse[0, 0], math.log(3))
    assert (out[1] == 0).all() and lse[1, 0] == -math.inf


def test_beam_select_by_hand():
    x = np.array([[[0.0, math.log(3.0)], [0.0, 0.0]]])
    p, t, s, d = o.beam_select(x, np.array([[-1.0, -0.5]]), np.array([[0, 0]]), eos=1)
    # beam 0: -1 + log(1/4), -1 + log(3/4) = -1.288; beam 1: -0.5 + log(1/2) = -1.193 twice (smaller id first)
    assert p.tolist() == [[1, 1]] and t.tolist() == [[0, 1]] and d.tolist() == [[0, 1]]
    assert np.allclose(s, -0.5 - math.log(2))
    p, t, s, d = o.beam_select(np.full((1, 2, 3), -math.inf), np.array([[-1.0, -2.0]]), np.array([[0, 1]]), eos=2)
    assert p.tolist() == [[1, 1]] and t.tolist() == [[2, -1]] and s.tolist() == [[-2.0, -math.inf]] and d.tolist() == [[1, 1]]


def test_beam_reorder_by_hand():
    table = np.array([[[4, 10, -1], [4, 11, -1]]])
    owned = np.array([[4, 8, 9, 10, 11, 12, 13]])          # shared | spares | generated 0 | generated 1
    r = o.beam_reorder(2, np.array([[0, 0]]), np.array([[5, 6]]), [3], [1], owned, table, np.array([[8, 9]]),
                       np.array([[[1, 2, 3, 0], [1, 2, 4, 0]]]))
    assert r["table"].tolist() == [[[4, 10, -1], [4, 9, -1]]] and r["spare"].tolist() == [[8, 11]]
    assert r["copies"] == [(10, 9, 1)] and r["slots"].tolist() == [[21, 19]]
    assert r["hist"].tolist() == [[[1, 2, 3, 5], [1, 2, 3, 6]]]
    r = o.beam_reorder(2, np.array([[1, 0]]), np.array([[5, 6]]), [4], [1], owned, table, np.array([[8, 9]]))
    assert r["table"].tolist() == [[[4, 11, 12], [4, 10, 13]]] and r["copies"] == [] and r["slots"].tolist() == [[24, 26]]
