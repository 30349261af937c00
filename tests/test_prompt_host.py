"""What decode.py hands to the calls for prompts and samples, and makes of their answers, on CPU tensors (prompt_library)."""
import numpy as np
import pytest
import torch

import prompt_library
from eagle_speculative_decoding_step_gb300 import decode


@pytest.fixture(autouse=True)
def on_cpu(monkeypatch):
    prompt_library.use(monkeypatch)


def model(seed=3):
    return decode.RandomModel(layers=2, hidden=64, nq=4, nkv=2, hd=16, inter=96, vocab=203, max_len=256, dtype="f32",
                              device="cpu", seed=seed)


def cache_of(m, blocks=60, bs=4, rows=8):
    return decode.PagedCache(2, blocks, bs, m.nq, m.nkv, m.hd, dtype="f32", max_rows=rows, device="cpu")


def one_by_one(m, tokens):
    """Logits after each of a request's tokens, fed one a step."""
    b = decode.Batch(m, cache_of(m), 1, 64, m.vocab)
    return torch.cat([b.feed(torch.tensor([t], dtype=torch.int32)) for t in tokens])


def prompts(*lengths, seed=0):
    r = np.random.default_rng(seed)
    return [r.integers(0, 203, n).tolist() for n in lengths]


@pytest.mark.parametrize("chunk", [1, 3, 4, 5, 512])
def test_a_prompt_in_chunks_is_the_prompt_token_by_token(chunk):
    m, p = model(), prompts(9, 1, 0, 14)
    b = decode.Batch(m, cache_of(m), 4, 64, m.vocab)
    out = b.extend(p, chunk=chunk)
    assert b.error() == 0 and b.length.tolist() == [9, 1, 0, 14]
    for i in (0, 1, 3):
        torch.testing.assert_close(out[i], one_by_one(m, p[i])[-1], atol=1e-4, rtol=1e-4)
    assert (out[2] == 0).all()
    # and it goes on as one that was fed token by token
    more = b.extend([[5], [], [7, 8], [6, 1, 2]], chunk=chunk)
    for i, t in ((0, p[0] + [5]), (2, [7, 8]), (3, p[3] + [6, 1, 2])):
        torch.testing.assert_close(more[i], one_by_one(m, t)[-1], atol=1e-4, rtol=1e-4)
    assert (more[1] == 0).all() and b.length.tolist() == [10, 1, 2, 17]


@pytest.mark.parametrize("chunk", [2, 5, 100])
def test_scores_of_a_prompt(chunk):
    m, p = model(), prompts(7, 1, 12, 0)
    b = decode.Batch(m, cache_of(m), 4, 64, m.vocab)
    scores = b.score(p, k=3, chunk=chunk)
    assert b.error() == 0 and scores[3] == {}
    for i in (0, 1, 2):
        logp = torch.log_softmax(one_by_one(m, p[i]).double(), -1)
        s, n = scores[i], len(p[i])
        assert s["logprob"].shape == (n,) and s["top_ids"].shape == (n, 3)
        want = logp[torch.arange(n - 1), torch.tensor(p[i][1:], dtype=torch.long)].float()
        torch.testing.assert_close(s["logprob"][:-1], want, atol=1e-4, rtol=1e-4)
        assert s["logprob"][-1] == -float("inf") and s["rank"][-1] == -1
        assert (s["top_ids"][:, 0].long() == logp.argmax(-1)).all()
        torch.testing.assert_close(s["entropy"], -(logp.exp() * logp).sum(-1).float(), atol=1e-4, rtol=1e-4)
        for r, t, row in zip(s["rank"][:-1].tolist(), p[i][1:], logp):
            assert r == int((row > row[t]).sum())


def test_forks_decode_as_requests_of_their_own():
    m, p = model(), prompts(10, 8)
    b = decode.Batch(m, cache_of(m), 6, 64, m.vocab)
    b.extend(p + [[]] * 4)
    b.drop([2, 3, 4, 5])                                       # (they hold nothing)
    held = b.cache.num_blocks - int(b.cache.n_free)
    b.fork([0, 0, 1], [2, 4, 5])
    # 10 tokens: two full blocks are shared, a partial one is copied; 8 tokens: nothing is
    assert b.cache.num_blocks - int(b.cache.n_free) == held + 2
    first = torch.tensor([1, 2, 3, 0, 4, 5], dtype=torch.int32)
    out = b.decode(first, 6)
    assert b.error() == 0
    for row, src in ((0, 0), (2, 0), (4, 0), (1, 1), (5, 1)):
        c = decode.Batch(m, cache_of(m), 1, 64, m.vocab)
        c.extend([p[src]])
        assert out[row].tolist() == c.decode(first[row:row + 1], 6)[0].tolist()
    assert b.length.tolist() == [16, 14, 16, 0, 16, 14]
    # a dropped row gives back what no other holds
    b.drop([0])
    c = decode.Batch(m, cache_of(m), 1, 64, m.vocab)
    c.extend([p[0]])
    ref = c.decode(first[2:3], 9)[0, 6:]
    torch.testing.assert_close(b.decode(out[:, -1].contiguous(), 3)[2], ref)
    b.release()
    assert int(b.cache.n_free) == b.cache.num_blocks and int(b.cache.shared.sum()) == 0
    assert sorted(b.cache.free.tolist()) == list(range(b.cache.num_blocks)) and b.error() == 0


def test_requests_that_end_leave_their_forks_alone():
    """The end token of one sample gives back its own blocks, not the prompt's."""
    m, p = model(), prompts(9)
    free = decode.Batch(m, cache_of(m), 3, 64, m.vocab)
    free.extend(p + [[], []])
    free.drop([1, 2])
    free.fork([0, 0], [1, 2])
    first = torch.tensor([7, 8, 9], dtype=torch.int32)
    seen = free.decode(first, 8)
    eos = int(seen[0, 2])                                      # where the first sample will end
    b = decode.Batch(m, cache_of(m), 3, 64, m.vocab, eos=eos)
    b.extend(p + [[], []])
    b.drop([1, 2])
    b.fork([0, 0], [1, 2])
    out = b.decode(first, 8)
    for row in range(3):
        want = seen[row].tolist()
        if eos in want:
            want = want[:want.index(eos) + 1]
        assert out[row].tolist()[:len(want)] == want
    assert b.error() == 0
    b.release()
    assert sorted(b.cache.free.tolist()) == list(range(b.cache.num_blocks))


def test_compaction_changes_no_answer():
    m, p = model(), prompts(9, 13, 6)
    got = []
    for compact in (False, True):
        b = decode.Batch(m, cache_of(m), 4, 64, m.vocab)
        b.extend(p + [[]])
        b.drop([0, 3])
        b.fork([1], [3])
        if compact:
            b.compact()
            used = sorted({int(i) for row, n in zip(b.table, b.length) for i in row[:-(-int(n) // 4)]})
            assert used == list(range(len(used))) and int(b.cache.n_free) == b.cache.num_blocks - len(used)
        got.append(b.decode(torch.tensor([0, 5, 6, 7], dtype=torch.int32), 7)[1:])
        assert b.error() == 0
    assert torch.equal(*got)


def test_a_cache_with_another_batch_is_not_compacted():
    m = model()
    c = cache_of(m)
    b, other = (decode.Batch(m, c, 1, 64, m.vocab) for _ in range(2))
    b.extend([[1, 2, 3]])
    other.extend([[4, 5, 6, 7, 8]])
    table = b.table.clone()
    b.compact()
    assert b.error() != 0 and torch.equal(b.table, table)


def test_a_row_takes_another_request_after_it_was_dropped():
    m, p = model(), prompts(5, 6)
    b = decode.Batch(m, cache_of(m), 2, 64, m.vocab)
    b.extend(p)
    b.drop([1])
    out = b.extend([[], [3, 4, 5]])
    torch.testing.assert_close(out[1], one_by_one(m, [3, 4, 5])[-1], atol=1e-4, rtol=1e-4)
    assert b.length.tolist() == [5, 3] and b.error() == 0


def test_a_request_that_the_pool_cannot_serve_stops_and_leaves_the_others_right():
    m, p = model(), prompts(6, 30, 5)
    b = decode.Batch(m, cache_of(m, blocks=6), 3, 64, m.vocab)
    out = b.extend(p, chunk=8)
    assert b.error() != 0 and b.stopped.tolist() == [False, True, False]
    for i in (0, 2):
        torch.testing.assert_close(out[i], one_by_one(m, p[i])[-1], atol=1e-4, rtol=1e-4)
    b = decode.Batch(m, cache_of(m, blocks=4), 3, 64, m.vocab)
    b.extend([p[0], [], []])
    b.drop([1, 2])
    b.fork([0, 0, ], [1, 2])                                   # two blocks left, one each
    assert b.length.tolist() == [6, 6, 6] and b.error() == 0
    c = decode.Batch(m, cache_of(m, blocks=3), 3, 64, m.vocab)
    c.extend([p[0], [], []])
    c.drop([1, 2])
    c.fork([0, 0], [1, 2])
    assert c.length.tolist() == [6, 6, 0] and c.error() != 0 and c.live.tolist() == [1, 1, 0]


def test_refusals():
    m = model()
    b = decode.Batch(m, cache_of(m), 2, 64, m.vocab)
    for call in (lambda: b.extend([[1]]), lambda: b.extend([[], []]), lambda: b.extend([[1], [2]], chunk=0), lambda: b.fork([0], []),
                 lambda: b.fork([0, 0], [1, 1]), lambda: b.fork([0], [2]), lambda: b.fork([-1], [1]), lambda: b.drop([2]), lambda: b.drop([0, -1])):
        with pytest.raises(ValueError):
            call()


def test_a_smaller_size_takes_no_block_from_a_fork():
    m, p = model(), prompts(10)
    first, got = torch.tensor([7, 8], dtype=torch.int32), []
    for shrink in (False, True):
        b = decode.Batch(m, cache_of(m), 2, 64, m.vocab)
        b.extend(p + [[]])
        b.drop([1])
        b.fork([0], [1])
        if shrink:
            b.resize(torch.tensor([3, 10], dtype=torch.int32))
            assert b.length.tolist() == [10, 10]
        got.append(b.decode(first, 6)[1])
        assert b.error() == 0
        b.release()
        assert sorted(b.cache.free.tolist()) == list(range(b.cache.num_blocks)) and int(b.cache.shared.sum()) == 0
    assert torch.equal(*got)
