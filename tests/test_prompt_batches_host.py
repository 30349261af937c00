"""Batches that take prompts, forks and smaller sizes at any point of their requests' lives, on CPU tensors (prompt_library)."""
import gc
import weakref

import pytest
import torch

import prompt_library
from eagle_speculative_decoding_step_gb300 import decode
from test_prompt_host import cache_of, model, one_by_one, prompts


@pytest.fixture(autouse=True)
def on_cpu(monkeypatch):
    prompt_library.use(monkeypatch)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32)


def all_blocks_are_back(b):
    return sorted(b.cache.free.tolist()) == list(range(b.cache.num_blocks)) and int(b.cache.shared.sum()) == 0


def ended(steps, forked=False):
    """A batch whose row 0 has just selected the end token, in the last of `steps` steps, and row 1 goes on; the same batch
    without an end token."""
    m, p, out = model(), prompts(9, 6), None
    for eos in (-1, None):
        b = decode.Batch(m, cache_of(m), 3, 64, m.vocab, eos=eos if eos is not None else int(out[0, steps - 1]))
        b.extend(p + [[]])
        if forked:
            b.drop([2])
            b.fork([0], [2])
        first = out
        out = b.decode(ints(7, 8, 9), steps)
    end = int(first[0, steps - 1])
    assert end not in first[0, :steps - 1].tolist() and end not in first[1].tolist() and end not in first[2].tolist()
    assert int(b.live[0]) == 0 and int(b.length[0]) > 0
    return m, b


@pytest.mark.parametrize("forked", [False, True])
@pytest.mark.parametrize("chunk", [2, 512])
def test_a_prompt_right_after_an_end_token(forked, chunk):
    m, b = ended(3, forked)
    lengths = b.length.tolist()
    out = b.extend([[3, 4, 5], [], []], chunk=chunk)
    torch.testing.assert_close(out[0], one_by_one(m, [3, 4, 5])[-1], atol=1e-4, rtol=1e-4)
    assert b.length.tolist() == [3] + lengths[1:] and b.live.tolist() == [1, 1, 1] and b.error() == 0
    logits = b.feed(ints(6, 1, 2))
    torch.testing.assert_close(logits[0], one_by_one(m, [3, 4, 5, 6])[-1], atol=1e-4, rtol=1e-4)
    b.release()
    assert all_blocks_are_back(b) and b.error() == 0


def test_scores_of_a_prompt_right_after_an_end_token():
    m, b = ended(4)
    s = b.score([[3, 4, 5], [], []], k=2)[0]
    logp = torch.log_softmax(one_by_one(m, [3, 4, 5]).double(), -1)
    torch.testing.assert_close(s["logprob"][:2], logp[torch.arange(2), torch.tensor([4, 5])].float(), atol=1e-4, rtol=1e-4)
    assert (s["top_ids"][:, 0].long() == logp.argmax(-1)).all() and b.error() == 0


def test_what_a_request_that_stopped_is_told():
    """Its tokens were not fed: logits of zeros, and scores as of a row without a logit.  (The pool serves requests in their
    order, so the one that it cannot serve is the last.)"""
    m, p = model(), prompts(6, 5, 30)
    for chunk in (8, 100):
        b = decode.Batch(m, cache_of(m, blocks=6), 3, 64, m.vocab)
        out = b.extend(p, chunk=chunk)
        assert b.stopped.tolist() == [False, False, True] and (out[2] == 0).all() and out[0].any() and out[1].any()
        b = decode.Batch(m, cache_of(m, blocks=6), 3, 64, m.vocab)
        s = b.score(p, k=2, chunk=chunk)
        assert b.stopped.tolist() == [False, False, True]
        fed = int(b.length[2])                                 # in the chunks before it stopped
        assert fed == (8 if chunk == 8 else 0)
        for key, nothing in (("logprob", -float("inf")), ("rank", -1), ("entropy", 0), ("lse", -float("inf")), ("top_ids", -1),
                             ("top_logprob", -float("inf"))):
            assert s[2][key].shape[0] == 30 and (s[2][key][fed:] == nothing).all(), key
        assert s[2]["lse"][:fed].isfinite().all() and s[0]["lse"].isfinite().all() and (s[1]["top_ids"] >= 0).all()


def forked_batch(m, p):
    """Rows 0 and 1: p[0] (10 tokens: two full blocks of 4 are shared, the third is each one's own)."""
    b = decode.Batch(m, cache_of(m), 2, 64, m.vocab)
    b.extend(p[:1] + [[]])
    b.drop([1])
    b.fork([0], [1])
    return b


@pytest.mark.parametrize("size", [18, 13, 12, 9, 8])
def test_a_forked_request_gives_back_tokens_that_are_its_own(size):
    """What comes after equals a request that never had the tokens, and the other row is as it was."""
    m, p = model(), prompts(10, 9)
    b = forked_batch(m, p)
    b.extend([p[1], []])
    free = int(b.cache.n_free)
    b.resize(ints(size, 10))
    assert b.length.tolist() == [size, 10] and int(b.cache.n_free) == free + 5 - -(-size // 4)
    out = b.extend([[5, 6, 7], [8]])
    kept = (p[0] + p[1])[:size]
    torch.testing.assert_close(out[0], one_by_one(m, kept + [5, 6, 7])[-1], atol=1e-4, rtol=1e-4)
    torch.testing.assert_close(out[1], one_by_one(m, p[0] + [8])[-1], atol=1e-4, rtol=1e-4)
    b.release()
    assert all_blocks_are_back(b) and b.error() == 0


@pytest.mark.parametrize("size", [1, 3, 4, 7])
def test_a_forked_request_keeps_blocks_that_another_row_holds(size):
    m, p = model(), prompts(10, 9)
    b = forked_batch(m, p)
    b.resize(ints(size, 10))
    assert b.length.tolist() == [10, 10]
    b.drop([1])                                                # nobody else holds them any more
    b.resize(ints(size, 0))
    assert b.length.tolist() == [size, 0]
    out = b.extend([[5, 6], []])
    torch.testing.assert_close(out[0], one_by_one(m, p[0][:size] + [5, 6])[-1], atol=1e-4, rtol=1e-4)
    b.release()
    assert all_blocks_are_back(b) and b.error() == 0


def test_a_batch_that_was_released_is_as_one_that_was_never_forked(monkeypatch):
    m, p = model(), prompts(10, 9)
    b = forked_batch(m, p)
    b.release()
    calls = []
    monkeypatch.setattr(decode.lib, "spec_block_release", lambda *a: calls.append(a))
    b.extend(p)
    b.resize(ints(4, 9))
    b.feed(ints(1, 2))
    assert b.length.tolist() == [5, 10] and calls == []


def test_a_score_that_needs_more_room_keeps_the_error_of_the_last_one(monkeypatch):
    m, p = model(), prompts(3, 30)
    b = decode.Batch(m, cache_of(m), 2, 64, m.vocab)
    b.score([p[0], []], k=1)
    b.lws[:4].view(torch.int32)[0] = -6                        # as a token outside the vocabulary leaves it
    have = b.lws.numel()
    monkeypatch.setattr(decode.lib, "spec_token_logprobs_workspace_bytes", lambda *a: 2 * have)
    b.score([[], p[1]], k=4)
    assert b.lws.numel() == 2 * have and b.error() == -6


def test_a_replaced_workspace_outlives_a_graph_that_was_captured_with_it(monkeypatch):
    """The graph's replays still work on it after a larger call has got another one."""
    m = model()
    kept = []
    for captured in (True, False):
        b = decode.Batch(m, cache_of(m), 1, 64, m.vocab)
        b.extend([[1, 2, 3]])
        c = b.cache
        attend = c.attend_chunks(b.kvs, ints(-1), ints(0, 1), ints(3))
        monkeypatch.setattr(decode, "_capturing", lambda device: captured)
        attend(0, torch.zeros(1, m.nq, m.hd), torch.zeros(1, m.nkv, m.hd), torch.zeros(1, m.nkv, m.hd))
        monkeypatch.setattr(decode, "_capturing", lambda device: False)
        old = weakref.ref(c.chunk_ws)
        have = c.chunk_ws.numel()
        with monkeypatch.context() as patch:
            patch.setattr(decode.lib, "spec_chunk_attention_workspace_bytes", lambda *a: 2 * have)
            b.extend([[4, 5]])
        gc.collect()
        assert c.chunk_ws.numel() == 2 * have and b.error() == 0
        kept.append(old() is not None)
    assert kept == [True, False]                               # (and no other is kept)


def test_a_workspace_is_not_made_while_a_graph_is_captured(monkeypatch):
    """Its zeros would be written by the replays only, and an eager call before the first one would find what was there."""
    m = model()
    c = cache_of(m)
    monkeypatch.setattr(decode, "_capturing", lambda device: True)
    with pytest.raises(RuntimeError):
        c.attend_chunks(c.views(torch.zeros(1, 4, dtype=torch.int32)), ints(0, 1), ints(0, 2), ints(2))
    monkeypatch.setattr(decode, "_capturing", lambda device: False)
    c.attend_chunks(c.views(torch.zeros(1, 4, dtype=torch.int32)), ints(0, 1), ints(0, 2), ints(2))
    monkeypatch.setattr(decode, "_capturing", lambda device: True)
    c.attend_chunks(c.views(torch.zeros(1, 4, dtype=torch.int32)), ints(0), ints(0, 1), ints(2))      # it is there


def test_the_fork_of_a_row_without_tokens_is_as_that_row():
    """One that takes tokens from its first on, one that was dropped, and one that the pool has no block for."""
    m, p = model(), prompts(6)
    b = decode.Batch(m, cache_of(m), 5, 64, m.vocab)
    b.extend(p + [[]] * 4)
    b.drop([2])
    b.fork([1, 2], [3, 4])
    assert b.live.tolist() == [1, 1, 0, 1, 0] and b.length.tolist() == [6, 0, 0, 0, 0] and b.error() == 0
    logits = b.feed(ints(4, 7, 1, 7, 1))
    assert b.length.tolist() == [7, 1, 0, 1, 0]
    torch.testing.assert_close(logits[3], one_by_one(m, [7])[0], atol=1e-4, rtol=1e-4)
    e = decode.Batch(m, cache_of(m), 3, 64, m.vocab)           # all as they were before the call
    e.extend(p + [[], []])
    e.fork([0, 1], [1, 2])
    assert e.length.tolist() == [6, 6, 0] and e.live.tolist() == [1, 1, 1] and e.error() == 0
    c = decode.Batch(m, cache_of(m, blocks=2), 2, 64, m.vocab)
    c.extend(p + [[]])
    c.fork([0], [1])
    assert c.length.tolist() == [6, 0] and c.live.tolist() == [1, 0] and c.error() != 0


def test_a_fork_that_is_refused_changes_nothing(monkeypatch):
    m, p = model(), prompts(6)
    b = decode.Batch(m, cache_of(m), 2, 64, m.vocab)
    b.extend(p + [[]])

    def refuse(*a):
        raise RuntimeError("more layers than one call copies")
    monkeypatch.setattr(decode.lib, "spec_block_fork", refuse)
    with pytest.raises(RuntimeError):
        b.fork([0], [1])
    assert not b.forked and b.live.tolist() == [1, 1] and b.length.tolist() == [6, 0]


@pytest.mark.parametrize("k", [-1, 33])
def test_a_score_with_too_many_alternatives_feeds_nothing(monkeypatch, k):
    m = model()
    b = decode.Batch(m, cache_of(m), 1, 64, m.vocab)
    b.extend([[1, 2]])
    size = decode.lib.spec_token_logprobs_workspace_bytes
    monkeypatch.setattr(decode.lib, "spec_token_logprobs_workspace_bytes", lambda n, V, k: size(n, V, k) if 0 <= k <= 32 else 0)
    with pytest.raises(ValueError):
        b.score([[3, 4]], k=k)
    assert b.length.tolist() == [2]
