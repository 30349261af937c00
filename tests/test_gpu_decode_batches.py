"""Plain batches on the GPU whose requests end at different steps: each request decodes what it decodes by itself."""
import numpy as np
import pytest
import torch

from eagle_speculative_decoding_step_gb300 import binding as lib
from eagle_speculative_decoding_step_gb300 import decode

pytestmark = pytest.mark.gpu
ERR_CAPACITY = -4
FIRST = (5, 17, 400, 33)


@pytest.fixture(autouse=True)
def full_fp32():
    before = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    yield
    torch.backends.cuda.matmul.allow_tf32 = before


def small(seed=3):
    return decode.RandomModel(layers=2, hidden=64, nq=4, nkv=2, hd=32, inter=96, vocab=503, max_len=256, dtype="f32", seed=seed)


def batch(m, n, blocks=200, bs=8, max_len=64, eos=-1):
    return decode.Batch(m, decode.PagedCache(2, blocks, bs, m.nq, m.nkv, m.hd, dtype="f32", max_rows=4), n, max_len, m.vocab, eos)


def ids(*a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def alone(steps, eos=-1):
    """Each of FIRST decoded by itself; the best logits lie far enough apart for the batch size not to matter."""
    m = small()
    return [batch(m, 1, eos=eos).decode(ids(f), steps)[0].tolist() for f in FIRST]


def test_requests_that_the_pool_cannot_serve_stop_and_the_others_go_on():
    want = alone(20)
    b = batch(small(), 4, blocks=6)                       # 8 tokens a block: two of the four get a second one
    got = b.decode(ids(*FIRST), 20).tolist()
    assert got[:2] == [w[:16] + [-1] * 4 for w in want[:2]]
    assert got[2:] == [w[:8] + [-1] * 12 for w in want[2:]]
    assert b.error() == ERR_CAPACITY and b.length.tolist() == [16, 16, 8, 8] and b.stopped.all()
    b.release()
    assert int(b.cache.n_free[0]) == 6 and b.length.tolist() == [0] * 4


def test_requests_at_the_end_of_their_tables_stop():
    want = alone(20)
    b = batch(small(), 4, max_len=16)
    got = b.decode(ids(*FIRST), 20).tolist()
    assert got == [w[:16] + [-1] * 4 for w in want] and b.error() != 0 and b.length.tolist() == [16] * 4


def test_finished_requests_give_their_blocks_back_and_a_batch_is_used_again():
    eos = alone(5)[1][-1]
    want = alone(20, eos)
    b = batch(small(), 4, eos=eos)
    got = b.decode(ids(*FIRST), 20).tolist()
    assert got == want and b.error() == 0
    ended = [i for i, w in enumerate(want) if eos in w[:-1]]
    assert 1 in ended and len(ended) < 4
    assert [int(n) == 0 for n in b.length] == [i in ended for i in range(4)]
    assert int(b.cache.n_free[0]) == 200 - 3 * (4 - len(ended))
    b.release()
    assert b.decode(ids(*FIRST[::-1]), 20).tolist() == want[::-1] and b.error() == 0


def beams(prompts, W, steps, blocks=200, bs=8):
    m = small()
    b = decode.BeamBatch(m, decode.PagedCache(2, blocks, bs, m.nq, m.nkv, m.hd, dtype="f32", max_rows=W * len(prompts)), prompts, W,
                         20, m.vocab)
    for _ in range(steps):
        b.step()
    return b


def test_beams_of_a_request_that_the_pool_cannot_serve_stop_and_the_others_go_on():
    prompts, W = [[5, 9, 7], [11, 4, 8]], 3
    first, want, start = beams(prompts, W, 6), beams(prompts, W, 12), beams(prompts, W, 0)
    need = 200 - int(start.cache.n_free[0])
    b = beams(prompts, W, 12, blocks=need + W)               # at the first border, after six tokens, there is room for one
    assert want.error() == 0 and lib.spec_get_device_error(b.tws) == ERR_CAPACITY and b.cache.error() == 0
    assert b.stopped.tolist() == [False, True]
    assert torch.equal(b.tokens[0], want.tokens[0]) and torch.equal(b.score[0], want.score[0])
    assert torch.equal(b.tokens[1, :, :9], first.tokens[1, :, :9]) and (b.tokens[1, :, 9:] == -1).all()
    assert torch.equal(b.score[1], first.score[1])
    b.release()
    assert int(b.cache.n_free[0]) == need + W
