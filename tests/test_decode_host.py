"""What decode.py hands to the library and makes of its answers, on CPU tensors (cpu_library): layouts of a model's rows,
requests that cannot go on, runs one after another."""
import numpy as np
import pytest
import torch

import cpu_library
from eagle_speculative_decoding_step_gb300 import decode


@pytest.fixture(autouse=True)
def on_cpu(monkeypatch):
    cpu_library.use(monkeypatch)


class Layouts(decode.RandomModel):
    """RandomModel whose rows reach ``attend`` in another layout (lay: of q, k, v), their values the same."""

    def __init__(self, lay=None, **kw):
        super().__init__(layers=2, hidden=64, nq=4, nkv=2, hd=16, inter=96, vocab=203, max_len=256, dtype="f32", device="cpu",
                         **kw)
        self.lay = lay or (lambda q, k, v: (q, k, v))

    def __call__(self, tok, pos, attend):
        return super().__call__(tok, pos, lambda i, q, k, v: attend(i, *self.lay(q, k, v)))


def cache_of(m, blocks=60, bs=4, rows=8):
    return decode.PagedCache(2, blocks, bs, m.nq, m.nkv, m.hd, dtype="f32", max_rows=rows, device="cpu")


def ids(*a):
    return torch.tensor(a, dtype=torch.int32)


def heads_first(x):
    """The same values, heads outermost in memory."""
    return x.transpose(0, 1).contiguous().transpose(0, 1)


def components_first(x):
    return x.transpose(1, 2).contiguous().transpose(1, 2)


LAYOUTS = dict(k_its_own=lambda q, k, v: (q, k.contiguous(), v), v_its_own=lambda q, k, v: (q, k, v.contiguous()),
               all_their_own=lambda q, k, v: (q.contiguous(), k.contiguous(), v.contiguous()),
               q_by_heads=lambda q, k, v: (heads_first(q), k, v), k_by_heads=lambda q, k, v: (q, heads_first(k), v),
               v_by_components=lambda q, k, v: (q, k, components_first(v)),
               flat=lambda q, k, v: (q.flatten(1), k.flatten(1), v.flatten(1)))


@pytest.mark.parametrize("beams", [False, True])
@pytest.mark.parametrize("name", LAYOUTS)
def test_rows_of_any_layout_give_the_same(name, beams):
    """K that was rotated is a tensor of its own while V is a slice of the fused product, and so on."""
    got = []
    for lay in (None, LAYOUTS[name]):
        m = Layouts(lay, seed=3)
        c = cache_of(m)
        if beams:
            b = decode.BeamBatch(m, c, [[5, 9, 7, 2, 1], [11]], 2, 6, m.vocab)
            for _ in range(6):
                b.step()
            got.append(b.tokens.clone())
        else:
            b = decode.Batch(m, c, 3, 16, m.vocab)
            got.append(b.decode(ids(5, 17, 100), 9))
        assert b.error() == 0
    assert torch.equal(*got)


def test_a_single_row_whose_first_stride_means_nothing():
    m = Layouts(lambda q, k, v: tuple(x.as_strided(x.shape, (1, x.stride(1), 1)) for x in (q, k, v)), seed=3)
    b, ref = (decode.Batch(x, cache_of(x), 1, 16, x.vocab) for x in (m, Layouts(seed=3)))
    assert torch.equal(b.decode(ids(5), 5), ref.decode(ids(5), 5))


def test_rows_of_another_type_or_shape_are_refused():
    for lay in (lambda q, k, v: (q.double(), k, v), lambda q, k, v: (q, k.bfloat16(), v), lambda q, k, v: (q, k, v.half()),
                lambda q, k, v: (q[:, :2], k, v), lambda q, k, v: (q, k[..., :8], v), lambda q, k, v: (q, k, v[:1]),
                lambda q, k, v: (q.transpose(1, 2), k, v)):
        m = Layouts(lay)
        b = decode.Batch(m, cache_of(m), 2, 16, m.vocab)
        with pytest.raises(ValueError):
            b.feed(ids(5, 6))


def test_a_row_without_a_token_is_not_looked_up():
    """Token ids that reach the model are ids: a row with no candidate, or that has ended without an end token, has -1."""
    m = Layouts(seed=3)
    seen = []
    b = decode.Batch(lambda tok, pos, attend: seen.append(tok) or m(tok, pos, attend) * float("nan"), cache_of(m), 2, 16, m.vocab)
    assert (b.decode(ids(5, 6), 4) == -1).all()
    assert all((t >= 0).all() for t in seen)


# ------------------------------------------------------------------ requests that cannot go on
def alone(first, steps, seed=3, eos=-1):
    """What a request decodes by itself."""
    m = Layouts(seed=seed)
    return decode.Batch(m, cache_of(m), 1, 64, m.vocab, eos).decode(ids(first), steps)[0].tolist()


def feed_one(b, i, tok):
    """One token of request i only."""
    one = torch.zeros(b.B, dtype=torch.int32)
    one[i] = 1
    b.resize(b.length + one)
    slots = torch.where(one == 1, b.slots[0], -1).int()
    return b.model(torch.full((b.B,), tok, dtype=torch.int32), (b.length - 1).clamp(min=0),
                   b.cache.attend(b.kvs, slots, b.length * one, b.max_len))[i]


def test_a_request_at_its_tables_end_leaves_the_others_right():
    m = Layouts(seed=5)
    toks = [[7, 8, 9, 10, 11, 12, 13, 14, 15, 16], [20, 21, 22, 23, 24], [30, 31, 32, 33, 34, 35, 36]]
    b = decode.Batch(m, cache_of(m), 3, 8, m.vocab)
    for i, n in enumerate((8, 3, 5)):
        for t in range(n):
            feed_one(b, i, toks[i][t])
    got = [b.feed(ids(toks[0][8 + s], toks[1][3 + s], toks[2][5 + s])) for s in range(2)]
    assert b.length.tolist() == [8, 5, 7] and b.error() == cpu_library.ERR_DEVICE and b.stopped.tolist() == [True, False, False]
    for i in (1, 2):
        one = decode.Batch(m, cache_of(m), 1, 8, m.vocab)
        ref = [one.feed(ids(t)) for t in toks[i]][-2:]
        for x, y in zip(got, ref):
            assert torch.allclose(x[i], y[0], atol=1e-5)


def test_a_request_that_the_pool_cannot_serve_stops_and_the_others_go_on():
    m = Layouts(seed=3)
    b = decode.Batch(m, cache_of(m, blocks=4, bs=4), 3, 16, m.vocab)      # a block each, and one more for request 0
    got = b.decode(ids(5, 17, 100), 8).tolist()
    assert got[0] == alone(5, 8)
    for row, first in ((1, 17), (2, 100)):
        assert got[row] == alone(first, 4) + [-1] * 4
    assert b.length.tolist() == [8, 4, 4] and b.stopped.tolist() == [False, True, True]
    assert b.error() == cpu_library.ERR_CAPACITY
    b.release()
    assert int(b.cache.n_free[0]) == 4 and not b.stopped.any()
    assert [int(x) for x in b.feed(ids(5, 17, 100)).argmax(1)] == [alone(f, 1)[0] for f in (5, 17, 100)]


def test_finished_requests_give_their_blocks_back():
    eos = alone(17, 3)[-1]
    want = [alone(f, 12, eos=eos) for f in (5, 17, 100)]
    assert want[1][2:] == [eos] * 10 and eos not in want[0]
    m = Layouts(seed=3)
    c = cache_of(m, blocks=20, bs=4)
    b = decode.Batch(m, c, 3, 16, m.vocab, eos)
    got = b.decode(ids(5, 17, 100), 12).tolist()
    assert got == want and b.error() == 0
    assert b.length[1] == 0 and int(c.n_free[0]) == 20 - sum(-(-int(n) // 4) for n in b.length)
    assert sorted(c.free[:int(c.n_free[0])].tolist() + b.table[b.table >= 0].tolist()) == list(range(20))


def test_a_batch_starts_anew_after_release():
    eos = alone(17, 3)[-1]
    m = Layouts(seed=3)
    b = decode.Batch(m, cache_of(m), 2, 16, m.vocab, eos)
    first = b.decode(ids(17, 5), 12).tolist()
    assert first == [alone(17, 12, eos=eos), alone(5, 12)]
    score = b.select.score[b.select.at].clone()
    b.release()
    assert b.decode(ids(5, 17), 12).tolist() == first[::-1] and b.error() == 0
    assert torch.allclose(b.select.score[b.select.at].flip(0), score)


def test_finished_requests_make_room_for_the_others():
    """Four blocks, all of which one request needs: the other one ends after three tokens."""
    eos = alone(17, 3)[-1]
    m = Layouts(seed=3)
    b = decode.Batch(m, cache_of(m, blocks=4, bs=4), 2, 16, m.vocab, eos)
    assert b.decode(ids(5, 17), 16).tolist() == [alone(5, 16), alone(17, 16, eos=eos)] and b.error() == 0


def beams_of(prompts, W, steps, blocks=200, bs=4, new=12, seed=3, eos=-1):
    m = Layouts(seed=seed)
    b = decode.BeamBatch(m, cache_of(m, blocks=blocks, bs=bs, rows=len(prompts) * W), prompts, W, new, m.vocab, eos)
    for _ in range(steps):
        b.step()
    return b


@pytest.mark.parametrize("eos", [-1, 190])
def test_beams_of_a_request_that_the_pool_cannot_serve_stop_and_the_others_go_on(eos):
    prompts, W = [[5, 9, 7], [11, 4, 8]], 2
    first = beams_of(prompts, W, 2, eos=eos)                  # two tokens are selected until the first border
    start = beams_of(prompts, W, 0)
    need = start.cache.num_blocks - int(start.cache.n_free[0])
    want = beams_of(prompts, W, 5, eos=eos)
    b = beams_of(prompts, W, 5, blocks=need + W, eos=eos)     # there are blocks for one request more
    assert want.error() == 0 and b.error() == cpu_library.ERR_CAPACITY and b.stopped.tolist() == [False, True]
    assert torch.equal(b.tokens[0], want.tokens[0]) and torch.equal(b.score[0], want.score[0])
    assert torch.equal(b.tokens[1, :, :5], first.tokens[1, :, :5]) and (b.tokens[1, :, 5:] == -1).all()
    assert torch.equal(b.score[1], first.score[1])
    b.release()
    assert int(b.cache.n_free[0]) == need + W


# ------------------------------------------------------------------ the cache's memory
@pytest.mark.parametrize("dtype,kv_dtype,es", [("f32", None, 4), ("bf16", None, 2), ("f16", "e4m3", 1)])
def test_a_cache_is_made_in_its_own_type(monkeypatch, dtype, kv_dtype, es):
    """Nothing larger than K or V is made on the way."""
    made = []
    for name in ("zeros", "empty", "full"):
        f = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, _f=f, **kw: made.append(_f(*a, **kw)) or made[-1])
    c = decode.PagedCache(3, 50, 8, 4, 2, 16, dtype=dtype, kv_dtype=kv_dtype, device="cpu")
    size = 3 * 50 * 8 * 2 * 16 * es
    assert c.k.numel() * c.k.element_size() == size == c.v.numel() * c.v.element_size()
    assert max(x.numel() * x.element_size() for x in made) == size
    assert c.k.shape == (3, 400, 2, 16) and (c.k.float() == 0).all() and (c.v.float() == 0).all()


# ------------------------------------------------------------------ layouts of the logits
def columns(x):
    """The same values, every second column of a wider tensor."""
    return x.repeat_interleave(2, 1)[:, ::2]


@pytest.mark.parametrize("name,lay", [("by_columns", lambda x: x.T.contiguous().T), ("every_second", columns),
                                      ("part", lambda x: torch.nn.functional.pad(x, (3, 5))[:, 3:-5]),
                                      ("one_more_axis", lambda x: x[:, None])])
@pytest.mark.parametrize("rows", [1, 3])
def test_logits_of_any_layout_select_the_same(name, lay, rows):
    m = Layouts(seed=3)
    got = [decode.Batch(f, cache_of(m), rows, 16, m.vocab).decode(ids(5, 17, 100)[:rows], 9)
           for f in (m, lambda *a: lay(m(*a)))]
    assert torch.equal(*got)


def test_logits_that_all_rows_share():
    """One row in memory for all of the batch."""
    m = Layouts(seed=3)
    got = [decode.Batch(lambda *a: f(m(*a)[:1]), cache_of(m), 3, 16, m.vocab).decode(ids(5, 17, 100), 4)
           for f in (lambda x: x.expand(3, -1), lambda x: x.repeat(3, 1))]
    assert torch.equal(*got) and (got[0] == got[0][:1]).all()


def test_logits_of_another_shape_or_type_are_refused():
    m = Layouts(seed=3)
    for lay in (lambda x: x[:, :-1], lambda x: x[:1], lambda x: x.double(), lambda x: x.long()):
        b = decode.Batch(lambda *a: lay(m(*a)), cache_of(m), 2, 16, m.vocab)
        with pytest.raises(ValueError):
            b.decode(ids(5, 6), 1)
