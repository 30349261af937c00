"""Prompts in chunks, their scores, forked, dropped and compacted requests through decode.py on the GPU, together as they are
used, against the same requests fed token by token and alone."""
import numpy as np
import pytest
import torch

from eagle_speculative_decoding_step_gb300 import decode

pytestmark = pytest.mark.gpu


def model(dtype="f32", hd=64, seed=3):
    return decode.RandomModel(layers=2, hidden=128, nq=4, nkv=2, hd=hd, inter=192, vocab=1003, max_len=512, dtype=dtype, seed=seed)


def cache_of(m, blocks=200, bs=16, **kw):
    kw = dict(dict(dtype="f32", max_rows=16), **kw)
    return decode.PagedCache(2, blocks, bs, m.nq, m.nkv, m.hd, **kw)


def prompts(*lengths, seed=0):
    r = np.random.default_rng(seed)
    return [r.integers(0, 1003, n).tolist() for n in lengths]


def one_by_one(m, tokens, **kw):
    b = decode.Batch(m, cache_of(m, **kw), 1, 256, m.vocab)
    return torch.cat([b.feed(torch.tensor([t], dtype=torch.int32, device="cuda")) for t in tokens])


# fp32: sums of at most 128 products and 200 keys in another order, through two layers and a head of weight 3: logits of
# about 3 move by less than 1e-3.  16-bit rows: a layer's activations are rounded to 2^-8 (bf16) or 2^-11 (f16) of themselves
# in both runs, some forty roundings deep.
TOL = {"f32": 1e-3, "bf16": 40 * 2.0 ** -8, "f16": 40 * 2.0 ** -11}


@pytest.mark.parametrize("t,kw", [("f32", {}), ("bf16", dict(dtype="bf16")), ("f16", dict(dtype="f16", window=50)),
                                  ("bf16", dict(dtype="bf16", kv_dtype="e4m3", k_scale=0.02, v_scale=0.02)), ("f32", dict(bs=5))])
@pytest.mark.parametrize("chunk", [33, 512])
def test_prompts_in_chunks(t, kw, chunk):
    m, p = model(t), prompts(90, 1, 0, 140, 64)
    b = decode.Batch(m, cache_of(m, **kw), 5, 256, m.vocab)
    scores = b.score(p, k=4, chunk=chunk)
    assert b.error() == 0 and b.length.tolist() == [90, 1, 0, 140, 64]
    for i in (0, 1, 3, 4):
        ref = torch.log_softmax(one_by_one(m, p[i], **kw).double(), -1)
        s = scores[i]
        want = ref[torch.arange(len(p[i]) - 1), torch.tensor(p[i][1:], dtype=torch.long)].float()
        torch.testing.assert_close(s["logprob"][:-1], want, atol=TOL[t], rtol=0)
        # the best token, unless two are as near as the runs
        best = ref.gather(1, s["top_ids"][:, :1].long())[:, 0]
        assert (ref.amax(-1) - best <= 2 * TOL[t]).all()


def test_forks_decode_as_requests_of_their_own_and_compaction_changes_nothing():
    m, p = model(), prompts(40, 32, 100)
    first = torch.arange(6, dtype=torch.int32, device="cuda") + 7
    outs = []
    for compact in (False, True):
        b = decode.Batch(m, cache_of(m), 6, 256, m.vocab)
        b.extend(p + [[]] * 3)
        b.drop([3, 4, 5])
        b.fork([0, 0, 2], [3, 4, 5])
        # 40 tokens: two full blocks are shared, one of 8 slots copied; 100: six shared, one copied
        assert b.cache.num_blocks - int(b.cache.n_free) == (3 + 1 + 1) + 2 + (7 + 1)
        out = [b.decode(first, 30)]
        b.drop([0, 1])
        if compact:
            b.compact()
            used = torch.unique(torch.cat([row[:-(-int(n) // 16)] for row, n in zip(b.table, b.length)]))
            assert used.tolist() == list(range(len(used)))
        out.append(b.decode(out[0][:, -1].contiguous(), 20))
        outs.append(torch.cat(out, 1)[2:])
        assert b.error() == 0
        b.release()
        assert sorted(b.cache.free.tolist()) == list(range(200)) and int(b.cache.shared.sum()) == 0
    assert torch.equal(*outs)
    for row, src in ((0, 2), (1, 0), (3, 2)):                  # of the rows 2, 3 and 5
        c = decode.Batch(m, cache_of(m), 1, 256, m.vocab)
        c.extend([p[src]])
        assert outs[0][row].tolist() == c.decode(first[row + 2:row + 3], 50)[0].tolist()


def test_an_end_token_gives_back_what_no_other_sample_holds():
    m, p = model(), prompts(50)
    first = torch.tensor([7, 8, 9], dtype=torch.int32, device="cuda")

    def run(eos):
        b = decode.Batch(m, cache_of(m), 3, 256, m.vocab, eos=eos)
        b.extend(p + [[], []])
        b.drop([1, 2])
        b.fork([0, 0], [1, 2])
        out = b.decode(first, 40)
        assert b.error() == 0
        b.release()
        assert sorted(b.cache.free.tolist()) == list(range(200))
        return out
    seen = run(-1)
    eos = int(seen[0, 5])
    out = run(eos)
    for row in range(3):
        want = seen[row].tolist()
        want = want[:want.index(eos) + 1] if eos in want else want
        assert out[row].tolist()[:len(want)] == want


def test_the_command_runs(capsys):
    decode.main()
    text = capsys.readouterr().out
    assert "free blocks: 2048 of 2048" in text and "mean log-probability" in text
