"""Whole decoding runs through the paged cache (decode.Batch, decode.BeamBatch) against a search
that keeps no cache: every step recomputes the model over the whole sequence in fp64."""
import math

import numpy as np
import pytest
import torch

from eagle_speculative_decoding_step_gb300 import decode
from oracle import decode as oracle

pytestmark = pytest.mark.gpu


class Plain:
    """RandomModel over whole sequences in fp64: logits of the last token."""

    def __init__(self, m):
        self.m = m
        self.embed, self.place, self.head = m.embed.double().cpu(), m.place.double().cpu(), m.head.double().cpu()
        self.layers = [{k: v.double().cpu() for k, v in w.items()} for w in m.layers]

    def logits(self, seq):
        m = self.m
        norm = lambda x: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
        n = len(seq)
        x = self.embed[torch.tensor(seq)] + self.place[:n]
        for w in self.layers:
            q, k, v = (norm(x) @ w["qkv"].T).split([m.nq * m.hd, m.nkv * m.hd, m.nkv * m.hd], 1)
            g = m.nq // m.nkv
            q, k, v = q.view(n, m.nq, m.hd), k.view(n, m.nkv, m.hd).repeat_interleave(g, 1), \
                v.view(n, m.nkv, m.hd).repeat_interleave(g, 1)
            s = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(m.hd)
            s = s.masked_fill(torch.ones(n, n).triu(1).bool(), -math.inf).softmax(-1)
            x = x + torch.einsum("hij,jhd->ihd", s, v).reshape(n, -1) @ w["o"].T
            up, gate = (norm(x) @ w["up"].T).chunk(2, 1)
            x = x + (up * torch.nn.functional.silu(gate)) @ w["down"].T
        return (norm(x)[-1] @ self.head.T).numpy()


def small(**kw):
    return decode.RandomModel(layers=2, hidden=64, nq=4, nkv=2, hd=32, inter=96, vocab=503, max_len=256, dtype="f32", **kw)


@pytest.fixture(autouse=True)
def full_fp32():
    before = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    yield
    torch.backends.cuda.matmul.allow_tf32 = before


@pytest.mark.parametrize("bs", [1, 8, 16])
def test_greedy_batch(bs):
    m = small(seed=3)
    cache = decode.PagedCache(2, 600, bs, m.nq, m.nkv, m.hd, dtype="f32", max_rows=3)
    b = decode.Batch(m, cache, 3, 64, m.vocab)
    tok = torch.tensor([5, 17, 400], dtype=torch.int32, device="cuda")
    got = b.decode(tok, 20).cpu().numpy()
    assert b.error() == 0 and int(b.length[0]) == 20
    ref = Plain(m)
    for i, first in enumerate([5, 17, 400]):
        seq = [first]
        for t in range(20):
            seq.append(int(np.argmax(ref.logits(seq))))
        assert got[i].tolist() == seq[1:]
    b.release()
    assert int(cache.n_free[0]) == 600 and sorted(cache.free.tolist()) == list(range(600))


@pytest.mark.parametrize("W,bs,eos", [(1, 16, -1), (4, 4, -1), (3, 8, 11), (5, 1, -1), (2, 16, 7)])
def test_beam_batch(W, bs, eos):
    m = small(seed=W)
    r = np.random.default_rng(bs)
    prompts = [r.integers(0, m.vocab, n).tolist() for n in (1, 5, 16, 17)]
    new = 10
    cache = decode.PagedCache(2, 900, bs, m.nq, m.nkv, m.hd, dtype="f32", max_rows=4 * W)
    bb = decode.BeamBatch(m, cache, prompts, W, new, m.vocab, eos=eos)
    for _ in range(new):
        bb.step()
    assert bb.error() == 0
    got, score, done = bb.tokens.cpu().numpy(), bb.score.cpu().numpy(), bb.done.cpu().numpy()
    ref = Plain(m)
    for b, p in enumerate(prompts):
        beams = [(list(p), 0.0, 0)] + [(list(p), -math.inf, 0)] * (W - 1)
        for _ in range(new):
            lg = np.stack([ref.logits(s) if not d and sc > -math.inf else np.zeros(m.vocab) for s, sc, d in beams])
            pa, tk, sc, dn = oracle.beam_select(lg[None], np.array([[x[1] for x in beams]]), np.array([[x[2] for x in beams]]), eos)
            # a finished beam is fed its end token again and again; its history takes it too
            beams = [(beams[int(pa[0, j])][0] + [int(tk[0, j])], float(sc[0, j]), int(dn[0, j])) for j in range(W)]
        for j, (s, sc, d) in enumerate(beams):
            if sc == -math.inf:
                assert score[b, j] == -math.inf
                continue
            assert got[b, j, :len(s)].tolist() == s, (b, j)
            assert (got[b, j, len(s):] == -1).all() and done[b, j] == d
            assert abs(score[b, j] - sc) < 1e-4 * abs(sc) + 1e-4
    bb.release()
    assert int(cache.n_free[0]) == 900 and sorted(cache.free.tolist()) == list(range(900))


def test_beam_batch_in_eight_bits_runs_and_gives_its_blocks_back():
    m = decode.RandomModel(seed=9)
    cache = decode.PagedCache(2, 700, 16, m.nq, m.nkv, m.hd, kv_dtype="e4m3", k_scale=0.02, v_scale=0.02, max_rows=8)
    bb = decode.BeamBatch(m, cache, [[1, 2, 3], list(range(40))], 4, 20, m.vocab)
    for _ in range(20):
        bb.step()
    assert bb.error() == 0
    s = bb.score.cpu()
    assert torch.isfinite(s).all() and (s[:, :-1] >= s[:, 1:]).all()
    bb.release()
    assert int(cache.n_free[0]) == 700
