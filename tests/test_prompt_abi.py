"""Refusals of the calls for prompts and samples (host checks, no GPU needed): every call below fails before any launch,
so the fake pointers are never dereferenced."""
import ctypes

import pytest

from eagle_speculative_decoding_step_gb300 import binding as lib
from eagle_speculative_decoding_step_gb300 import build

F = 4096                          # non-null, 256-byte aligned
ARG, SHAPE, UNSUPPORTED, CAPACITY, WS, ALIGN = -1, -2, -3, -4, -8, -9
BIG = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def so():
    build.build()
    return lib.load()


def call(name, *args):
    return getattr(lib.load(), name)(*args)


def desc(nq=8, nkv=2, hd=64, t="bf16", c=None, **kw):
    return lib.make_attn_desc(nq, nkv, hd, t, c, **kw)


def kv(k=F, v=F, table=F, bs=16, mb=8, slots=1024):
    return lib.KV(k, v, table, bs, mb, slots)


def chunk(d=None, q=F, q_ld=0, cache=None, cu=F, lens=F, B=4, n=64, max_chunk=0, max_len=0, out=F, out_ld=0, lse=F, ws=F,
          wsb=BIG):
    return call("spec_chunk_attention", ctypes.byref(d or desc()), q, q_ld, ctypes.byref(cache or kv()), cu, lens, B, n,
                max_chunk, max_len, out, out_ld, lse, ws, wsb, None)


def test_chunk_attention_refusals():
    for kw in (dict(q=None), dict(cu=None), dict(lens=None), dict(out=None), dict(cache=kv(table=None)), dict(cache=kv(k=None)),
               dict(cache=kv(v=None))):
        assert chunk(**kw) == ARG, kw
    for d in (desc(nq=7), desc(nq=0), desc(nkv=0), desc(hd=24), desc(hd=0), desc(hd=272), desc(nq=258), desc(window=-1)):
        assert chunk(d=d) == SHAPE
    for kw in (dict(B=0), dict(n=0), dict(n=-1), dict(max_chunk=-1), dict(max_len=-1), dict(q_ld=8), dict(out_ld=511),
               dict(cache=kv(bs=0)), dict(cache=kv(mb=0)), dict(cache=kv(slots=0)), dict(cache=kv(mb=1 << 28))):
        assert chunk(**kw) == SHAPE, kw
    for d in (desc(c="f32"), desc(t="f32", c="e4m3"), desc(t="e4m3"), desc(t="bf16", c="f16")):
        assert chunk(d=d) == UNSUPPORTED
    for x in (-1.0, float("nan"), float("inf")):
        assert chunk(d=desc(scale=x)) == ARG
        assert chunk(d=desc(c="e4m3", k_scale=x)) == ARG and chunk(d=desc(c="e4m3", v_scale=x)) == ARG
    assert chunk(n=1 << 28) == CAPACITY and chunk(d=desc(nq=1 << 24, nkv=1 << 24), n=1) == CAPACITY
    assert chunk(q=F + 8) == ALIGN and chunk(out=F + 2) == ALIGN and chunk(q_ld=516) == ALIGN and chunk(out_ld=516) == ALIGN
    assert chunk(cache=kv(k=F + 8)) == ALIGN and chunk(d=desc(t="f32"), q_ld=514) == ALIGN
    assert chunk(ws=None) == WS and chunk(ws=F + 128) == WS and chunk(wsb=256) == WS
    size = lib.spec_chunk_attention_workspace_bytes
    assert chunk(wsb=size(desc(), 4, 64) - 1) == WS
    assert size(desc(nq=7), 4, 64) == 0 and size(desc(), 0, 64) == 0 and size(desc(), 4, 0) == 0 and size(desc(), 4, 1 << 28) == 0
    n = [size(desc(), B, rows) for B, rows in ((1, 1), (1, 100), (40, 100), (40, 9000), (5000, 9000))]
    assert n == sorted(n)


def logprobs(n=4, V=100, t=1, logits=F, ld=0, tok=F, k=5, lp=F, rank=F, ent=F, lse=F, ids=F, top=F, ws=F, wsb=BIG):
    return call("spec_token_logprobs", n, V, t, logits, ld, tok, k, lp, rank, ent, lse, ids, top, ws, wsb, None)


def test_token_logprobs_refusals():
    for kw in (dict(logits=None), dict(ids=None), dict(top=None), dict(tok=None), dict(tok=None, rank=None),
               dict(tok=None, lp=None)):
        assert logprobs(**kw) == ARG, kw
    for kw in (dict(n=0), dict(V=0), dict(k=-1), dict(k=33), dict(ld=99), dict(ld=-1)):
        assert logprobs(**kw) == SHAPE, kw
    assert logprobs(t=3) == UNSUPPORTED and logprobs(t=-1) == UNSUPPORTED and logprobs(V=(1 << 20) + 1) == CAPACITY
    assert logprobs(logits=F + 1) == ALIGN and logprobs(t=0, logits=F + 2) == ALIGN
    assert logprobs(ws=None) == WS and logprobs(ws=F + 64) == WS and logprobs(wsb=300) == WS
    size = lib.spec_token_logprobs_workspace_bytes
    assert logprobs(wsb=size(4, 100, 5) - 1) == WS
    assert size(0, 100, 5) == 0 and size(4, 0, 5) == 0 and size(4, 100, 33) == 0 and size(4, (1 << 20) + 1, 0) == 0
    for n in ([size(n, 128256, 5) for n in range(1, 9000, 7)], [size(4, V, 5) for V in range(1, 1 << 20, 997)],
              [size(4, 128256, k) for k in range(33)]):
        assert n == sorted(n)                                  # a workspace serves every smaller call


STATE = ["table_in", "table_out", "len_in", "len_out", "shared_in", "shared_out", "free_in", "free_out", "n_free_in",
         "n_free_out"]


def state(B=4, bs=16, mb=8, nb=64, **over):
    return lib.BlockState(B, bs, mb, nb, *[over.get(n, F + 256 * i) for i, n in enumerate(STATE)])


def fork(st=None, n=2, src=F, dst=F, kvs=None, layers=None, row=256, ws=F, wsb=BIG):
    kvs = kvs or [kv(), kv()]
    a = (lib.KV * len(kvs))(*kvs)
    return call("spec_block_fork", ctypes.byref(st or state()), n, src, dst, len(kvs) if layers is None else layers, a, row, ws,
                wsb, None)


def release(st=None, drop=F, ws=F, wsb=BIG):
    return call("spec_block_release", ctypes.byref(st or state()), drop, ws, wsb, None)


def compact(st=None, kvs=None, layers=None, row=256, ws=F, wsb=BIG):
    kvs = kvs or [kv(), kv()]
    a = (lib.KV * len(kvs))(*kvs)
    return call("spec_block_compact", ctypes.byref(st or state()), len(kvs) if layers is None else layers, a, row, ws, wsb, None)


@pytest.mark.parametrize("f", [fork, release, compact])
def test_block_state_refusals(f):
    for name in STATE:
        assert f(state(**{name: None})) == ARG
    for kw in (dict(B=0), dict(bs=0), dict(mb=0), dict(nb=0), dict(bs=-1)):
        assert f(state(**kw)) == SHAPE
    # (the caches of the copying calls are of the state's block size and pool)
    for kw in (dict(B=8193), dict(mb=1 << 27), dict(B=4096, mb=1 << 15), dict(nb=1 << 27)):
        assert f(state(**kw)) == CAPACITY
    assert f(ws=None) == WS and f(ws=F + 16) == WS and f(wsb=512) == WS
    assert f(wsb=lib.spec_block_state_workspace_bytes(4, 64) - 1) == WS
    assert lib.spec_block_state_workspace_bytes(0, 64) == 0 and lib.spec_block_state_workspace_bytes(4, 0) == 0
    assert lib.spec_block_state_workspace_bytes(8193, 64) == 0


def test_block_fork_refusals():
    assert fork(src=None) == ARG and fork(dst=None) == ARG and release(drop=None) == ARG
    for n in (0, -1, 5):
        assert fork(n=n) == SHAPE


@pytest.mark.parametrize("f", [fork, compact])
def test_copying_refusals(f):
    assert f(kvs=[kv(k=None)]) == ARG and f(kvs=[kv(), kv(v=None)]) == ARG
    for kw in (dict(layers=0), dict(layers=65), dict(row=0), dict(row=-16), dict(kvs=[kv(bs=8)]), dict(kvs=[kv(slots=1023)])):
        assert f(**kw) == SHAPE, kw
