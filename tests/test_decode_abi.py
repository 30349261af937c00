"""Refusals of the decoding calls (host checks, no GPU needed): every call below fails
before any launch, so the fake pointers are never dereferenced."""
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


def tables(B=4, bs=16, mb=8, nb=64, cap=10, ws=F, wsb=BIG, **ptr):
    names = ["len_old", "len_new", "table_in", "table_out", "free_in", "n_free_in", "free_out", "n_free_out", "len_out",
             "cu_new", "slots", "pos"]
    p = {n: F for n in names}
    p.update(ptr)
    return call("spec_block_tables", B, bs, mb, nb, *[p[n] for n in names], cap, ws, wsb, None)


def test_block_tables_refusals():
    for kw in (dict(B=0), dict(bs=0), dict(mb=0), dict(nb=-1), dict(cap=0)):
        assert tables(**kw) == SHAPE
    for n in ("len_old", "len_new", "table_in", "table_out", "free_in", "n_free_in", "free_out", "n_free_out", "len_out",
              "cu_new", "slots"):
        assert tables(**{n: None}) == ARG
    assert tables(B=8193) == CAPACITY
    assert tables(B=1024, mb=1 << 16, bs=16) == CAPACITY          # 2^30 tokens
    assert tables(nb=1 << 26, bs=16) == CAPACITY
    assert tables(ws=None) == WS and tables(ws=F + 8) == WS and tables(wsb=100) == WS
    assert lib.spec_block_tables_workspace_bytes(4) > 0 and lib.spec_block_tables_workspace_bytes(0) == 0


def test_block_tables_refuses_a_slot_map_past_its_32_bit_counts():
    for cap in (1 << 30, 2 ** 31 - 100000, 2 ** 31 - 1):
        assert tables(cap=cap, ws=None) == CAPACITY


def desc(nq=8, nkv=2, hd=64, t="bf16", c=None, **kw):
    return lib.make_attn_desc(nq, nkv, hd, t, c, **kw)


def kv(k=F, v=F, table=F, bs=16, mb=8, slots=1024):
    return lib.KV(k, v, table, bs, mb, slots)


def append(d=None, k=F, v=F, ld=0, slots=F, n=4, cache=None, ws=F):
    return call("spec_cache_append", ctypes.byref(d or desc()), k, v, ld, slots, n, ctypes.byref(cache or kv()), ws, None)


def test_cache_append_refusals():
    assert append(k=None) == ARG and append(slots=None) == ARG and append(cache=kv(v=None)) == ARG
    assert append(n=0) == SHAPE and append(ld=100) == SHAPE and append(d=desc(hd=72)) == SHAPE
    assert append(d=desc(hd=272)) == SHAPE and append(cache=kv(slots=0)) == SHAPE
    assert append(d=desc(t="e4m3")) == UNSUPPORTED and append(d=desc(t="f32", c="e4m3")) == UNSUPPORTED
    assert append(d=desc(t="bf16", c="f16")) == UNSUPPORTED
    assert append(d=desc(c="e4m3", k_scale=0.0)) == ARG and append(d=desc(c="e4m3", v_scale=float("nan"))) == ARG
    assert append(k=F + 1) == ALIGN and append(cache=kv(k=F + 1)) == ALIGN
    assert append(ws=F + 16) == WS


def test_cache_append_strided_refusals():
    def strided(k_ld=0, v_ld=0, k=F, v=F, n=4):
        return call("spec_cache_append_strided", ctypes.byref(desc()), k, k_ld, v, v_ld, F, n, ctypes.byref(kv()), F, None)
    assert strided(k_ld=127) == SHAPE and strided(v_ld=127) == SHAPE and strided(k_ld=-128, v_ld=128) == SHAPE
    assert strided(k=None) == ARG and strided(v=None) == ARG and strided(v=F + 1) == ALIGN and strided(n=0) == SHAPE


def attend(d=None, q=F, q_ld=0, cache=None, lens=F, B=4, max_len=0, out=F, out_ld=0, lse=F, ws=F, wsb=BIG):
    return call("spec_paged_attention", ctypes.byref(d or desc()), q, q_ld, ctypes.byref(cache or kv()), lens, B, max_len,
                out, out_ld, lse, ws, wsb, None)


def test_paged_attention_refusals():
    assert attend(q=None) == ARG and attend(lens=None) == ARG and attend(out=None) == ARG
    assert attend(cache=kv(table=None)) == ARG and attend(cache=kv(k=None)) == ARG
    for d in (desc(nq=7), desc(nq=0), desc(hd=24), desc(hd=320), desc(nq=258, nkv=2), desc(window=-1)):
        assert attend(d=d) == SHAPE
    assert attend(B=0) == SHAPE and attend(max_len=-1) == SHAPE and attend(q_ld=8) == SHAPE and attend(out_ld=500) == SHAPE
    assert attend(cache=kv(bs=0)) == SHAPE and attend(cache=kv(mb=1 << 28)) == SHAPE
    assert attend(d=desc(c="f32")) == UNSUPPORTED and attend(d=desc(t="f32", c="e4m3")) == UNSUPPORTED
    assert attend(d=desc(scale=-1.0)) == ARG and attend(d=desc(scale=float("nan"))) == ARG
    assert attend(d=desc(c="e4m3", v_scale=-1.0)) == ARG
    assert attend(q=F + 8) == ALIGN and attend(cache=kv(v=F + 2)) == ALIGN and attend(q_ld=516) == ALIGN
    assert attend(ws=None) == WS and attend(ws=F + 128) == WS and attend(wsb=8) == WS
    assert lib.spec_attention_workspace_bytes(desc(), 4) >= 256
    assert lib.spec_attention_workspace_bytes(desc(nq=7), 4) == 0 and lib.spec_attention_workspace_bytes(desc(), 0) == 0


def select(B=2, W=4, V=100, t=1, logits=F, ld=0, score=F, done=F, eos=2, parent=F, tok=F, so=F + 256, do=F + 512, ws=F,
           wsb=BIG):
    return call("spec_beam_select", B, W, V, t, logits, ld, score, done, eos, parent, tok, so, do, ws, wsb, None)


def test_beam_select_refusals():
    assert select(logits=None) == ARG and select(done=None) == ARG and select(tok=None) == ARG
    assert select(so=F) == ARG and select(do=F) == ARG                 # outputs that are inputs
    assert select(t=3) == UNSUPPORTED and select(t=-1) == UNSUPPORTED
    assert select(B=0) == SHAPE and select(W=33) == SHAPE and select(V=0) == SHAPE and select(eos=100) == SHAPE
    assert select(W=32, V=1 << 25) == SHAPE and select(ld=99) == SHAPE and select(B=20000) == SHAPE
    assert select(logits=F + 1) == ALIGN
    assert select(ws=None) == WS and select(wsb=16) == WS and select(ws=F + 64) == WS
    assert lib.spec_beam_workspace_bytes(2, 4, 100) > 0 and lib.spec_beam_workspace_bytes(2, 33, 100) == 0


def test_a_beam_workspace_serves_every_smaller_batch():
    """A smaller batch cuts its rows into more chunks; the size is that of the largest need up to B."""
    for W, V in ((1, 128256), (4, 128256), (8, 151936), (8, 40000), (5, 33), (32, 262144), (3, 8193)):
        n = [lib.spec_beam_workspace_bytes(B, W, V) for B in range(1, 400)]
        assert n == sorted(n), (W, V)
    for B, V in ((1, 5000), (3, 128256), (40, 128256)):
        n = [lib.spec_beam_workspace_bytes(B, W, V) for W in range(1, 33)]
        assert n == sorted(n)
        n = [lib.spec_beam_workspace_bytes(B, 4, v) for v in range(1, V, 997)]
        assert n == sorted(n)


def reorder(kvs=None, n=None, row_bytes=256, ws=F, **over):
    f = dict(B=2, W=4, block_size=16, max_blocks=8, owned_ld=40, hist_ld=100)
    f.update({n: F + 256 * i for i, n in enumerate(["parent", "tok", "seq_len", "prompt_blocks", "owned", "table_in",
                                                  "table_out", "spare_in", "spare_out", "slots", "hist_in", "hist_out"])})
    f.update(over)
    kvs = kvs or [kv()]
    a = (lib.KV * len(kvs))(*kvs)
    return call("spec_beam_reorder", ctypes.byref(lib.BeamState(**f)), len(kvs) if n is None else n, a, row_bytes, ws, None)


def test_beam_reorder_refusals():
    assert reorder(parent=None) == ARG and reorder(slots=None) == ARG and reorder(hist_in=None) == ARG
    assert reorder(table_out=F + 256 * 5) == ARG and reorder(spare_out=F + 256 * 7) == ARG      # in place
    assert reorder(hist_out=F + 256 * 10) == ARG and reorder(kvs=[kv(k=None)]) == ARG
    for kw in (dict(B=0), dict(W=33), dict(block_size=0), dict(max_blocks=0), dict(owned_ld=0), dict(hist_ld=0),
               dict(row_bytes=0), dict(n=0), dict(n=65), dict(kvs=[kv(bs=8)]), dict(kvs=[kv(slots=8)])):
        assert reorder(**kw) == SHAPE
    assert reorder(ws=F + 4) == WS
