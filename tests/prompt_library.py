"""The calls for prompts and samples on CPU tensors, by the oracle, beside cpu_library's decoding calls."""
import numpy as np
import torch

import cpu_library as base
from eagle_speculative_decoding_step_gb300 import binding as lib
from oracle import prompts as oracle


def chunk_attention(desc, q, kv, cu_rows, seq_len, B, n_rows, out, lse, ws, max_chunk=0, max_len=0, q_ld=0, out_ld=0):
    width = desc.n_q_heads * desc.head_dim
    rows = base._rows(q, n_rows, width, q_ld).numpy().reshape(n_rows, desc.n_q_heads, desc.head_dim)
    table = base._at(kv.block_table, np.int32, B, kv.max_blocks)
    k, v = base._cache(kv, desc)
    o, l = oracle.chunk_attention(rows, k, v, table, kv.block_size, cu_rows.numpy(), seq_len.numpy(), desc.window, desc.scale)
    last = int(cu_rows[-1])
    base._rows(out, n_rows, width, out_ld)[:last].copy_(torch.from_numpy(o.reshape(n_rows, width)[:last]))
    if lse is not None:
        lse[:last].copy_(torch.from_numpy(l[:last]))


def token_logprobs(n, V, dtype, logits, tok, k, logprob, rank, entropy, lse, top_ids, top_logprob, ws, ld=0):
    r = oracle.token_logprobs(base._rows(logits, n, V, ld).numpy(), tok.numpy(), k)
    for name, t in dict(logprob=logprob, rank=rank, entropy=entropy, lse=lse, top_ids=top_ids, top_logprob=top_logprob).items():
        t.copy_(torch.from_numpy(np.asarray(r[name])))


def _state(st):
    t = st._keep
    return dict(zip(("table", "length", "shared", "free"), (x.numpy() for x in t[0:8:2])), n_free=int(t[8]))


def _put(st, r):
    for x, name in zip(st._keep[1:8:2], ("table", "length", "shared", "free")):
        x.copy_(torch.from_numpy(r[name]).to(torch.int32))
    st._keep[9][0] = r["n_free"]


def _move(kv_layers, row_bytes, bs, copies):
    for kv in kv_layers:
        for address in (kv.k, kv.v):
            cache = base._at(address, np.uint8, kv.num_slots, row_bytes)
            for f, d, n in copies:
                cache[d * bs:d * bs + n] = cache[f * bs:f * bs + n]


def block_fork(st, n, src, dst, kv_layers, row_bytes, ws):
    r = oracle.block_fork(st.block_size, **_state(st), src=src.numpy(), dst=dst.numpy())
    if r["bad"] or r["short"]:
        base._report(ws, base.ERR_DEVICE if r["bad"] else base.ERR_CAPACITY)
    _put(st, r)
    _move(kv_layers, row_bytes, st.block_size, r["copies"])


def block_release(st, drop, ws):
    r = oracle.block_release(st.block_size, **_state(st), drop=drop.numpy())
    if r["bad"]:
        base._report(ws, base.ERR_DEVICE)
    _put(st, r)


def block_compact(st, kv_layers, row_bytes, ws):
    r = oracle.block_compact(st.block_size, **_state(st))
    if r["refused"]:
        base._report(ws, base.ERR_CAPACITY)
    _put(st, r)
    _move(kv_layers, row_bytes, st.block_size, r["copies"])


def use(monkeypatch):
    base.use(monkeypatch)
    for f in (chunk_attention, token_logprobs, block_fork, block_release, block_compact):
        monkeypatch.setattr(lib, "spec_" + f.__name__, f)
    for name in ("chunk_attention", "token_logprobs", "block_state"):
        monkeypatch.setattr(lib, "spec_%s_workspace_bytes" % name, lambda *a: 512)
