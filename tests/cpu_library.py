"""The decoding calls of the binding on CPU tensors, by the oracle: what decode.py hands to the library, and what it
makes of the answers, without a GPU.  32-bit rows and caches.  Rows are read where a pointer and its stride say; a
row that would lie outside its tensor's memory raises."""
import ctypes

import numpy as np
import torch

from eagle_speculative_decoding_step_gb300 import binding as lib
from oracle import decode as oracle

ERR_DEVICE, ERR_CAPACITY = -6, -4


def _report(ws, code):
    word = ws[:4].view(torch.int32)
    if int(word) == 0:
        word[0] = code


def _rows(t, n, width, ld):
    """[n, width] elements from t's first one on, ld apart (0: width), as the library would take them."""
    if ld and ld < width:
        raise IndexError("rows of %d elements, %d apart" % (width, ld))
    last = t.storage_offset() + (n - 1) * (ld or width) + width
    if last * t.element_size() > t.untyped_storage().nbytes():
        raise IndexError("row %d ends %d elements past its tensor's memory" % (n - 1, last - t.untyped_storage().nbytes()
                                                                               // t.element_size()))
    return torch.as_strided(t, (n, width), (ld or width, 1), t.storage_offset())


def _at(address, dtype, *shape):
    size = int(np.prod(shape)) * np.dtype(dtype).itemsize
    return np.frombuffer((ctypes.c_char * size).from_address(address), dtype=dtype).reshape(shape)


def _cache(kv, desc):
    shape = (kv.num_slots, desc.n_kv_heads, desc.head_dim)
    return _at(kv.k, np.float32, *shape), _at(kv.v, np.float32, *shape)


def block_tables(B, block_size, max_blocks, num_blocks, len_old, len_new, table_in, table_out, free_in, n_free_in, free_out,
                 n_free_out, len_out, cu_new, slots, pos, slots_cap, ws):
    old, new = len_old.numpy().copy(), len_new.numpy().copy()
    bad = (new < 0) | (new > max_blocks * block_size)
    if bad.any():
        _report(ws, ERR_DEVICE)
    new[bad] = old[bad]
    r = oracle.block_tables(block_size, num_blocks, old, new, table_in.numpy(), free_in.numpy(), int(n_free_in[0]), slots_cap)
    if r["short"] or r["cu"][-1] > slots_cap:
        _report(ws, ERR_CAPACITY)
    outs = [(table_out, "table"), (free_out, "free"), (len_out, "length"), (cu_new, "cu"), (slots, "slots")]
    for t, name in outs + ([(pos, "pos")] if pos is not None else []):
        t.copy_(torch.from_numpy(np.asarray(r[name])).to(torch.int32).view(t.shape))
    n_free_out[0] = r["n_free"]


def cache_append(desc, k, v, ld, slots, n, kv, ws=None, v_ld=None):
    width = desc.n_kv_heads * desc.head_dim
    at = slots.numpy()
    for cache, x, step in zip(_cache(kv, desc), (k, v), (ld, ld if v_ld is None else v_ld)):
        rows = _rows(x, n, width, step).numpy().reshape(n, desc.n_kv_heads, desc.head_dim)
        cache[at[at >= 0]] = rows[at >= 0]


def paged_attention(desc, q, kv, seq_len, B, out, lse, ws, max_len=0, q_ld=0, out_ld=0):
    width = desc.n_q_heads * desc.head_dim
    rows = _rows(q, B, width, q_ld).numpy().reshape(B, desc.n_q_heads, desc.head_dim)
    table = _at(kv.block_table, np.int32, B, kv.max_blocks)
    k, v = _cache(kv, desc)
    o, l = oracle.paged_attention(rows, k, v, table, kv.block_size, seq_len.numpy(), desc.window, desc.scale)
    _rows(out, B, width, out_ld).copy_(torch.from_numpy(o.reshape(B, width)))
    if lse is not None:
        lse.copy_(torch.from_numpy(l))


def beam_select(B, W, V, dtype, logits, score, done, eos, parent, tok, score_out, done_out, ws, ld=0):
    x = _rows(logits, B * W, V, ld).numpy().reshape(B, W, V)
    r = oracle.beam_select(x, score.numpy(), done.numpy(), eos)
    for t, a in zip((parent, tok, score_out, done_out), r):
        t.copy_(torch.from_numpy(np.asarray(a)).view(t.shape))


def beam_reorder(state, kv_layers, row_bytes, ws=None):
    parent, tok, seq_len, prompt_blocks, owned, table_in, table_out, spare_in, spare_out, slots, hist_in, hist_out = state._keep
    B, W, bs = state.B, state.W, state.block_size
    r = oracle.beam_reorder(bs, parent.view(B, W).numpy(), tok.view(B, W).numpy(), seq_len.numpy(), prompt_blocks.numpy(),
                            owned.numpy(), table_in.view(B, W, -1).numpy(), spare_in.view(B, W).numpy(),
                            None if hist_in is None else hist_in.view(B, W, -1).numpy())
    # a block that is missing stays missing, and nothing is copied
    at = np.minimum(seq_len.numpy() // bs, state.max_blocks - 1)
    for b in range(B):
        for j in range(W):
            src, here = table_in.view(B, W, -1)[b, int(parent.view(B, W)[b, j]), at[b]], r["table"][b, j]
            if here[at[b]] >= 0 and seq_len[b] % bs and int(parent.view(B, W)[b, j]) != j and src < 0:
                here[at[b]] = -1
            if here[at[b]] < 0:
                r["slots"][b, j] = -1
    for t, name in ((table_out, "table"), (spare_out, "spare"), (slots, "slots"), (hist_out, "hist")):
        if t is not None:
            t.copy_(torch.from_numpy(np.asarray(r[name])).view(t.shape))
    for kv in kv_layers:
        for address in (kv.k, kv.v):
            cache = _at(address, np.uint8, kv.num_slots, row_bytes)
            for f, d, n in (c for c in r["copies"] if min(c[:2]) >= 0):
                cache[d * bs:d * bs + n] = cache[f * bs:f * bs + n]


def use(monkeypatch):
    """The binding's decoding calls go to the functions above."""
    for name, f in (("block_tables", block_tables), ("cache_append", cache_append), ("paged_attention", paged_attention),
                    ("beam_select", beam_select), ("beam_reorder", beam_reorder)):
        monkeypatch.setattr(lib, "spec_" + name, f)
    for name in ("spec_block_tables_workspace_bytes", "spec_attention_workspace_bytes", "spec_beam_workspace_bytes"):
        monkeypatch.setattr(lib, name, lambda *a: 512)
    monkeypatch.setattr(lib, "spec_get_device_error", lambda ws: int(ws[:4].view(torch.int32)))
