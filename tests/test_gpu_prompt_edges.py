"""GPU cases at the edges of the calls for prompts and samples, against the fp64 oracle (tolerances: test_gpu_prompts)."""
import numpy as np
import pytest
import torch

from eagle_speculative_decoding_step_gb300 import binding as lib
from eagle_speculative_decoding_step_gb300 import decode
from oracle import prompts as oracle
from test_gpu_prompts import HALF, TYPE_PAIRS, TYPES, Chunk, caches, error, i32, moved, pool_case, run_blocks, same

pytestmark = pytest.mark.gpu
ERR_TIMEOUT = -7


def far_below_zero(x, at=225.0):
    """Every score of x near -at: q = -a (1, 1, ...) + noise, k = 4 (1, 1, ...) + noise, 4 a sqrt(hd) = at."""
    g = torch.Generator(device="cuda").manual_seed(17)
    a = at / (4 * x.hd ** 0.5)
    x.wide.copy_(0.5 * torch.randn(x.wide.shape, generator=g, device="cuda") - a)
    same = torch.uint8 if x.c == "e4m3" else x.k.dtype
    k = ((4 + 0.5 * torch.randn(x.k.shape, generator=g, device="cuda")) / x.ks).to(TYPES[x.c])
    x.k.view(same).copy_(k.view(same))


@pytest.mark.parametrize("t,c", TYPE_PAIRS)
@pytest.mark.parametrize("hd", [64, 256])
@pytest.mark.parametrize("chunks,window", [([(40, 300), (3, 3)], 0),              # whole items
                                           ([(1, 5000)], 0), ([(3, 4100), (1, 2)], 0),     # pieces of one row's keys
                                           ([(150, 420), (1, 300)], 70),          # rows that see nothing of an item's first tile
                                           ([(200, 1900)], 700)])                 # or of a piece
def test_chunk_attention_scores_far_below_zero(t, c, hd, chunks, window):
    """The first scores that a row sees are no reference of 0: 2^(0 - s) would overflow."""
    x = Chunk(chunks, 4, 2, hd, t, c, window=window, seed=21)
    far_below_zero(x)
    out, lse, ws = x.run()
    assert error(ws) == 0
    x.check(out, lse)
    assert (lse[:int(x.cu[-1])] < -150).all()


@pytest.mark.parametrize("in_place", [False, True])
def test_block_fork_of_an_empty_row_leaves_no_entries(in_place):
    """Rows without tokens whose table entries are whatever was there: a copy of one holds nothing, its entries are -1."""
    st, empty, _ = pool_case(3, [(20, [30, 25]), (0, [9])], 8, 6, empty=4)
    a = np.nonzero(st["length"] == 30)[0][0]
    for row in empty:
        st["table"][row] = np.arange(st["table"].shape[1]) + row
    src, dst = [empty[0], a, empty[0]], [empty[1], empty[2], empty[3]]
    kv, args = caches(1, len(st["free"]), 8, 1, 16, "bf16")
    ref = oracle.block_fork(8, **st, src=src, dst=dst)
    want = moved(kv, ref["copies"], 8)
    got, err = run_blocks("fork", 8, st, in_place, src, dst, kv=args)
    assert err == 0 and not ref["bad"] and same(kv, want)
    for k in ("table", "length", "shared", "free", "n_free"):
        np.testing.assert_array_equal(got[k], ref[k], err_msg=k)
    assert (got["table"][[empty[1], empty[3]]] == -1).all() and (got["table"][empty[0]] == st["table"][empty[0]]).all()


def test_chunks_in_a_graph_while_other_batches_need_more_room():
    """A captured pass works on the workspace that it was captured with after larger calls have got another one."""
    nq, nkv, hd = 4, 2, 64
    c = decode.PagedCache(1, 400, 16, nq, nkv, hd, max_rows=8)
    g = torch.Generator(device="cuda").manual_seed(2)

    def chunk(n, first):
        """Slots of one request's n tokens from block `first` on, and what the attention takes and is called with."""
        table = torch.arange(first, first + 100, dtype=torch.int32, device="cuda").view(1, 100)
        slots = torch.arange(first * 16, first * 16 + n, dtype=torch.int32, device="cuda")
        cu, length = i32([0, n]), i32([n])
        q, k, v = (torch.randn(n, h, hd, generator=g, device="cuda").bfloat16() for h in (nq, nkv, nkv))
        return (c.views(table), slots, cu, length), (0, q, k, v)
    at, qkv = chunk(200, 0)
    want = c.attend_chunks(*at)(*qkv).clone()
    old = c.chunk_ws
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = c.attend_chunks(*at)(*qkv)
    data = old.data_ptr()
    del old
    big, other = chunk(1500, 150)
    c.attend_chunks(*big)(*other)
    assert c.chunk_ws.data_ptr() != data and [w.data_ptr() for w in c.captured_ws] == [data]
    mine = torch.full((64 << 20,), 85, dtype=torch.uint8, device="cuda")          # what the pool would have given that memory to
    for _ in range(2):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert (mine == 85).all() and c.error() == 0
    table, slots, cu, length = chunk(5000 // 16 * 16, 0)[0]
    with pytest.raises(RuntimeError, match="before it is captured"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            c.attend_chunks(table, slots, cu, length)


SIXTEEN = [p for p in TYPE_PAIRS if p[0] != "f32"]
# few rows (128 packed ones at most), many, and head sizes above 128: keys that are shared out differently
FORMS = [(64, [(4, 3000), (8, 40), (1, 1), (0, 9)], 0), (128, [(30, 2500), (1, 700)], 600), (80, [(1, 260)] * 20, 0),
         (128, [(150, 420), (260, 1500)], 300), (256, [(150, 700), (3, 2500)], 0), (192, [(90, 420), (2, 2)], 70)]


@pytest.mark.parametrize("t,c", SIXTEEN)
@pytest.mark.parametrize("bs", [1, 8, 24])
@pytest.mark.parametrize("hd,chunks,window", FORMS)
def test_chunk_attention_blocks_without_runs_of_16(t, c, bs, hd, chunks, window):
    """Whole and split items, windows, batches of single tokens, in blocks that are no multiple of 16 slots."""
    x = Chunk(chunks, 4, 2, hd, t, c, bs=bs, window=window, seed=hd + bs)
    x.poison()
    out, lse, ws = x.run()
    assert error(ws) == 0
    x.check(out, lse)


@pytest.mark.parametrize("t,c", SIXTEEN)
@pytest.mark.parametrize("bs", [8, 16, 24])
@pytest.mark.parametrize("hd,chunks,window", [(64, [(40, 300), (30, 30), (55, 131)], 0), (128, [(40, 300), (30, 30), (55, 1200)], 50),
                                              (256, [(90, 300), (40, 40), (30, 900)], 0), (192, [(90, 300), (40, 40), (130, 131)], 70),
                                              (128, [(90, 300), (40, 40), (130, 900)], 0)])
def test_chunk_attention_values_that_are_not_finite_in_any_block(t, c, bs, hd, chunks, window):
    """A key's V that is not finite, among each request's newest keys and where a window begins."""
    x = Chunk(chunks, 4, 2, hd, t, c, bs=bs, seed=3, window=window)
    v = x.v.view(torch.uint8) if c == "e4m3" else x.v
    nan = torch.tensor(float("nan"), device="cuda").to(x.v.dtype).view(v.dtype)
    for b, (n, length) in enumerate(chunks):
        first = length - n
        for key, head, comp in ((first, 0, 3), (first + n // 2, 1, 17), (length - 1, 0, hd - 1), (max(0, first - window + n // 3), 1, 0)):
            v[x.slot(b, key), head, comp] = nan
    out, lse, ws = x.run()
    assert error(ws) == 0
    x.check(out, lse)


def hold(ws, cta):
    ws[64:68].copy_(torch.tensor([cta], dtype=torch.int32).view(torch.uint8))


WAITS = [("bf16", "bf16", 64, [(300, 2000)], 16), ("f16", "f16", 64, [(8, 3000), (8, 40)], 16), ("bf16", "bf16", 256, [(20, 2000)], 24),
         ("bf16", "e4m3", 128, [(300, 2000)], 16), ("f16", "e4m3", 64, [(4, 3000)], 16), ("bf16", "bf16", 64, [(8, 60)], 16)]


@pytest.mark.parametrize("t,c,hd,chunks,bs", WAITS)
def test_chunk_attention_waits_that_run_out(t, c, hd, chunks, bs):
    """A CTA that never gets its keys gives up after the limit: the call ends and says so, and the next call is right."""
    x = Chunk(chunks, 4, 2, hd, t, c, bs=bs, seed=31)
    ref, rlse, ws = x.run()
    assert error(ws) == 0
    hold(ws, 2)
    x.run(ws=ws)
    torch.cuda.synchronize()
    assert error(ws) == ERR_TIMEOUT
    out, lse, other = x.run()
    assert error(other) == 0 and torch.equal(out, ref) and torch.equal(lse, rlse)


@pytest.mark.parametrize("t,c,hd,chunks,bs", WAITS)
@pytest.mark.parametrize("cta", [1, 20])
def test_chunk_attention_after_waits_that_ran_out(t, c, hd, chunks, bs, cta):
    """Pieces of items that a CTA gave up on are counted all the same: the workspace serves the next call."""
    x = Chunk(chunks, 4, 2, hd, t, c, bs=bs, seed=31)
    ref, rlse, ws = x.run()
    hold(ws, cta)
    x.run(ws=ws)
    torch.cuda.synchronize()
    assert error(ws) == (ERR_TIMEOUT if cta <= 2 or chunks[0][1] > 60 else 0)      # (60 keys: two items, of a CTA each)
    first = lib.spec_chunk_attention_workspace_bytes(x.desc, 1, 1) - 256           # (a call of one row has a few counters)
    assert not ws[first:].any()
    lib.spec_clear_device_error(ws)
    out, lse, _ = x.run(ws=ws)
    assert error(ws) == 0 and torch.equal(out, ref) and torch.equal(lse, rlse)


@pytest.mark.parametrize("t,c", TYPE_PAIRS)
def test_chunks_of_one_token_and_the_decode_step(t, c):
    """spec_paged_attention's answer, up to what the two lose: a weight's rounding to the type of the rows here (u of it, and in
    f16 2^-34 of the largest) and 2^-17 of it there, of M = sum p |v|; both outputs' rounding, u of them; and the scores' and
    sums' (test_gpu_prompts), which the two do in different orders."""
    x = Chunk([(1, n) for n in (700, 1, 33, 64, 1500, 260)], 8, 2, 128, t, c, seed=9, pad=0)
    out, lse, _ = x.run()
    o, le = torch.empty_like(out), torch.empty_like(lse)
    ws = torch.zeros(lib.spec_attention_workspace_bytes(x.desc, 6), dtype=torch.uint8, device="cuda")
    kv = lib.make_kv(dict(k=x.k, v=x.v, block_table=i32(x.table), block_size=x.bs, max_blocks=x.table.shape[1],
                          num_slots=x.num_slots))
    lib.spec_paged_attention(x.desc, x.q, kv, i32(x.length), 6, o, le, ws, q_ld=x.wide.stride(0))
    q = x.q.double().cpu().numpy().reshape(x.n, x.nq, x.hd)
    k, v = x.k.double().cpu().numpy() * x.ks, x.v.double().cpu().numpy() * x.vs
    ref, rlse, mass, size = oracle.chunk_attention(q, k, v, x.table, x.bs, x.cu, x.length, spread=True)
    n, u = 1500.0, HALF[t]
    ds = 2 * ((x.hd + 4) * 2.0 ** -23 * size + 2.0 ** -21)
    tol = mass * ((0.0 if t == "f32" else u + 2.0 ** -17) + 2 * ds[..., None] + 2 * n * 2.0 ** -23) + 2 * u * np.abs(ref)
    if t == "f16":
        tol = tol + n * 2.0 ** -34 * np.abs(v).max() + 2 * 2.0 ** -24
    tol = tol * (1 + 4 * u)                                    # (products of two of these)
    far, lfar = (np.abs(a.double().cpu().numpy() - b.double().cpu().numpy()) for a, b in ((out, o), (lse, le)))
    assert (far / tol).max() <= 1.0, "%.3f of the tolerance" % (far / tol).max()
    assert (lfar <= ds + 2 * n * 2.0 ** -23 + np.abs(rlse) * 2.0 ** -21).all()
