"""GPU cases at the edges of the calls for prompts and samples, against the fp64 oracle (tolerances: test_gpu_prompts)."""
import numpy as np
import pytest
import torch

from eagle_speculative_decoding_step_gb300 import decode
from oracle import prompts as oracle
from test_gpu_prompts import TYPE_PAIRS, TYPES, Chunk, caches, error, i32, moved, pool_case, run_blocks, same

pytestmark = pytest.mark.gpu


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
