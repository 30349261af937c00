"""GPU parity of the calls for prompts and samples (chunk attention, token log-probabilities, forked, released and
compacted blocks) against the fp64 oracle.

Tolerances, with u the half step of a type (bf16 2^-8, f16 2^-11, fp32 2^-24):
  * a score s is a sum of hd products, each input exact: |ds| <= (hd + 4) 2^-23 S, S = max_j scale sum_c |q_c k_jc| (2^-23:
    a tensor core's sums truncate), and 2^-21 for the exponential; weights change by 2 |ds| of themselves at most (numerator
    and sum);
  * a weight enters the product with V in the type of the rows: u of itself, and 2^-34 of the largest weight in f16, which
    has no smaller numbers; fp32 rows: 0;
  * sums over n keys: n 2^-23 of the sum of magnitudes, M = sum_j p_j |v_j|;
  * the output is rounded once: u of itself.
"""
import numpy as np
import pytest
import torch

from eagle_speculative_decoding_step_gb300 import binding as lib
from oracle import prompts as oracle

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
ERR_DEVICE, ERR_CAPACITY = -6, -4
KS, VS = 0.0625, 0.03125


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def zeros(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def error(ws):
    return lib.spec_get_device_error(ws)


# ------------------------------------------------------------------ attention of a chunk of new tokens
class Chunk:
    """A batch: chunks [(new tokens, tokens in all)]."""

    def __init__(self, chunks, nq, nkv, hd, t="bf16", c=None, bs=16, window=0, seed=0, pad=3, q_off=8, sigma=1.0, scale=0.0):
        self.chunks, self.nq, self.nkv, self.hd, self.t, self.c, self.bs = chunks, nq, nkv, hd, t, c or t, bs
        self.window, self.scale = window, scale
        r = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        B = len(chunks)
        have = [-(-n // bs) for _, n in chunks]
        total = sum(have) + 3
        ids = r.permutation(total)
        self.table = np.full((B, max(have) + 2), -1)
        at = 0
        for b in range(B):
            self.table[b, :have[b]] = ids[at:at + have[b]]
            at += have[b]
        self.length = np.array([n for _, n in chunks])
        self.cu = np.concatenate([[0], np.cumsum([n for n, _ in chunks])])
        self.n = int(self.cu[-1]) + pad
        self.ks, self.vs = (KS, VS) if self.c == "e4m3" else (1.0, 1.0)
        wide = torch.randn(self.n, nq * hd + 2 * q_off, generator=g, device="cuda") * sigma
        self.wide = wide.to(TYPES[t])
        self.q = self.wide[:, q_off:q_off + nq * hd]
        self.k = (torch.randn(total * bs, nkv, hd, generator=g, device="cuda") / self.ks).to(TYPES[self.c])
        self.v = (torch.randn(total * bs, nkv, hd, generator=g, device="cuda") / self.vs).to(TYPES[self.c])
        self.desc = lib.make_attn_desc(nq, nkv, hd, t, self.c, window=window, k_scale=KS, v_scale=VS, scale=scale)
        self.num_slots = total * bs

    def slot(self, b, key):
        return int(self.table[b, key // self.bs]) * self.bs + key % self.bs

    def poison(self):
        """Whatever no row may see: slots of no request, and past a request's end."""
        used = np.zeros(self.num_slots, dtype=bool)
        for b, n in enumerate(self.length):
            used[[self.slot(b, j) for j in range(n)]] = True
        same = torch.uint8 if self.c == "e4m3" else torch.int32 if self.c == "f32" else torch.int16
        bits = {"e4m3": 0x7f, "f32": 0x7fc00000, "bf16": 0x7fc0, "f16": 0x7e00}[self.c]
        for x in (self.k, self.v):
            x.view(same)[torch.from_numpy(~used).cuda()] = bits

    def run(self, ws=None, lse=True, max_chunk=True, max_len=True, out=None, n=None):
        n = self.n if n is None else n
        ws = zeros(lib.spec_chunk_attention_workspace_bytes(self.desc, len(self.chunks), n)) if ws is None else ws
        out = torch.full((self.n, self.nq, self.hd), 7.0, device="cuda").to(TYPES[self.t]) if out is None else out
        le = torch.full((self.n, self.nq), 7.0, device="cuda") if lse else None
        kv = lib.make_kv(dict(k=self.k, v=self.v, block_table=i32(self.table), block_size=self.bs,
                              max_blocks=self.table.shape[1], num_slots=self.num_slots))
        self.args = (i32(self.cu), i32(self.length))
        lib.spec_chunk_attention(self.desc, self.q, kv, *self.args, len(self.chunks), n, out, le, ws,
                                 max_chunk=max(a for a, _ in self.chunks) if max_chunk else 0,
                                 max_len=int(self.length.max()) if max_len else 0, q_ld=self.wide.stride(0),
                                 out_ld=out.stride(0))
        return out, le, ws

    def check(self, out, lse):
        q = self.q.double().cpu().numpy().reshape(self.n, self.nq, self.hd)
        k, v = self.k.double().cpu().numpy() * self.ks, self.v.double().cpu().numpy() * self.vs
        ref, rlse, mass, size = oracle.chunk_attention(q, k, v, self.table, self.bs, self.cu, self.length, self.window,
                                                       self.scale, spread=True)
        last = int(self.cu[-1])
        got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert (got[last:] == 7).all() and (glse[last:] == 7).all()              # rows of no request
        got, glse, ref, rlse, mass, size = (x[:last] for x in (got, glse, ref, rlse, mass, size))
        n = float(self.length.max())
        ds = (self.hd + 4) * 2.0 ** -23 * size + 2.0 ** -21
        u = HALF[self.t]
        weights = 0.0 if self.t == "f32" else u
        tol = mass * (weights + 2 * ds[..., None] + n * 2.0 ** -23) + u * np.abs(ref) + 2.0 ** -24 * (self.t == "f16")
        if self.t == "f16":
            tol = tol + n * 2.0 ** -34 * np.abs(v[np.isfinite(v)]).max()
        np.testing.assert_array_equal(np.isfinite(got), np.isfinite(ref))
        ok = np.isfinite(ref)
        worst = (np.abs(got - ref)[ok] / np.maximum(tol[ok], 1e-300)).max(initial=0.0)
        assert worst <= 1.0, "out: %.3f of the tolerance" % worst
        np.testing.assert_array_equal(np.isneginf(glse), np.isneginf(rlse))
        fin = np.isfinite(rlse)
        err = np.abs(glse[fin] - rlse[fin]) - (ds + n * 2.0 ** -23 + np.abs(rlse) * 2.0 ** -22)[fin]
        assert err.max(initial=-1.0) <= 0, "lse: %.3g over the tolerance" % err.max()
        return worst


MIX = [(5, 5), (1, 300), (0, 40), (70, 200), (1, 1), (33, 33), (128, 131), (9, 0)]
TYPE_PAIRS = [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "e4m3"), ("f16", "e4m3")]


@pytest.mark.parametrize("t,c", TYPE_PAIRS)
@pytest.mark.parametrize("nq,nkv,hd", [(8, 2, 128), (4, 4, 64), (5, 1, 80), (6, 3, 96), (16, 1, 256), (4, 2, 192), (2, 1, 16),
                                       (128, 1, 32), (14, 2, 112)])
def test_chunk_attention(t, c, nq, nkv, hd):
    x = Chunk(MIX, nq, nkv, hd, t, c, seed=hd + nq)
    x.poison()
    out, lse, ws = x.run()
    assert error(ws) == 0
    x.check(out, lse)


@pytest.mark.parametrize("t,c", TYPE_PAIRS)
@pytest.mark.parametrize("bs", [1, 3, 8, 16, 24, 40, 64, 128, 256])
def test_chunk_attention_block_sizes(t, c, bs):
    x = Chunk([(40, 300), (3, 129), (200, 200), (1, 7)], 4, 2, 64, t, c, bs=bs, seed=bs)
    x.poison()
    out, lse, ws = x.run()
    assert error(ws) == 0
    x.check(out, lse)


@pytest.mark.parametrize("t,c", TYPE_PAIRS)
@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 128, 200, 5000, 2 ** 31 - 1])
def test_chunk_attention_windows(t, c, window):
    x = Chunk([(150, 420), (1, 300), (64, 64), (7, 0), (2, 500), (20, 15)], 4, 2, 128, t, c, window=window, seed=window % 1000)
    x.poison()
    out, lse, ws = x.run()
    assert error(ws) == 0
    x.check(out, lse)


@pytest.mark.parametrize("t,c,hd", [("bf16", "bf16", 128), ("f16", "f16", 64), ("bf16", "e4m3", 128), ("f32", "f32", 64),
                                    ("bf16", "bf16", 256), ("f16", "e4m3", 192)])
@pytest.mark.parametrize("chunks", [[(1, 5000)], [(3, 4097), (1, 2)], [(260, 1500)], [(600, 600)], [(1, 1)], [(0, 0), (0, 9), (2, 2)],
                                    [(1, 200)] * 40, [(129, 2000), (128, 128), (127, 127), (257, 300)]])
def test_chunk_attention_lengths(t, c, hd, chunks):
    """Single tokens over long contexts (split and joined), long chunks, many requests, requests without tokens."""
    x = Chunk(chunks, 8, 2, hd, t, c, seed=len(chunks))
    x.poison()
    for bounds in (True, False):
        out, lse, ws = x.run(max_chunk=bounds, max_len=bounds)
        assert error(ws) == 0
        x.check(out, lse)


@pytest.mark.parametrize("t,c", TYPE_PAIRS)
def test_chunk_attention_large_scores(t, c):
    """Scores far apart: the running maxima move, and weights vanish."""
    x = Chunk([(100, 700), (1, 900)], 4, 1, 64, t, c, seed=5, sigma=8.0)
    out, lse, ws = x.run()
    assert error(ws) == 0
    x.check(out, lse)


@pytest.mark.parametrize("t,c", TYPE_PAIRS)
def test_chunk_attention_rising_scores(t, c):
    """Keys in the order of their scores for one query: every tile raises the maximum."""
    x = Chunk([(1, 1000)], 1, 1, 64, t, c, bs=16, seed=11, sigma=4.0)
    k = x.k.float()[[x.slot(0, j) for j in range(1000)], 0]
    s = (k @ x.q[0, :64].float())
    at = torch.tensor([x.slot(0, j) for j in range(1000)], device="cuda")
    same = torch.uint8 if c == "e4m3" else x.k.dtype
    for reverse in (False, True):
        x.k.view(same)[at, 0] = k.to(x.k.dtype).view(same)[torch.argsort(s, descending=reverse)]
        out, lse, ws = x.run()
        x.check(out, lse)


@pytest.mark.parametrize("t,c", TYPE_PAIRS)
@pytest.mark.parametrize("hd", [64, 256])
@pytest.mark.parametrize("window", [0, 70])
def test_chunk_attention_values_that_are_not_finite(t, c, hd, window):
    """A key's V or K that is not finite reaches the rows that attend to it, and no others."""
    x = Chunk([(90, 300), (40, 40), (130, 131)], 4, 2, hd, t, c, seed=3, window=window)
    nan = torch.tensor(float("nan"), device="cuda").to(x.v.dtype).view(torch.uint8 if c == "e4m3" else x.v.dtype)
    v = x.v.view(torch.uint8) if c == "e4m3" else x.v
    for b, key, head, comp in ((0, 250, 0, 3), (0, 299, 1, 17), (1, 39, 0, 0), (1, 20, 1, 63), (2, 127, 0, 5), (2, 128, 1, 9),
                               (0, 228, 0, 40)):
        v[x.slot(b, key), head, comp] = nan
    if c != "e4m3":
        x.v[x.slot(1, 30), 1, 2] = float("inf")
        x.v[x.slot(2, 100), 0, 1] = -float("inf")
    out, lse, ws = x.run()
    assert error(ws) == 0
    x.check(out, lse)
    # a K value: the scores of rows before it do not have it
    before, blse = out.clone(), lse.clone()
    k = x.k.view(torch.uint8) if c == "e4m3" else x.k
    k[x.slot(1, 25), 0, 1] = nan
    out, lse, _ = x.run()
    row = 90 + 25
    keep = torch.ones(x.n, dtype=torch.bool, device="cuda")
    keep[row:130] = False
    assert torch.equal(out[keep].nan_to_num(3.0), before[keep].nan_to_num(3.0)) and torch.equal(lse[keep], blse[keep])
    assert not lse[row:130, :2].isfinite().any() and torch.equal(lse[row:130, 2:], blse[row:130, 2:])
    assert not out[row:130, :2].isfinite().any()


def test_chunk_attention_equal_keys_average_the_values():
    x = Chunk([(64, 200)], 2, 1, 64, "f32", "f32", seed=2)
    x.k.zero_()
    out, lse, _ = x.run()
    v = x.v.double().cpu().numpy()[[x.slot(0, j) for j in range(200)], 0]
    mean = np.cumsum(v, 0)[136:] / np.arange(137, 201)[:, None]
    np.testing.assert_allclose(out[:64, 0].double().cpu().numpy(), mean, atol=200 * 2.0 ** -23 * np.abs(v).max())
    np.testing.assert_allclose(lse[:64, 1].double().cpu().numpy(), np.log(np.arange(137, 201)), rtol=2.0 ** -20)


@pytest.mark.parametrize("t,hd", [("bf16", 128), ("f32", 64), ("bf16", 256)])
def test_chunk_attention_one_workspace_serves_all_shapes_and_repeats(t, hd):
    """Calls of all shapes in turn on one workspace; a call gives the same bits again."""
    shapes = [[(1, 4000)], [(50, 50)] * 9, [(300, 900)], [(1, 30)] * 60, [(2, 2000), (400, 400)]]
    xs = [Chunk(s, nq, nkv, hd, t, seed=i) for i, s in enumerate(shapes) for nq, nkv in ((8, 2), (3, 3))]
    ws = zeros(max(lib.spec_chunk_attention_workspace_bytes(x.desc, 60, x.n) for x in xs))
    first = [x.run(ws=ws)[:2] for x in xs]
    for x, (out, lse) in zip(xs, first):
        x.check(out, lse)
    for x, (out, lse) in list(zip(xs, first))[::-1]:
        o, le, _ = x.run(ws=ws)
        assert torch.equal(o, out) and torch.equal(le, lse)
    assert error(ws) == 0


def test_chunk_attention_many_requests():
    """More requests than one launch takes."""
    r = np.random.default_rng(0)
    chunks = [(int(n), int(n + m)) for n, m in zip(r.integers(0, 6, 2500), r.integers(0, 40, 2500))]
    for t in ("bf16", "f32"):
        x = Chunk(chunks, 2, 1, 64, t, seed=1)
        out, lse, ws = x.run()
        assert error(ws) == 0
        x.check(out, lse)


@pytest.mark.parametrize("t,c", TYPE_PAIRS)
def test_chunk_attention_bad_inputs(t, c):
    x = Chunk([(20, 100), (30, 90), (10, 50)], 4, 2, 64, t, c, seed=8)
    x.table[0, 3] = 10 ** 6                                    # a block outside the cache: its keys are left out
    out, lse, ws = x.run()
    assert error(ws) == ERR_DEVICE
    x.check(out, lse)
    x.table[0, 3] = -5
    out, lse, ws = x.run()
    assert error(ws) == ERR_DEVICE
    x.check(out, lse)
    y = Chunk([(20, 100), (30, 90), (10, 50)], 4, 2, 64, t, c, seed=8)
    ok, olse, _ = y.run()
    for cu in ([0, 20, 15, 60], [-4, 20, 50, 60], [0, 20, 50, 1000]):
        z = Chunk([(20, 100), (30, 90), (10, 50)], 4, 2, 64, t, c, seed=8)
        z.cu = np.array(cu)
        _, _, ws = z.run()
        assert error(ws) == ERR_DEVICE
    y.length[1] = 10 ** 6                                      # another request's length: the others are right
    out, lse, ws = y.run()
    assert error(ws) == ERR_DEVICE
    keep = [*range(20), *range(50, 60)]
    assert torch.equal(out[keep], ok[keep]) and torch.equal(lse[keep], olse[keep])


@pytest.mark.parametrize("t,c", TYPE_PAIRS)
def test_chunk_attention_rows_that_fall_again_and_again(t, c):
    """Requests that overlap would have more items than the workspace has counters: no row is computed, and nothing outside
    the workspace is written."""
    x = Chunk([(64, 64)] * 41, 2, 1, 64, t, c, seed=9)
    x.cu = np.array([0, x.n] * 21)
    need = lib.spec_chunk_attention_workspace_bytes(x.desc, 41, x.n)
    room = torch.full((need + 4096,), 85, dtype=torch.uint8, device="cuda")
    room[:need] = 0
    out, lse, _ = x.run(ws=room[:need])
    assert error(room[:need]) == ERR_DEVICE
    assert (out == 7).all() and (lse == 7).all() and (room[need:] == 85).all()
    room[:256] = 0                                             # the workspace serves the next call
    y = Chunk([(64, 64)] * 41, 2, 1, 64, t, c, seed=9)
    out, lse, _ = y.run(ws=room[:need])
    assert error(room[:need]) == 0
    y.check(out, lse)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_chunk_attention_output_strides_and_no_lse(t):
    x = Chunk([(37, 90), (5, 60)], 6, 3, 80, t, seed=4)
    ref, lse, _ = x.run()
    wide = torch.full((x.n, 2, 6, 80), 9.0, device="cuda").to(TYPES[t])
    x.run(out=wide[:, 1], lse=False)
    assert torch.equal(wide[:-3, 1], ref[:-3]) and (wide[:, 0] == 9).all() and (wide[-3:] == 9).all()


@pytest.mark.parametrize("t,c,hd", [("bf16", "bf16", 128), ("bf16", "e4m3", 64), ("f32", "f32", 64)])
def test_chunk_attention_in_a_graph_and_on_another_stream(t, c, hd):
    """Captured once, replayed with other lengths and on two graphs that share a workspace."""
    x = Chunk([(30, 700), (1, 65), (200, 200)], 8, 2, hd, t, c, seed=6)
    ref, rlse, ws = x.run()
    out, lse = torch.zeros_like(ref), torch.zeros_like(rlse)
    kv = lib.make_kv(dict(k=x.k, v=x.v, block_table=i32(x.table), block_size=x.bs, max_blocks=x.table.shape[1],
                          num_slots=x.num_slots))
    cu, length = i32(x.cu), i32(x.length)
    graphs = []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            lib.spec_chunk_attention(x.desc, x.q, kv, cu, length, 3, x.n, out, lse, ws, q_ld=x.wide.stride(0))
        graphs.append(g)
    for g in graphs * 2:
        out.fill_(7), lse.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(lse, rlse)
    x.length = np.array([31, 40, 199])
    x.cu = np.array([0, 3, 3, 150])
    ref, rlse, _ = x.run(max_chunk=False, max_len=False)
    cu.copy_(i32(x.cu)), length.copy_(i32(x.length))
    out.fill_(7), lse.fill_(7)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, rlse)
    assert error(ws) == 0


def test_chunk_of_one_token_is_the_decode_step():
    """The same numbers as spec_paged_attention, up to the rounding of both."""
    x = Chunk([(1, n) for n in (700, 1, 33, 64)], 8, 2, 128, "bf16", seed=9, pad=0)
    out, lse, _ = x.run()
    kv = lib.make_kv(dict(k=x.k, v=x.v, block_table=i32(x.table), block_size=x.bs, max_blocks=x.table.shape[1],
                          num_slots=x.num_slots))
    o, le = torch.empty_like(out), torch.empty_like(lse)
    ws = zeros(lib.spec_attention_workspace_bytes(x.desc, 4))
    lib.spec_paged_attention(x.desc, x.q, kv, i32(x.length), 4, o, le, ws, q_ld=x.wide.stride(0))
    # both within half a step of the output, and one rounding of the weights, of the same number; |out| <= max |v| < 5
    torch.testing.assert_close(out.float(), o.float(), atol=3 * 5 * 2.0 ** -8, rtol=0)
    torch.testing.assert_close(lse, le, atol=1e-5, rtol=0)


# ------------------------------------------------------------------ log-probabilities of given tokens
def run_logprobs(logits, tok, k, ld=0, ws=None, n=None, V=None):
    n, V = n or logits.shape[0], V or logits.shape[-1]
    f = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    i = lambda *s: torch.full(s, 7, device="cuda", dtype=torch.int32)  # noqa: E731
    o = dict(logprob=f(n), rank=i(n), entropy=f(n), lse=f(n), top_ids=i(n, max(k, 1)), top_logprob=f(n, max(k, 1)))
    if k:
        o.update(top_ids=i(n, k), top_logprob=f(n, k))
    name = {v: key for key, v in TYPES.items()}[logits.dtype]
    ws = zeros(lib.spec_token_logprobs_workspace_bytes(n, V, k)) if ws is None else ws
    lib.spec_token_logprobs(n, V, name, logits, tok, k, ws=ws, ld=ld, **o)
    return o, ws


def check_logprobs(o, logits, tok, k):
    x = logits.double().cpu().numpy()
    r = oracle.token_logprobs(x, tok.cpu().numpy(), k)
    np.testing.assert_array_equal(o["rank"].cpu().numpy(), r["rank"])
    if k:
        np.testing.assert_array_equal(o["top_ids"].cpu().numpy(), r["top_ids"])
    V = x.shape[1]
    # a sum of V exponentials (2^-22 each) in 16 or 32 of them a thread, then trees: 64 additions of 2^-24 in all; the
    # logarithm's result is below 12 and rounded to 2^-22 of it at most, as are differences of up to 2^7 against the maximum
    big = np.abs(np.where(np.isfinite(x), x, 0)).max(-1)
    spread = 2 * np.minimum(big, 3e38)
    tol = 2.0 ** -22 + 64 * 2.0 ** -24 + 12 * 2.0 ** -22 + spread * 2.0 ** -23
    for name in ("logprob", "lse"):
        got = o[name].double().cpu().numpy()
        np.testing.assert_array_equal(np.isneginf(got), np.isneginf(r[name]), err_msg=name)
        fin = np.isfinite(r[name])
        extra = (big * 2.0 ** -23 if name == "lse" else 0) + np.abs(np.where(fin, r[name], 0)) * 2.0 ** -23
        assert (np.abs(got - np.where(fin, r[name], got)) <= tol + extra)[fin].all(), name
    if k:
        got = o["top_logprob"].double().cpu().numpy()
        np.testing.assert_array_equal(np.isneginf(got), np.isneginf(r["top_logprob"]))
        fin = np.isfinite(r["top_logprob"])
        lim = (tol[:, None] + np.abs(np.where(fin, r["top_logprob"], 0)) * 2.0 ** -23)
        assert (np.abs(got - np.where(fin, r["top_logprob"], got)) <= lim)[fin].all()
    # entropy: log2 S - W / S, W = sum e t with |t| / 12 entropic weight: a few times the sums' errors times log V
    got = o["entropy"].double().cpu().numpy()
    assert (np.abs(got - r["entropy"]) <= (tol - spread * 2.0 ** -23) * (2 + np.log(V)) + spread * 2.0 ** -22).all()
    assert (got >= 0).all()


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,V,k,ld", [(1, 1, 1, 0), (3, 7, 5, 0), (5, 500, 20, 0), (2, 8191, 32, 8200), (3, 8193, 5, 0),
                                      (7, 16385, 3, 16391), (4, 40000, 0, 0), (2, 128256, 20, 0), (1, 151936, 32, 151937),
                                      (9, 33, 32, 0), (2, 300001, 5, 0)])
def test_token_logprobs(t, n, V, k, ld):
    g = torch.Generator(device="cuda").manual_seed(n + V)
    wide = (torch.randn(n, (ld or V), generator=g, device="cuda") * 3).to(TYPES[t])
    x = wide[:, :V]
    tok = torch.randint(0, V, (n,), generator=g, device="cuda", dtype=torch.int32)
    tok[0] = x[0].argmax().int()
    if n > 2:
        tok[2] = -1
        x[1, torch.rand(V, generator=g, device="cuda") < 0.5] = -float("inf")
        x[1, int(tok[1])] = -1.0
    if n > 4:
        x[3] = -float("inf")
        x[4, 0], x[4, min(V - 1, 5)] = float("nan"), float("inf")
        tok[4] = 0
    o, ws = run_logprobs(x, tok, k, ld=ld)
    assert error(ws) == 0
    check_logprobs(o, x, tok, k)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("what", ["equal", "lowest", "rising", "falling", "few", "ties", "peaked", "one", "wide"])
def test_token_logprobs_hard_rows(t, what):
    """Rows without an order to go by, sorted ones, ties, almost no finite logit, values at the ends of the type."""
    V, n, k = 20000, 2, 32
    g = torch.Generator(device="cuda").manual_seed(1)
    low, top = torch.finfo(TYPES[t]).min, torch.finfo(TYPES[t]).max
    x = torch.zeros(n, V, device="cuda")
    if what == "lowest":
        x.fill_(low)
    elif what == "rising":
        x += torch.arange(V, device="cuda") * 1e-3
    elif what == "falling":
        x -= torch.arange(V, device="cuda") * 1e-3
    elif what == "few":
        x.fill_(-float("inf"))
        x[:, ::2500] = torch.randn(n, 8, generator=g, device="cuda")
    elif what == "ties":
        x += torch.randint(0, 3, (n, V), generator=g, device="cuda")
    elif what == "peaked":
        x += torch.randn(n, V, generator=g, device="cuda")
        x[:, 777] = 60.0
    elif what == "one":
        x.fill_(-float("inf"))
        x[:, V - 1] = 3.0
    elif what == "wide":
        x += torch.randn(n, V, generator=g, device="cuda")
        x[0, 5], x[0, 6], x[1, 7] = top, low, low
    x = x.to(TYPES[t])
    tok = torch.tensor([777, V - 1], dtype=torch.int32, device="cuda")
    o, ws = run_logprobs(x, tok, k)
    assert error(ws) == 0
    check_logprobs(o, x, tok, k)


def test_token_logprobs_of_rows_at_any_address():
    g = torch.Generator(device="cuda").manual_seed(0)
    for t in ("bf16", "f32"):
        flat = torch.randn(3 * 20011 + 20, generator=g, device="cuda").to(TYPES[t])
        for off in range(9):
            x = flat[off:off + 3 * 20011].view(3, 20011)[:, :20000]
            tok = torch.tensor([0, 19999, 7], dtype=torch.int32, device="cuda")
            o, _ = run_logprobs(x, tok, 5, ld=20011)
            check_logprobs(o, x, tok, 5)


def test_token_logprobs_parts_and_bad_tokens():
    x = torch.randn(3, 5000, device="cuda")
    tok = i32([4999, 5000, -7])
    o, ws = run_logprobs(x, tok, 2)
    assert error(ws) == ERR_DEVICE
    check_logprobs(o, x, torch.tensor([4999, -1, -1]), 2)
    assert o["rank"].tolist()[1:] == [-1, -1]
    lse, ws = torch.empty(3, device="cuda"), zeros(lib.spec_token_logprobs_workspace_bytes(3, 5000, 0))
    lib.spec_token_logprobs(3, 5000, "f32", x, None, 0, None, None, None, lse, None, None, ws)
    assert torch.equal(lse, o["lse"]) and error(ws) == 0
    top, ids = torch.empty(3, 4, device="cuda"), torch.empty(3, 4, device="cuda", dtype=torch.int32)
    ws = zeros(lib.spec_token_logprobs_workspace_bytes(3, 5000, 4))
    lib.spec_token_logprobs(3, 5000, "f32", x, None, 4, None, None, None, None, ids, top, ws)
    assert torch.equal(ids[:, :2], o["top_ids"]) and torch.equal(top[:, :2], o["top_logprob"])


def test_token_logprobs_many_rows_on_one_workspace_and_in_a_graph():
    """More rows than one launch takes, then smaller calls on the same workspace, the same bits again."""
    g = torch.Generator(device="cuda").manual_seed(3)
    ws = zeros(lib.spec_token_logprobs_workspace_bytes(9000, 40000, 32))
    for n, V, k, t in ((9000, 700, 5, "bf16"), (50, 40000, 32, "f32"), (9000, 20001, 1, "f16"), (1, 40000, 7, "bf16")):
        x = torch.randn(n, V, generator=g, device="cuda").to(TYPES[t])
        tok = torch.randint(0, V, (n,), generator=g, device="cuda", dtype=torch.int32)
        o, _ = run_logprobs(x, tok, k, ws=ws)
        rows = list(range(0, n, max(1, n // 20)))
        check_logprobs({key: v[rows] for key, v in o.items()}, x[rows], tok[rows], k)
        p, _ = run_logprobs(x, tok, k, ws=ws)
        assert all(torch.equal(o[key], p[key]) for key in o)
        out = {key: torch.zeros_like(v) for key, v in o.items()}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lib.spec_token_logprobs(n, V, t, x, tok, k, ws=ws, **out)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o[key], out[key]) for key in o)
    assert error(ws) == 0


# ------------------------------------------------------------------ blocks that several requests share
def pool_case(seed, families, bs, spare, empty=0, mb=None):
    """families: (tokens of the shared prefix, [tokens of each row])."""
    r = np.random.default_rng(seed)
    rows = [n for _, x in families for n in x]
    used = sum(p // bs + sum(-(-n // bs) - p // bs for n in x) for p, x in families)
    N, B = used + spare, len(rows) + empty
    mb = mb or max(-(-n // bs) for n in rows) + 1
    ids, place = r.permutation(N), r.permutation(B)
    table, length, shared = np.full((B, mb), -1), np.zeros(B, dtype=int), np.zeros(N, dtype=int)
    at, row = 0, 0
    for p, x in families:
        w = p // bs
        mine, at = ids[at:at + w], at + w
        shared[mine] = len(x) - 1
        for n in x:
            b, more = place[row], -(-n // bs) - w
            table[b, :w], table[b, w:w + more], length[b] = mine, ids[at:at + more], n
            at, row = at + more, row + 1
    free = np.full(N, -1)
    free[:N - at] = ids[at:]
    return dict(table=table, length=length, shared=shared, free=free, n_free=N - at), place[row:], r


def families_of(seed, count, fan, most, grow):
    r = np.random.default_rng(seed)
    out = []
    for _ in range(count):
        p = int(r.integers(0, most))
        out.append((p, [p + 1 + int(x) for x in r.integers(0, grow, int(r.integers(1, fan + 1)))]))
    return out


def run_blocks(call, bs, st, in_place, *args, kv=None):
    """State after a call (and the workspace's error word)."""
    t = {k: i32(v if k != "n_free" else [v]) for k, v in st.items()}
    o = t if in_place else {k: torch.full_like(v, -77) for k, v in t.items()}
    s = lib.make_block_state(bs, t["table"], o["table"], t["length"], o["length"], t["shared"], o["shared"], t["free"], o["free"],
                             t["n_free"], o["n_free"])
    B, N = t["table"].shape[0], t["free"].numel()
    ws = torch.randint(0, 255, (lib.spec_block_state_workspace_bytes(B, N),), dtype=torch.uint8, device="cuda")
    ws[:256] = 0                                               # nothing else of it is read before it is written
    if call == "fork":
        lib.spec_block_fork(s, len(args[0]), i32(args[0]), i32(args[1]), *kv, ws)
    elif call == "release":
        lib.spec_block_release(s, i32(args[0]), ws)
    else:
        lib.spec_block_compact(s, *kv, ws)
    got = {k: v.cpu().numpy() for k, v in o.items()}
    got["n_free"] = int(got["n_free"][0])
    return got, error(ws)


def caches(layers, N, bs, nkv, hd, t):
    g = torch.Generator(device="cuda").manual_seed(7)
    kv = [torch.randn(layers, N * bs, nkv, hd, generator=g, device="cuda").to(TYPES[t]) for _ in range(2)]
    kvs = lib.make_kv_layers([dict(k=kv[0][i], v=kv[1][i], block_table=None, block_size=bs, max_blocks=0, num_slots=N * bs)
                              for i in range(layers)])
    return kv, (kvs, nkv * hd * kv[0].element_size())


def moved(kv, copies, bs):
    out = []
    for x in kv:
        y = x.clone() if x.dtype != TYPES["e4m3"] else x.view(torch.uint8).clone()
        src = x if x.dtype != TYPES["e4m3"] else x.view(torch.uint8)
        for f, t, n in copies:
            y[:, t * bs:t * bs + n] = src[:, f * bs:f * bs + n]
        out.append(y)
    return out


def same(kv, want):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(kv, want))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("live,fan,bs,spare,layers,nkv,hd,t", [
    (1, 1, 16, 3, 1, 8, 128, "bf16"), (5, 3, 16, 40, 2, 2, 64, "f16"), (40, 4, 8, 90, 3, 1, 80, "f32"), (7, 5, 1, 9, 1, 1, 16, "e4m3"),
    (3, 2, 128, 4, 2, 4, 128, "bf16"), (900, 7, 16, 6000, 1, 1, 16, "bf16"), (6, 2, 24, 5, 64, 1, 16, "bf16")])
def test_block_fork(live, fan, bs, spare, layers, nkv, hd, t, in_place):
    fam = [(p, x) for p, x in families_of(live, live, 2, 5 * bs + 20, 3 * bs + 2)]
    rows = sum(len(x) for _, x in fam)
    st, empty, r = pool_case(live + bs, fam, bs, spare, empty=live * fan)
    holders = np.nonzero(st["length"])[0]
    src, dst = holders[r.integers(0, rows, live * fan)], empty
    ref = oracle.block_fork(bs, **st, src=src, dst=dst)
    kv, args = caches(layers, len(st["free"]), bs, nkv, hd, t)
    want = moved(kv, ref["copies"], bs)
    got, err = run_blocks("fork", bs, st, in_place, src, dst, kv=args)
    assert not ref["bad"] and err == (ERR_CAPACITY if ref["short"] else 0)
    for k in ("table", "length", "shared", "free", "n_free"):
        np.testing.assert_array_equal(got[k], ref[k], err_msg=k)
    assert same(kv, want)


@pytest.mark.parametrize("in_place", [False, True])
def test_block_fork_bad_forks(in_place):
    """Rows outside the batch, a row that is not empty, the same row twice, an empty source, bad ids and lengths."""
    st, empty, _ = pool_case(3, [(20, [30, 25]), (0, [9])], 8, 6, empty=5)
    a, b = np.nonzero(st["length"] == 30)[0][0], np.nonzero(st["length"] == 9)[0][0]
    e = empty
    src = [a, a, b, e[1], 99, a, -1]
    dst = [e[0], e[0], a, e[2], e[3], -3, e[3]]
    kv, args = caches(1, len(st["free"]), 8, 1, 16, "bf16")
    ref = oracle.block_fork(8, **st, src=src, dst=dst)
    want = moved(kv, ref["copies"], 8)
    got, err = run_blocks("fork", 8, st, in_place, src, dst, kv=args)
    assert ref["bad"] and err == ERR_DEVICE and same(kv, want)
    for k in ("table", "length", "shared", "free", "n_free"):
        np.testing.assert_array_equal(got[k], ref[k], err_msg=k)
    for bad in (-3, 10 ** 6):                                  # an id in the source's table, and in the pool
        for where in ("table", "free"):
            s2 = {k: np.array(v) for k, v in st.items()}
            if where == "table":
                s2["table"][a, 1], s2["table"][b, 1] = bad, bad
            else:
                s2["free"][s2["n_free"] - 1] = bad
            ref = oracle.block_fork(8, **s2, src=[a, b], dst=[e[0], e[1]])
            kv, args = caches(1, len(st["free"]), 8, 1, 16, "bf16")
            want = moved(kv, ref["copies"], 8)
            got, err = run_blocks("fork", 8, s2, in_place, [a, b], [e[0], e[1]], kv=args)
            assert err == ERR_DEVICE and same(kv, want)
            for k in ("table", "length", "shared", "n_free"):
                np.testing.assert_array_equal(got[k], ref[k], err_msg=k)
    s2 = {k: np.array(v) for k, v in st.items()}
    s2["length"][a] = 10 ** 6
    got, err = run_blocks("fork", 8, s2, in_place, [a], [e[0]], kv=args)
    assert err == ERR_DEVICE and got["length"][e[0]] == 0 and got["n_free"] == st["n_free"]
    s2["length"][a], s2["n_free"] = 30, 10 ** 6
    _, err = run_blocks("fork", 8, s2, False, [a], [e[0]], kv=args)
    assert err == ERR_DEVICE


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("live,fan,bs,most,share", [(1, 1, 16, 40, 1.0), (6, 4, 16, 300, 0.5), (200, 5, 8, 200, 0.6),
                                                    (1500, 5, 16, 60, 0.3), (3, 40, 1, 50, 0.9), (20, 3, 16, 500, 0.0),
                                                    (300, 5, 8, 900, 0.5)])
def test_block_release(live, fan, bs, most, share, in_place):
    st, _, r = pool_case(live, families_of(live, live, fan, most, 3 * bs), bs, 10)
    drop = (r.random(len(st["length"])) < share).astype(int) * 5
    ref = oracle.block_release(bs, **st, drop=drop)
    got, err = run_blocks("release", bs, st, in_place, drop)
    assert not ref["bad"] and err == 0
    for k in ("table", "length", "shared", "free", "n_free"):
        np.testing.assert_array_equal(got[k], ref[k], err_msg=k)


@pytest.mark.parametrize("in_place", [False, True])
def test_block_release_bad_rows(in_place):
    st, _, _ = pool_case(5, [(40, [50, 60, 45]), (0, [20])], 8, 4)
    first, other = np.nonzero(st["length"] == 50)[0][0], np.nonzero(st["length"] == 20)[0][0]
    drop = np.ones(4, dtype=int)
    for change in (lambda s: s["table"].__setitem__((first, 1), 10 ** 6), lambda s: s["length"].__setitem__(other, -2),
                   lambda s: s["shared"].__setitem__(s["table"][first, 0], 0)):
        s2 = {k: np.array(v) for k, v in st.items()}
        change(s2)
        ref = oracle.block_release(8, **s2, drop=drop)
        got, err = run_blocks("release", 8, s2, in_place, drop)
        assert ref["bad"] and err == ERR_DEVICE
        for k in ("table", "length", "shared", "free", "n_free"):
            np.testing.assert_array_equal(got[k], ref[k], err_msg=k)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("live,fan,bs,most,spare,layers,nkv,hd,t", [
    (1, 1, 16, 40, 0, 1, 2, 64, "bf16"), (4, 3, 16, 200, 30, 2, 2, 64, "f16"), (50, 3, 8, 150, 900, 2, 1, 80, "f32"),
    (300, 4, 16, 90, 3000, 1, 1, 16, "e4m3"), (9, 2, 1, 30, 17, 1, 3, 16, "bf16"), (2, 2, 128, 600, 90, 3, 2, 128, "bf16"),
    (2, 1, 16, 40, 40000, 1, 1, 16, "bf16")])
def test_block_compact(live, fan, bs, most, spare, layers, nkv, hd, t, in_place):
    st, _, _ = pool_case(live + 1, families_of(live, live, fan, most, 2 * bs), bs, spare, empty=2)
    ref = oracle.block_compact(bs, **st)
    kv, args = caches(layers, len(st["free"]), bs, nkv, hd, t)
    want = moved(kv, ref["copies"], bs)
    got, err = run_blocks("compact", bs, st, in_place, kv=args)
    assert not ref["refused"] and err == 0
    for k in ("table", "length", "shared", "free", "n_free"):
        np.testing.assert_array_equal(got[k], ref[k], err_msg=k)
    assert same(kv, want)


@pytest.mark.parametrize("in_place", [False, True])
def test_block_compact_refuses_a_pool_it_does_not_see_all_of(in_place):
    st, _, _ = pool_case(2, [(16, [30, 40]), (3, [8])], 8, 9)
    kv, args = caches(1, len(st["free"]), 8, 1, 16, "bf16")
    before = [x.clone() for x in kv]
    row = np.nonzero(st["length"] == 30)[0][0]
    changes = ((lambda s: s.__setitem__("n_free", s["n_free"] - 1), ERR_CAPACITY),
               (lambda s: s["table"].__setitem__((row, 1), -4), ERR_DEVICE), (lambda s: s["length"].__setitem__(row, 10 ** 5), ERR_DEVICE))
    for change, code in changes:
        s2 = {k: np.array(v) for k, v in st.items()}
        change(s2)
        got, err = run_blocks("compact", 8, s2, in_place, kv=args)
        assert err in (code, ERR_CAPACITY) and same(kv, before)
        for k in ("table", "length", "shared", "n_free"):
            np.testing.assert_array_equal(got[k], s2[k], err_msg=k)
        np.testing.assert_array_equal(got["free"][:s2["n_free"]], s2["free"][:s2["n_free"]])


def test_copies_of_rows_of_any_size():
    """Slots of 1 to 96 bytes, at addresses that no vector fits."""
    for row, off in ((1, 0), (6, 2), (12, 4), (34, 1), (96, 16), (20, 4)):
        st, empty, _ = pool_case(1, [(0, [13]), (0, [30])], 8, 9, empty=2)
        src, dst = np.nonzero(st["length"])[0], empty
        N = len(st["free"])
        flat = torch.randint(0, 255, (N * 8 * row + 64,), dtype=torch.uint8, device="cuda")
        base = flat[off:off + N * 8 * row]
        ref = oracle.block_fork(8, **st, src=src, dst=dst)
        want = base.clone().view(N * 8, row)
        for f, t, n in ref["copies"]:
            want[t * 8:t * 8 + n] = base.view(N * 8, row)[f * 8:f * 8 + n]
        kvs = lib.make_kv_layers([dict(k=base, v=base, block_table=None, block_size=8, max_blocks=0, num_slots=N * 8)])
        _, err = run_blocks("fork", 8, st, False, src, dst, kv=(kvs, row))
        assert err == 0 and torch.equal(base.view(N * 8, row), want)


def test_blocks_in_a_graph():
    """Fork, release, compact captured together: the state comes back to where it was, again and again."""
    bs = 8
    st, empty, _ = pool_case(4, [(20, [30, 41]), (5, [9])], bs, 30, empty=3)
    t = {k: i32(v if k != "n_free" else [v]) for k, v in st.items()}
    s = lib.make_block_state(bs, t["table"], t["table"], t["length"], t["length"], t["shared"], t["shared"], t["free"], t["free"],
                             t["n_free"], t["n_free"])
    kv, args = caches(2, len(st["free"]), bs, 1, 16, "bf16")
    src, dst, drop = i32(np.nonzero(st["length"])[0]), i32(empty), torch.zeros(6, dtype=torch.int32, device="cuda")
    drop[torch.from_numpy(empty).cuda()] = 1
    ws = zeros(lib.spec_block_state_workspace_bytes(6, len(st["free"])))
    lib.spec_block_compact(s, *args, ws)
    torch.cuda.synchronize()
    start = {k: v.clone() for k, v in t.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.spec_block_fork(s, 3, src, dst, *args, ws)
        lib.spec_block_release(s, drop, ws)
        lib.spec_block_compact(s, *args, ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert error(ws) == 0
    for k in t:
        assert torch.equal(t[k], start[k]), k
