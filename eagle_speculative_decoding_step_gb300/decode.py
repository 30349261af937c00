"""Decoding without speculation over the paged K/V cache, on libeaglespec: requests
that are too many to speculate on, or that ask for beams.

``PagedCache`` owns the K/V tensors of all layers, the pool of free blocks and the
workspaces.  ``Batch`` decodes one continuation a request: every step the block
tables grow (and finished requests give their blocks back), the new rows are
appended, each new token attends to its request's cache, and the best token is
selected.  ``BeamBatch`` decodes W beams a request: after every selection the beams'
tables, histories and partial blocks are reordered.  [NEURON] "Speculative Decoding
(EAGLE3) in the vLLM Neuron Framework", "KV Cache Sharing" and "EagleProposer": the
cache, its block tables and slot mapping.

A model is a callable ``model(tok, pos, attend) -> logits``: tok and pos [n] int32,
logits [n, V]; in each layer it calls ``attend(layer, q, k, v)`` with q [n, nq, hd],
k and v [n, nkv, hd] of the new tokens and gets [n, nq, hd].  Everything between the
model's own operators is a library call on the current stream, without a host
synchronisation.

``python -m eagle_speculative_decoding_step_gb300.decode`` decodes with a small
random model (``RandomModel``).
"""
import numpy as np
import torch

from . import binding as lib

_LOGITS = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}
_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


def _ints(*shape, device, fill=0):
    return torch.full(shape, fill, dtype=torch.int32, device=device)


def _rows(x, n, heads, hd, dtype, name):
    """x [n, heads, hd] or [n, heads * hd] as rows (copied if a row is not in one piece), and the
    elements from one to the next."""
    at, step = x.shape, x.stride()
    if at == (n, heads, hd) and x.dtype == dtype and step[2] == 1 and step[1] == hd and step[0] >= heads * hd:
        return x, step[0]
    whole = x.numel() == n * heads * hd and x.shape[0] == n
    if not whole or x.dtype != dtype or tuple(x.shape[-2:]) not in ((heads, hd), (n, heads * hd)):
        raise ValueError("%s is %s %s, the cache takes %s %s" % (name, x.dtype, tuple(x.shape), dtype, (n, heads, hd)))
    x = x.reshape(n, heads * hd)
    if x.stride(1) != 1 or (n > 1 and x.stride(0) < heads * hd):
        x = x.contiguous()
    return x, x.stride(0) if n > 1 else heads * hd


class PagedCache:
    """K/V of ``layers`` layers in ``num_blocks`` blocks of ``block_size`` slots, and the
    pool of free blocks."""

    def __init__(self, layers, num_blocks, block_size, n_q_heads, n_kv_heads, head_dim, dtype="bf16", kv_dtype=None,
                 k_scale=1.0, v_scale=1.0, window=0, max_rows=64, device="cuda"):
        self.layers, self.num_blocks, self.block_size, self.device = layers, num_blocks, block_size, device
        self.n_q_heads, self.n_kv_heads, self.head_dim, self.dtype = n_q_heads, n_kv_heads, head_dim, _TORCH[dtype]
        self.desc = lib.make_attn_desc(n_q_heads, n_kv_heads, head_dim, dtype, kv_dtype, window=window, k_scale=k_scale,
                                       v_scale=v_scale)
        stored = _TORCH[kv_dtype or dtype]
        shape = (layers, num_blocks * block_size, n_kv_heads, head_dim)
        same = torch.uint8 if stored == torch.float8_e4m3fn else stored        # zero bits are zeros in every type
        self.k, self.v = (torch.zeros(shape, dtype=same, device=device).view(stored) for _ in range(2))
        self.row_bytes = n_kv_heads * head_dim * self.k.element_size()
        self.free = torch.arange(num_blocks - 1, -1, -1, dtype=torch.int32, device=device)
        self.n_free = _ints(1, device=device, fill=num_blocks)
        self.ws = torch.zeros(lib.spec_attention_workspace_bytes(self.desc, max_rows), dtype=torch.uint8, device=device)
        self.max_rows = max_rows

    def views(self, table):
        """KV structs of all layers under a block table."""
        return lib.make_kv_layers([dict(k=self.k[i], v=self.v[i], block_table=table, block_size=self.block_size,
                                        max_blocks=table.shape[1], num_slots=self.k.shape[1])
                                   for i in range(self.layers)])

    def attend(self, kvs, slots, seq_len, max_len=0):
        """The ``attend`` of a model whose row i writes slot slots[i] and then attends to its
        request's first seq_len[i] cache entries.  q, k and v are of the cache's row type, each with
        strides of its own."""
        n = slots.numel()
        if n > self.max_rows:
            raise ValueError("%d rows, the cache was made for %d" % (n, self.max_rows))

        def call(layer, q, k, v):
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            q, q_ld = _rows(q, n, self.n_q_heads, self.head_dim, self.dtype, "q")
            k, k_ld = _rows(k, n, self.n_kv_heads, self.head_dim, self.dtype, "k")
            v, v_ld = _rows(v, n, self.n_kv_heads, self.head_dim, self.dtype, "v")
            lib.spec_cache_append(self.desc, k, v, k_ld, slots, n, kvs[layer], self.ws, v_ld=v_ld)
            lib.spec_paged_attention(self.desc, q, kvs[layer], seq_len, n, out, None, self.ws, max_len=max_len, q_ld=q_ld)
            return out
        return call

    def error(self):
        """The attention's error word (synchronises)."""
        return lib.spec_get_device_error(self.ws)


class _Select:
    """Selection of W continuations for B requests, double-buffered scores."""

    def __init__(self, B, W, V, eos, device):
        self.B, self.W, self.V, self.eos = B, W, V, eos
        self.ws = torch.zeros(lib.spec_beam_workspace_bytes(B, W, V), dtype=torch.uint8, device=device)
        self.score = [torch.zeros(B, W, device=device) for _ in range(2)]
        self.done = [_ints(B, W, device=device) for _ in range(2)]
        self.parent, self.tok = _ints(B, W, device=device), _ints(B, W, device=device)
        self.at = 0

    def __call__(self, logits):
        """logits [B * W, V] in fp32, bf16 or fp16 (copied if a row is not in one piece)."""
        n, V, a, b = self.B * self.W, self.V, self.at, 1 - self.at
        name = _LOGITS.get(logits.dtype)
        if name is None or logits.numel() != n * V or logits.shape[-1] != V:
            raise ValueError("logits are %s %s, not %s of floats" % (logits.dtype, tuple(logits.shape), (n, V)))
        x = logits.reshape(n, V)
        if x.stride(1) != 1 or (n > 1 and x.stride(0) < V):
            x = x.contiguous()
        lib.spec_beam_select(self.B, self.W, V, name, x, self.score[a], self.done[a], self.eos, self.parent, self.tok,
                             self.score[b], self.done[b], self.ws, ld=x.stride(0) if n > 1 else V)
        self.at = b

    def begin(self):
        """Every beam live, with score 0."""
        self.score[self.at].zero_()
        self.done[self.at].zero_()

    def finish(self, which):
        """The beams of which [B, W] select nothing more."""
        self.done[self.at] |= which


class Batch:
    """One continuation a request (a batch of up to B requests of up to max_len tokens).

    A request that cannot take another token, because its table is full or the pool has no block for
    it, is ``stopped`` [B]: it keeps its blocks and length, its tokens are -1 from there on, and
    ``error`` says what was missing.  The others go on.  A request that has selected the end token gives
    its blocks back with the next ``feed`` and goes on selecting that token; ``release`` ends all of them."""

    def __init__(self, model, cache, B, max_len, vocab, eos=-1):
        self.model, self.cache, self.B = model, cache, B
        dev, mb = cache.device, -(-max_len // cache.block_size)
        self.max_len = mb * cache.block_size
        self.length = _ints(B, device=dev)
        self.table = _ints(B, mb, device=dev, fill=-1)
        self.kvs = cache.views(self.table)
        self.slots, self.pos = _ints(B + 1, device=dev), _ints(B + 1, device=dev)      # (one past the end for cu's last)
        self.cu = _ints(B + 1, device=dev)
        self.tws = torch.zeros(lib.spec_block_tables_workspace_bytes(B), dtype=torch.uint8, device=dev)
        self.live, self.kept = _ints(B, device=dev, fill=1), _ints(B, device=dev, fill=1)    # takes tokens; keeps its blocks
        self.select = _Select(B, 1, vocab, eos, dev)

    @property
    def stopped(self):
        return self.kept > self.live

    def resize(self, want):
        """Grow to (or give back down to) want [B] tokens by at most B new ones in all: their slots and
        positions are in ``slots`` and ``pos``, those of request b from ``cu``[b] on (a request that is
        refused for its length has none there)."""
        c = self.cache
        lib.spec_block_tables(self.B, c.block_size, self.table.shape[1], c.num_blocks, self.length, want, self.table,
                              self.table, c.free, c.n_free, c.free, c.n_free, self.length, self.cu, self.slots, self.pos,
                              self.B + 1, self.tws)

    def feed(self, tok):
        """One more token of every request that can take one, tok [B] (of a row that has none: below 0);
        logits [B, V], which mean nothing in the other rows."""
        want = torch.addcmul(self.live, self.length, self.kept)         # a token more; the same; none
        self.resize(want)
        self.live = self.live * (self.length == want)
        slots = torch.where(self.live.bool(), self.slots.index_select(0, self.cu[:-1]), -1)
        length = self.length * self.live
        return self.model(tok.clamp(min=0), length - self.live, self.cache.attend(self.kvs, slots, length, self.max_len))

    def decode(self, tok, steps):
        """Feeds tok [B] and then each step's best token: tokens [B, steps]."""
        out = []
        for _ in range(steps):
            logits = self.feed(tok)
            self.select(logits)
            tok = torch.where(self.stopped, -1, self.select.tok[:, 0])
            out.append(tok)
            done = self.select.done[self.select.at].view(-1)
            self.kept, self.live = (torch.addcmul(x, self.live, done, value=-1) for x in (self.kept, self.live))
        return torch.stack(out, 1)

    def release(self):
        """Gives all blocks back; the batch can take other requests."""
        self.resize(torch.zeros_like(self.length))
        self.live, self.kept = torch.ones_like(self.live), torch.ones_like(self.kept)
        self.select.begin()

    def error(self):
        return lib.spec_get_device_error(self.tws) or self.cache.error()


class BeamBatch:
    """Beam search: W beams of each of the given prompts (host lists of token ids, not empty), up to
    max_new new tokens.

    A request that the pool has no blocks for is ``stopped`` [B]: its beams keep their scores, their
    tokens are -1 from there on, and ``error`` says what was missing.  The others go on."""

    def __init__(self, model, cache, prompts, W, max_new, vocab, eos=-1):
        self.model, self.cache, self.W, self.B = model, cache, W, len(prompts)
        B, bs, dev = self.B, cache.block_size, cache.device
        n = np.array([len(p) for p in prompts])
        # the last prompt token is fed with the beams: it is the first that they write
        whole = (n - 1) // bs
        groups = -(-(int((n - 1 - whole * bs).max()) + max_new + 1) // bs) + 1      # private blocks of a beam, at most
        self.whole = torch.from_numpy(whole.astype(np.int32)).to(dev)
        owned_ld = int(whole.max()) + W + groups * W
        self.owned = _ints(B, owned_ld, device=dev, fill=-1)
        self.held = _ints(B, device=dev)                    # tokens the owned blocks have room for
        self.stopped = torch.zeros(B, dtype=torch.bool, device=dev)
        self.want = ((self.whole + 2 * W) * bs).int()       # shared blocks, spares, the first private ones
        self.cap = int(whole.sum() + 2 * W * B) * bs
        self.slot_map, self.cu = _ints(self.cap, device=dev), _ints(B + 1, device=dev)
        self.tws = torch.zeros(lib.spec_block_tables_workspace_bytes(B), dtype=torch.uint8, device=dev)
        self._own()
        mb = int(whole.max()) + groups
        i = torch.arange(mb, device=dev)
        first = (self.whole + W)[:, None] + torch.arange(W, device=dev)
        tail = self.owned.gather(1, first.long())                                   # [B, W]
        shared = torch.where(i < self.whole[:, None], self._pad(self.owned, mb), -1)
        t = torch.where(i == self.whole[:, None, None], tail[:, :, None], shared[:, None, :].expand(B, W, mb))
        self.table = [t.reshape(B * W, mb).int().contiguous(), _ints(B * W, mb, device=dev, fill=-1)]
        spare = self.owned.gather(1, (self.whole[:, None] + torch.arange(W, device=dev)).long())
        self.spare = [spare.reshape(-1).int().contiguous(), _ints(B * W, device=dev)]
        hist = np.full((B, W, int(n.max()) + max_new + 1), -1, dtype=np.int32)
        for b, p in enumerate(prompts):
            hist[b, :, :len(p)] = p
        self.hist = [torch.from_numpy(hist.reshape(B * W, -1)).to(dev), _ints(B * W, hist.shape[-1], device=dev, fill=-1)]
        self.kvs = [cache.views(t) for t in self.table]
        self.slots = _ints(B * W, device=dev, fill=-1)
        self.length = _ints(B, device=dev)
        self.max_len = mb * bs
        self.select = _Select(B, W, vocab, eos, dev)
        self.select.score[0][:, 1:] = -float("inf")         # the beams part at the first selection
        self.at = 0
        self._prompts(prompts, n)

    @staticmethod
    def _pad(x, n):
        return x[:, :n] if x.shape[1] >= n else torch.nn.functional.pad(x, (0, n - x.shape[1]), value=-1)

    def _own(self):
        c = self.cache
        lib.spec_block_tables(self.B, c.block_size, self.owned.shape[1], c.num_blocks, self.held, self.want, self.owned,
                              self.owned, c.free, c.n_free, c.free, c.n_free, self.held, self.cu, self.slot_map, None,
                              self.cap, self.tws)
        self.stopped = self.stopped | (self.held != self.want)

    def _prompts(self, prompts, n):
        """All but the last prompt token, one a step, by beam 0 of each request."""
        W, dev, bs = self.W, self.cache.device, self.cache.block_size
        rows = self.table[0][::W].contiguous()
        kvs = self.cache.views(rows)
        for t in range(int(n.max()) - 1):
            tok = torch.tensor([p[t] if t + 1 < len(p) else 0 for p in prompts], dtype=torch.int32, device=dev)
            live = torch.tensor([t + 1 < len(p) for p in prompts], device=dev)
            slots = torch.where(live, rows[:, t // bs] * bs + t % bs, -1).int()
            self.length = torch.where(live, self.length + 1, self.length).int()
            pos = torch.full_like(tok, t)
            self.model(tok, pos, self.cache.attend(kvs, slots, torch.where(live, self.length, 0).int(), self.max_len))
        # every beam starts from beam 0's state
        self._reorder(torch.zeros(self.B, W, dtype=torch.int32, device=dev))
        self.tok = torch.tensor([p[-1] for p in prompts], dtype=torch.int32, device=dev).repeat_interleave(W)
        self.new = 0

    def _reorder(self, parent, tok=None):
        """Beams continue their parents, and have slots for their next tokens.  tok: what they
        append to their histories, which hold one token more than the cache (None: nothing)."""
        c, a, b = self.cache, self.at, 1 - self.at
        hist = (self.hist[a], self.hist[b]) if tok is not None else (None, None)
        st = lib.make_beam_state(self.B, self.W, c.block_size, self.table[a].shape[1], parent,
                                 tok if tok is not None else parent, self.length, self.whole, self.owned, self.table[a],
                                 self.table[b], self.spare[a], self.spare[b], self.slots, *hist)
        lib.spec_beam_reorder(st, self.kvs[a], c.row_bytes, self.tws)
        if tok is None:
            self.hist.reverse()
        self.at = b

    def step(self):
        """One token a beam."""
        W, bs = self.W, self.cache.block_size
        pos, length = self.length.repeat_interleave(W), self.length + 1
        kvs = self.kvs[self.at]
        seen = length.masked_fill(self.stopped, 0).repeat_interleave(W)
        logits = self.model(self.tok, pos, self.cache.attend(kvs, self.slots, seen, self.max_len))
        stopped = self.stopped[:, None]
        self.select.finish(stopped)
        self.select(logits)
        tok = torch.where(stopped, -1, self.select.tok)
        self.length = length
        # a request that comes to a block border needs W more blocks
        border = (length % bs == 0) > self.stopped
        need = (self.length // bs - self.whole + 1) * W + W + self.whole
        self.want = torch.where(border, torch.maximum(self.held, need * bs), self.held).int()
        self._own()
        self._reorder(self.select.parent, tok)
        self.tok = tok.reshape(-1).clamp(min=0)
        self.new += 1

    @property
    def score(self):
        return self.select.score[self.select.at]

    @property
    def done(self):
        return self.select.done[self.select.at]

    @property
    def tokens(self):
        """[B, W, length] tokens of the beams, best beam first, -1 past the end."""
        return self.hist[self.at].view(self.B, self.W, -1)

    def release(self):
        """Gives all blocks back."""
        self.want = torch.zeros_like(self.held)
        self._own()

    def error(self):
        return lib.spec_get_device_error(self.tws) or self.cache.error()


class RandomModel:
    """A small decoder with random weights: RMS norms, grouped-query attention over the paged
    cache, SwiGLU, learned positions.  Its products are torch's; it stands for the
    user's own model."""

    def __init__(self, layers=2, hidden=256, nq=8, nkv=2, hd=64, inter=512, vocab=4096, max_len=4096, dtype="bf16", seed=0,
                 device="cuda"):
        g = torch.Generator().manual_seed(seed)
        w = lambda *s: (torch.randn(*s, generator=g) * s[-1] ** -0.5).to(device).to(_TORCH[dtype])  # noqa: E731
        self.nq, self.nkv, self.hd, self.vocab = nq, nkv, hd, vocab
        self.embed, self.place, self.head = w(vocab, hidden) * 8, w(max_len, hidden) * 8, w(vocab, hidden) * 3
        self.layers = [dict(qkv=w((nq + 2 * nkv) * hd, hidden), o=w(hidden, nq * hd), up=w(2 * inter, hidden),
                            down=w(hidden, inter)) for _ in range(layers)]

    @staticmethod
    def norm(x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)

    def __call__(self, tok, pos, attend):
        x = self.embed[tok.long()] + self.place[pos.long()]
        n, nq, nkv, hd = x.shape[0], self.nq, self.nkv, self.hd
        for i, w in enumerate(self.layers):
            qkv = self.norm(x) @ w["qkv"].T
            q, k, v = qkv.split([nq * hd, nkv * hd, nkv * hd], 1)
            a = attend(i, q.view(n, nq, hd), k.view(n, nkv, hd), v.view(n, nkv, hd))
            x = x + a.reshape(n, nq * hd) @ w["o"].T
            up, gate = (self.norm(x) @ w["up"].T).chunk(2, 1)
            x = x + (up * torch.nn.functional.silu(gate)) @ w["down"].T
        return self.norm(x) @ self.head.T


def main():
    B, W, new = 8, 4, 32
    model = RandomModel()
    cache = PagedCache(2, 2048, 16, model.nq, model.nkv, model.hd, max_rows=B * W)
    r = np.random.default_rng(0)
    prompts = [r.integers(0, model.vocab, r.integers(3, 60)).tolist() for _ in range(B)]
    beams = BeamBatch(model, cache, prompts, W, new, model.vocab, eos=2)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    beams.step()                                        # loads the library's kernels
    a.record()
    for _ in range(new - 1):
        beams.step()
    b.record()
    torch.cuda.synchronize()
    if beams.error():
        raise RuntimeError("device error word %d" % beams.error())
    print("%d requests x %d beams, %d tokens: %.2f ms a step" % (B, W, new, a.elapsed_time(b) / (new - 1)))
    for i in range(2):
        print("request %d: score %.3f, tokens %s" % (i, float(beams.score[i, 0]), beams.tokens[i, 0, len(prompts[i]):].tolist()))
    beams.release()
    print("free blocks: %d of %d" % (int(cache.n_free[0]), cache.num_blocks))


if __name__ == "__main__":
    main()
