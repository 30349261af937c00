"""Decoding without speculation over the paged K/V cache: block tables, cache append, attention of one new token,
beam selection and beam reordering -- each in its plain form and as the library's call.

A case names its operator ("op") and its sizes.  Request lengths are a fixed multiset of the case (spread evenly from
"lo" to "hi"), dealt to the requests in an order that the seed makes, so that the work of a case is known without its
inputs; everything else of the inputs comes from the seed.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
K_SCALE, V_SCALE = 0.0625, 0.03125      # what a unit-variance row is stored with in 8 bits


# ------------------------------------------------------------------ cases
def listed():
    heads = dict(nq=32, nkv=8, hd=128, block=16)
    return [
        # one decode or verification step of a serving batch: every request grows by its 1 to 8 accepted tokens, and
        # few of them cross a block border
        dict(name="tables_step", op="tables", B=64, block=16, max_blocks=512, lo=512, hi=8000, grow=8, new=0, done=0),
        # a scheduler's large tick: half the requests run on, prompts of up to 8K tokens enter, finished ones leave
        dict(name="tables_prompts", op="tables", B=512, block=16, max_blocks=544, lo=256, hi=8192, grow=8, new=192,
             done=64),
        # the K/V rows of one verified batch of 32 requests, 8 tokens each, as slices of the fused QKV product
        dict(name="append_step", op="append", n=256, nkv=8, hd=128, qkv=6144, type="bf16", cache="bf16", block=16),
        # a prompt chunk of 32K tokens into an 8-bit cache
        dict(name="append_prompt", op="append", n=32768, nkv=8, hd=128, qkv=6144, type="bf16", cache="e4m3", block=16),
        # the smallest call: four requests of the chain workload's context, one token each; latency counts
        dict(name="attn_small", op="attn", B=4, lo=200, hi=256, empty=0, type="bf16", cache="bf16", window=0, **heads),
        # one request over a 128K context: one row of work, split over the length and joined
        dict(name="attn_long", op="attn", B=1, lo=131071, hi=131071, empty=0, type="f16", cache="f16", window=0, **heads),
        # a full serving batch at mixed lengths
        dict(name="attn_batch", op="attn", B=64, lo=1024, hi=8190, empty=0, type="bf16", cache="bf16", window=0, **heads),
        # 8-bit cache, sliding window, some rows with nothing to attend to (slots of a padded batch)
        dict(name="attn_e4m3_window", op="attn", B=96, lo=1, hi=4001, empty=8, type="bf16", cache="e4m3", window=1024,
             **heads),
        # one request with four beams over a full vocabulary
        dict(name="select_one", op="select", B=1, W=4, V=128256, type="bf16"),
        # a batch of beam requests, 32-bit logits
        dict(name="select_batch", op="select", B=32, W=8, V=151936, type="f32"),
        # the draft layer's cache under four beams
        dict(name="reorder_one", op="reorder", B=1, W=4, lo=700, hi=700, layers=1, nkv=8, hd=128, type="bf16", block=16,
             max_blocks=128),
        # a 32-layer cache under sixteen requests of eight beams
        dict(name="reorder_batch", op="reorder", B=16, W=8, lo=900, hi=3999, layers=32, nkv=8, hd=128, type="bf16",
             block=16, max_blocks=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "attn", "attn", "attn", "select", "reorder"])
    if op == "tables":
        B = _log(rng, 1, 512)
        block = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
        hi = _log(rng, 16, 6000)
        new, done = rng.randint(0, B // 3), rng.randint(0, B // 4)
        grow = rng.randint(1, 9)
        return dict(op=op, B=B, block=block, max_blocks=(hi + grow) // block + rng.randint(2, 9), lo=rng.randint(1, hi),
                    hi=hi, grow=grow, new=new, done=done)
    if op == "append":
        typ = rng.choice(["bf16", "bf16", "f16", "f32"])
        cache = typ if typ == "f32" or rng.random() < 0.6 else "e4m3"
        nkv, hd = rng.choice([1, 2, 3, 5, 8, 16]), rng.choice([64, 80, 128, 128, 256])
        n = min(_log(rng, 1, 30000), 30000 * 1024 // (nkv * hd * BYTES[typ] // 2))
        qkv = nkv * hd * rng.choice([2, 5, 10])
        return dict(op=op, n=n, nkv=nkv, hd=hd, qkv=qkv, type=typ, cache=cache, block=rng.choice([1, 16, 24, 64]))
    if op == "attn":
        typ = rng.choice(["bf16", "bf16", "f16", "f32"])
        cache = typ if typ == "f32" or rng.random() < 0.7 else "e4m3"
        nkv, group = rng.choice([1, 2, 3, 4, 8, 8, 16]), rng.choice([1, 2, 4, 4, 5, 8, 16])
        hd = rng.choice([64, 80, 96, 128, 128, 128, 256])
        B = _log(rng, 1, 200)
        row = 2 * nkv * hd * BYTES[cache]
        # keys of a request, from one to what fills the budget
        most = max(1, min(120000, int(700e6 / 4 * BYTES[cache]) // (B * row)))
        hi = _log(rng, 1, most)
        return dict(op=op, B=B, lo=rng.randint(1, hi), hi=hi, empty=rng.randint(0, B // 4), type=typ, cache=cache,
                    window=rng.choice([0, 0, 0, 64, 300, 1024]), nq=nkv * group, nkv=nkv, hd=hd,
                    block=rng.choice([1, 8, 16, 16, 24, 32, 64, 128]))
    if op == "select":
        W = rng.choice([1, 2, 3, 4, 5, 8, 10, 16])
        typ = rng.choice(["f32", "bf16", "f16"])
        V = _log(rng, 500, 152000)
        return dict(op=op, B=min(_log(rng, 1, 64), max(1, 36000000 // (W * V))), W=W, V=V, type=typ)
    W, B, layers = rng.choice([1, 2, 3, 4, 5, 8, 10, 16]), _log(rng, 1, 24), rng.choice([1, 1, 2, 12, 24, 36])
    typ, nkv, hd = rng.choice(["bf16", "f16", "f32", "e4m3"]), rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 128])
    block = rng.choice([1, 8, 16, 16, 24, 32])
    hi = _log(rng, 20, 2600)
    B = max(1, min(B, int(2.4e9 // (layers * 2 * nkv * hd * BYTES[typ] * (hi + 7 * W * block + block)))))
    return dict(op=op, B=B, W=W, lo=rng.randint(17, hi), hi=hi, layers=layers, nkv=nkv, hd=hd, type=typ, block=block,
                max_blocks=hi // block + rng.randint(1, 40))


def _lengths(c):
    B, lo, hi = c["B"], c["lo"], c["hi"]
    v = [hi - (hi - lo) * i // max(1, B - 1) for i in range(B)]
    for i in range(c.get("empty", 0)):
        v[B - 1 - i] = 0
    return v


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _cuda(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a), dtype=dtype).to(DEV)


def prepare(case, seed):
    return {"tables": _prepare_tables, "append": _prepare_append, "attn": _prepare_attn, "select": _prepare_select,
            "reorder": _prepare_reorder}[case["op"]](case, seed)


def _prepare_tables(c, seed):
    r = np.random.RandomState(seed)
    B, bs = c["B"], c["block"]
    old = np.array(_lengths(c))
    new = old + 1 + np.arange(B) % c["grow"]
    new[:c["new"]] = old[:c["new"]]                                # prompts that enter
    old[:c["new"]] = 0
    if c["done"]:
        new[B - c["done"]:] = 0                                    # finished requests
    order = r.permutation(B)
    old, new = old[order], new[order]
    have = -(-old // bs)
    spare = int((-(-new // bs)).sum()) + 8
    ids = r.permutation(int(have.sum()) + spare)
    table = np.full((B, c["max_blocks"]), -1)
    at = 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    free = np.full(len(ids), -1)
    free[:len(ids) - at] = ids[at:]
    total = int(np.maximum(new - old, 0).sum())
    return dict(c=c, old=_cuda(old), new=_cuda(new), table=_cuda(table), free=_cuda(free), n_free=_cuda([len(ids) - at]),
                cap=total + 5)


def _prepare_append(c, seed):
    g, r = _gen(seed), np.random.RandomState(seed)
    n, nkv, hd, t = c["n"], c["nkv"], c["hd"], TYPES[c["type"]]
    slots = -(-(n + 40) // c["block"]) * c["block"]
    qkv = torch.randn(n, c["qkv"], generator=g, device=DEV, dtype=torch.float32).to(t)
    w = nkv * hd
    cache = torch.zeros(2, slots, nkv, hd, device=DEV, dtype=torch.float32).to(TYPES[c["cache"]])
    at = r.permutation(slots // c["block"])[:, None] * c["block"] + np.arange(c["block"])
    at = at.reshape(-1)[:n].copy()
    at[r.rand(n) < 0.02] = -1                                      # padded rows
    return dict(c=c, k=qkv[:, -2 * w:-w], v=qkv[:, -w:], cache_k=cache[0], cache_v=cache[1], slots=_cuda(at))


def _prepare_attn(c, seed):
    g, r = _gen(seed), np.random.RandomState(seed)
    B, nq, nkv, hd, bs = c["B"], c["nq"], c["nkv"], c["hd"], c["block"]
    length = np.array(_lengths(c))[r.permutation(B)]
    blocks = -(-length // bs)
    total = int(blocks.sum()) + 3
    ids = r.permutation(total)
    table = np.full((B, max(1, int(blocks.max()) + 1)), -1)
    ends = np.cumsum(blocks)
    for b in range(B):
        table[b, :blocks[b]] = ids[ends[b] - blocks[b]:ends[b]]
    q = torch.randn(B, nq, hd, generator=g, device=DEV).to(TYPES[c["type"]])
    stored = TYPES[c["cache"]]
    scales = (K_SCALE, V_SCALE) if c["cache"] == "e4m3" else (1.0, 1.0)
    kv = []
    for scale in scales:
        x = torch.empty(total * bs, nkv, hd, device=DEV, dtype=stored)
        for part in x.split(1 << 16):
            part.copy_(torch.randn(part.shape, generator=g, device=DEV) / scale)
        kv.append(x)
    return dict(c=c, q=q, k=kv[0], v=kv[1], table=_cuda(table), length=_cuda(length), scales=scales,
                longest=int(length.max()))


def _prepare_select(c, seed):
    g, r = _gen(seed), np.random.RandomState(seed)
    B, W, V = c["B"], c["W"], c["V"]
    logits = torch.empty(B, W, V, device=DEV, dtype=TYPES[c["type"]])
    for b in range(B):
        logits[b] = torch.randn(W, V, generator=g, device=DEV) * 2.5
    score = -3.0 * r.rand(B, W).cumsum(1) - 5.0
    done = np.zeros((B, W))
    for b in range(B):
        what = r.rand()
        if what < 0.15:
            score[b, 1:] = -np.inf                                 # the first step: only beam 0 lives
        elif what < 0.5:
            done[b, r.randint(W)] = 1                              # a finished beam
        if r.rand() < 0.2:                                         # constrained decoding: some ids are masked
            logits[b, :, torch.rand(V, generator=g, device=DEV) < 0.4] = -math.inf
    if B > 2:
        logits[1, W - 1] = -math.inf                               # a row that its mask leaves empty
    return dict(c=c, logits=logits, score=_cuda(score, torch.float32), done=_cuda(done), eos=2)


def _prepare_reorder(c, seed):
    g, r = _gen(seed), np.random.RandomState(seed)
    B, W, bs, mb = c["B"], c["W"], c["block"], c["max_blocks"]
    length = np.array(_lengths(c))[r.permutation(B)]
    prompt = length - 1 - r.randint(0, np.minimum(length - 1, 3 * bs) + 1)     # tokens before the beams part
    whole = prompt // bs
    at = length // bs
    gens = at - whole + 1
    owned_n = whole + W + gens * W
    total = int((at + 7 * W).sum())                                # the largest that owned_n can sum up to
    ids = r.permutation(total)
    owned = np.full((B, int(at.max()) + 7 * W), -1)
    table = np.full((B, W, mb), -1)
    spare = np.zeros((B, W))
    ends = np.cumsum(owned_n)
    for b in range(B):
        own_b = ids[ends[b] - owned_n[b]:ends[b]]
        owned[b, :owned_n[b]] = own_b
        p = whole[b]
        table[b, :, :p] = own_b[:p]
        spare[b] = own_b[p:p + W]
        for i in range(p, at[b]):                                  # generated blocks that are full: any beam's
            table[b, :, i] = own_b[p + W + (i - p) * W + r.randint(0, W, W)]
        if length[b] % bs:
            table[b, :, at[b]] = own_b[p + W + (at[b] - p) * W + np.arange(W)]
    hist = r.randint(0, 100000, (B * W, int(length.max()) + 1))
    stored = TYPES[c["type"]]
    kv = torch.empty(2, c["layers"], total * bs, c["nkv"], c["hd"], device=DEV, dtype=stored)
    for x in kv.view(-1, total * bs, c["nkv"], c["hd"]):
        x.copy_(torch.randn(x.shape, generator=g, device=DEV))
    parent = np.sort(r.randint(0, W, (B, W)), axis=1)
    return dict(c=c, parent=_cuda(parent), tok=_cuda(r.randint(0, 100000, (B, W))), length=_cuda(length), whole=_cuda(whole),
                owned=_cuda(owned), table=_cuda(table.reshape(B * W, mb)), spare=_cuda(spare.reshape(-1)), hist=_cuda(hist),
                k=kv[0], v=kv[1])


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["c"]["op"]
    if own:
        return {"tables": _own_tables, "append": _own_append, "attn": _own_attn, "select": _own_select,
                "reorder": _own_reorder}[op](state)
    return {"tables": _plain_tables, "append": _plain_append, "attn": _plain_attn, "select": _plain_select,
            "reorder": _plain_reorder}[op](state)


def _plain_tables(s):
    c = s["c"]
    bs, (B, mb), F = c["block"], s["table"].shape, s["free"].numel()
    old, new, n = s["old"].long(), s["new"].long(), s["n_free"].long()[0]
    have, want = (old + bs - 1) // bs, (new + bs - 1) // bs
    rel, need = (have - want).clamp(min=0), (want - have).clamp(min=0)
    rel_end, need_end = rel.cumsum(0), need.cumsum(0)
    avail = n + rel_end[-1]
    served = (need == 0) | (need_end <= avail)
    taken = torch.where(served, need, 0).sum()
    # the pool with the released blocks on top: P = free[0:n] ++ released
    j = torch.arange(F, device=DEV)
    from_rel = (j - n).clamp(min=0)
    row = torch.searchsorted(rel_end, from_rel, right=True).clamp(max=B - 1)
    col = (want[row] + from_rel - (rel_end[row] - rel[row])).clamp(0, mb - 1)
    P = torch.where(j < n, s["free"].long(), s["table"][row, col].long())
    free = torch.where(j < avail - taken, P, -1)
    # tables: kept entries, then the blocks taken, then -1
    i = torch.arange(mb, device=DEV)
    want = torch.where(served, want, have)
    nth = (need_end - need)[:, None] + i - have[:, None]
    got = P[(avail - 1 - nth).clamp(0, F - 1)]
    table = torch.where(i < torch.minimum(have, want)[:, None], s["table"].long(), torch.where(i < want[:, None], got, -1))
    # slots and positions of the new tokens
    count = (new - old).clamp(min=0)
    end = count.cumsum(0)
    t = torch.arange(s["cap"], device=DEV)
    b = torch.searchsorted(end, t, right=True).clamp(max=B - 1)
    pos = old[b] + t - (end[b] - count[b])
    slot = table[b, (pos // bs).clamp(max=mb - 1)] * bs + pos % bs
    slot = torch.where((t < end[-1]) & served[b], slot, -1)
    pos = torch.where(t < end[-1], pos, 0)
    cu = torch.cat([end.new_zeros(1), end])
    out = dict(table=table, free=free, n_free=(avail - taken).view(1), length=torch.where(served, new, old), cu=cu,
               slots=slot, pos=pos)
    return {k: v.int() for k, v in out.items()}


def _stored(x, cache, scale):
    if cache.dtype == TYPES["e4m3"]:
        return (x.float() / scale).clamp(-448, 448).to(cache.dtype)
    return x.to(cache.dtype)


def _plain_append(s):
    nkv, hd = s["c"]["nkv"], s["c"]["hd"]
    at = s["slots"].long()
    keep = (at >= 0).nonzero()[:, 0]
    for x, cache, scale in ((s["k"], s["cache_k"], K_SCALE), (s["v"], s["cache_v"], V_SCALE)):
        new = _stored(x[keep].view(-1, nkv, hd), cache, scale)
        same = torch.uint8 if cache.dtype == TYPES["e4m3"] else cache.dtype
        cache.view(same)[at[keep]] = new.view(same)
    return {"k": s["cache_k"], "v": s["cache_v"]}


def _plain_attn(s):
    c = s["c"]
    B, nq, nkv, hd, bs = c["B"], c["nq"], c["nkv"], c["hd"], c["block"]
    t = torch.arange(s["longest"], device=DEV)
    length = s["length"].long()
    seen = t < length[:, None]
    if c["window"]:
        seen &= t >= length[:, None] - c["window"]
    slot = (s["table"].long()[:, t // bs] * bs + t % bs).clamp(min=0)
    k = (s["k"].view(torch.uint8)[slot].view(s["k"].dtype) if c["cache"] == "e4m3" else s["k"][slot]).float()
    v = (s["v"].view(torch.uint8)[slot].view(s["v"].dtype) if c["cache"] == "e4m3" else s["v"][slot]).float()
    k, v = k * s["scales"][0], v * s["scales"][1]
    v = torch.where(seen[:, :, None, None], v, 0)
    q = s["q"].float().view(B, nkv, nq // nkv, hd) / math.sqrt(hd)
    x = q @ k.permute(0, 2, 3, 1)
    x = torch.where(seen[:, None, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    base = torch.where(m.isfinite(), m, 0)
    e = torch.exp(x - base)
    total = e.sum(-1, keepdim=True)
    out = (e @ v.transpose(1, 2)) / torch.where(total > 0, total, 1)
    lse = torch.where(total > 0, base + torch.log(total), -math.inf)
    return {"out": out.view(B, nq, hd).to(s["q"].dtype), "lse": lse.view(B, nq)}


def _plain_select(s):
    B, W, V = s["logits"].shape
    # 64 bits: scores of different beams are compared with one another
    x = s["logits"].double()
    x = torch.where(x.isfinite(), x, -math.inf)
    m = x.amax(-1, keepdim=True)
    base = torch.where(m.isfinite(), m, 0)
    lse = base + torch.log(torch.exp(x - base).sum(-1, keepdim=True))
    score, done = s["score"].double()[:, :, None], s["done"][:, :, None] != 0
    at_eos = torch.arange(V, device=DEV) == s["eos"]
    cand = torch.where(done, torch.where(at_eos, score, -math.inf), score + (x - lse))
    cand = torch.where(score.isfinite() & (done | x.isfinite()), cand, -math.inf).view(B, W * V)
    # everything at or over the W-th largest, by descending score and then by place
    border = cand.topk(W, dim=-1).values[:, -1:]
    b, at = ((cand >= border) & (cand > -math.inf)).nonzero(as_tuple=True)
    val = cand[b, at]
    order = torch.argsort(val, descending=True, stable=True)
    order = order[torch.argsort(b[order], stable=True)]
    b, at, val = b[order], at[order], val[order]
    count = torch.bincount(b, minlength=B)
    rank = torch.arange(len(b), device=DEV) - (count.cumsum(0) - count)[b]
    b, at, val, rank = b[rank < W], at[rank < W], val[rank < W], rank[rank < W]
    parent = torch.arange(W, device=DEV, dtype=torch.int32).repeat(B, 1)
    tok = torch.full((B, W), -1, device=DEV, dtype=torch.int32)
    out = torch.full((B, W), -math.inf, device=DEV, dtype=torch.float32)
    parent[b, rank], tok[b, rank], out[b, rank] = (at // V).int(), (at % V).int(), val.float()
    was_done = s["done"].gather(1, parent.long()) != 0
    fin = (tok < 0) | was_done | (tok == s["eos"])
    return {"parent": parent, "tok": tok, "score": out, "done": fin.int()}


def _plain_reorder(s):
    c = s["c"]
    B, W, bs, mb = c["B"], c["W"], c["block"], c["max_blocks"]
    beam = torch.arange(W, device=DEV).repeat(B)
    req = torch.arange(B, device=DEV).repeat_interleave(W)
    src = req * W + s["parent"].long().view(-1)
    me = req * W + beam
    length, whole = s["length"].long()[req], s["whole"].long()[req]
    at, rest = length // bs, length % bs
    table, spare = s["table"].long(), s["spare"].long()
    cur = table[me, at.clamp(max=mb - 1)]
    moved = (rest > 0) & (src != me)
    fresh = s["owned"].long()[req, (whole + W + (at - whole) * W + beam).clamp(max=s["owned"].shape[1] - 1)]
    tail = torch.where(rest == 0, fresh, torch.where(moved, spare, cur))
    i = torch.arange(mb, device=DEV)
    out = torch.where(i < at[:, None], table[src], torch.where(i == at[:, None], tail[:, None], -1))
    h = torch.arange(s["hist"].shape[1], device=DEV)
    hist = torch.where(h < length[:, None], s["hist"][src], torch.where(h == length[:, None], s["tok"].view(-1, 1), -1))
    # the partial block's rows, into the child's spare block, in every layer
    r = torch.arange(bs, device=DEV)
    pick = (moved[:, None] & (r < rest[:, None])).nonzero(as_tuple=True)
    frm = table[src[pick[0]], at[pick[0]]] * bs + pick[1]
    to = spare[pick[0]] * bs + pick[1]
    for x in (s["k"], s["v"]):
        x = x.view(torch.uint8) if c["type"] == "e4m3" else x
        x[:, to] = x[:, frm]
    return {"table": out.int(), "spare": torch.where(moved, cur, spare).int(), "hist": hist.int(),
            "slots": (tail * bs + rest).int(), "k": s["k"], "v": s["v"]}


# ------------------------------------------------------------------ the library's calls
def _lib():
    from eagle_speculative_decoding_step_gb300 import binding
    return binding


def _kept(s, make):
    """What a program keeps between calls on the same buffers: descriptors, workspace, output buffers."""
    if "kept" not in s:
        s["kept"] = make(_lib())
    return s["kept"]


def _ints(*shape):
    return torch.empty(*shape, device=DEV, dtype=torch.int32)


def _zeros(nbytes):
    return torch.zeros(nbytes, device=DEV, dtype=torch.uint8)


def _own_tables(s):
    lib, c = _lib(), s["c"]
    B, mb = s["table"].shape
    k = _kept(s, lambda lib: dict(
        ws=_zeros(lib.spec_block_tables_workspace_bytes(B)),
        out=dict(table=_ints(B, mb), free=_ints(s["free"].numel()), n_free=_ints(1), length=_ints(B), cu=_ints(B + 1),
                 slots=_ints(s["cap"]), pos=_ints(s["cap"]))))
    o = k["out"]
    lib.spec_block_tables(B, c["block"], mb, s["free"].numel(), s["old"], s["new"], s["table"], o["table"], s["free"],
                          s["n_free"], o["free"], o["n_free"], o["length"], o["cu"], o["slots"], o["pos"], s["cap"], k["ws"])
    return dict(o)


def _attn_desc(lib, c, nq):
    return lib.make_attn_desc(nq, c["nkv"], c["hd"], c["type"], c["cache"], window=c.get("window", 0),
                              k_scale=K_SCALE, v_scale=V_SCALE)


def _own_append(s):
    lib, c = _lib(), s["c"]
    k = _kept(s, lambda lib: dict(
        ws=_zeros(256), desc=_attn_desc(lib, c, c["nkv"]),
        kv=lib.make_kv(dict(k=s["cache_k"], v=s["cache_v"], block_table=None, block_size=c["block"], max_blocks=0,
                            num_slots=s["cache_k"].shape[0]))))
    lib.spec_cache_append(k["desc"], s["k"], s["v"], c["qkv"], s["slots"], c["n"], k["kv"], k["ws"])
    return {"k": s["cache_k"], "v": s["cache_v"]}


def _own_attn(s):
    lib, c = _lib(), s["c"]

    def make(lib):
        desc = _attn_desc(lib, c, c["nq"])
        return dict(desc=desc, ws=_zeros(lib.spec_attention_workspace_bytes(desc, c["B"])),
                    kv=lib.make_kv(dict(k=s["k"], v=s["v"], block_table=s["table"], block_size=c["block"],
                                        max_blocks=s["table"].shape[1], num_slots=s["k"].shape[0])),
                    out=torch.empty_like(s["q"]), lse=torch.empty(c["B"], c["nq"], device=DEV))
    k = _kept(s, make)
    lib.spec_paged_attention(k["desc"], s["q"], k["kv"], s["length"], c["B"], k["out"], k["lse"], k["ws"],
                             max_len=s["longest"])
    return {"out": k["out"], "lse": k["lse"]}


def _own_select(s):
    lib, c = _lib(), s["c"]
    B, W, V = s["logits"].shape
    k = _kept(s, lambda lib: dict(
        ws=_zeros(lib.spec_beam_workspace_bytes(B, W, V)),
        out=dict(parent=_ints(B, W), tok=_ints(B, W), score=torch.empty(B, W, device=DEV), done=_ints(B, W))))
    o = k["out"]
    lib.spec_beam_select(B, W, V, c["type"], s["logits"], s["score"], s["done"], s["eos"], o["parent"], o["tok"],
                         o["score"], o["done"], k["ws"])
    return dict(o)


def _own_reorder(s):
    lib, c = _lib(), s["c"]
    B, W = c["B"], c["W"]

    def make(lib):
        o = dict(table=torch.empty_like(s["table"]), spare=torch.empty_like(s["spare"]), hist=torch.empty_like(s["hist"]),
                 slots=_ints(B * W))
        st = lib.make_beam_state(B, W, c["block"], c["max_blocks"], parent=s["parent"], tok=s["tok"], seq_len=s["length"],
                                 prompt_blocks=s["whole"], owned=s["owned"], table_in=s["table"], table_out=o["table"],
                                 spare_in=s["spare"], spare_out=o["spare"], slots=o["slots"], hist_in=s["hist"],
                                 hist_out=o["hist"])
        kvs = lib.make_kv_layers([dict(k=s["k"][i], v=s["v"][i], block_table=None, block_size=c["block"], max_blocks=0,
                                       num_slots=s["k"].shape[1]) for i in range(c["layers"])])
        return dict(ws=_zeros(256), out=o, st=st, kvs=kvs)
    k = _kept(s, make)
    lib.spec_beam_reorder(k["st"], k["kvs"], c["nkv"] * c["hd"] * BYTES[c["type"]], k["ws"])
    return {**k["out"], "k": s["k"], "v": s["v"]}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "tables":
        B, bs = c["B"], c["block"]
        length = _lengths(c)
        grown = sum(length[:c["new"]]) + sum(1 + i % c["grow"] for i in range(c["new"], B - c["done"]))
        kept = sum(-(-n // bs) for n in length[c["new"]:B - c["done"]])
        moved = sum(-(-n // bs) for n in length[:c["new"]]) + sum(-(-n // bs) for n in length[B - c["done"]:])
        return {"bytes": 4 * (4 * B + 2 * kept + 2 * moved + 2 * grown), "flops": 0}
    if c["op"] == "append":
        w = c["nkv"] * c["hd"]
        return {"bytes": c["n"] * (4 + 2 * w * (BYTES[c["type"]] + BYTES[c["cache"]])), "flops": 0}
    if c["op"] == "attn":
        keys = sum(min(n, c["window"]) if c["window"] else n for n in _lengths(c))
        q = c["B"] * c["nq"] * c["hd"]
        return {"bytes": keys * c["nkv"] * c["hd"] * 2 * BYTES[c["cache"]] + 2 * q * BYTES[c["type"]] + 4 * c["B"] * c["nq"],
                "flops": 4 * keys * c["nq"] * c["hd"]}
    if c["op"] == "select":
        n = c["B"] * c["W"]
        return {"bytes": n * c["V"] * BYTES[c["type"]] + 24 * n, "flops": 3 * n * c["V"]}
    # three of four children have another parent; a partial block holds half its rows
    bs, rows = c["block"], c["B"] * c["W"]
    length = _lengths(c)
    moved = 0.75 * rows * (bs - 1) / 2 if c["W"] > 1 else 0
    row = c["nkv"] * c["hd"] * BYTES[c["type"]]
    ints = sum(n // bs + 1 + n + 1 for n in length) * c["W"]
    return {"bytes": 8 * ints + 4 * moved * row * c["layers"], "flops": 0}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "append":
        out = {}
        for name, scale in (("k", K_SCALE), ("v", V_SCALE)):
            rows = s[name].double().cpu().numpy().reshape(c["n"], c["nkv"], c["hd"])
            cache = np.zeros((s["cache_k"].shape[0], c["nkv"], c["hd"]))
            at = s["slots"].cpu().numpy()
            cache[at[at >= 0]] = rows[at >= 0] / (scale if c["cache"] == "e4m3" else 1.0)
            out[name] = torch.from_numpy(cache)
        return out
    if c["op"] == "attn":
        B, nq, nkv, hd, bs = c["B"], c["nq"], c["nkv"], c["hd"], c["block"]
        out = torch.zeros(B, nq, hd, dtype=torch.float64, device=DEV)
        lse = torch.full((B, nq), -math.inf, dtype=torch.float64, device=DEV)
        for b, n in enumerate(s["length"].tolist()):
            lo = max(0, n - c["window"]) if c["window"] else 0
            if n <= lo:
                continue
            t = torch.arange(lo, n, device=DEV)
            at = s["table"][b].long()[t // bs] * bs + t % bs
            for h in range(nkv):
                k = s["k"][:, h].view(torch.uint8)[at].view(s["k"].dtype) if c["cache"] == "e4m3" else s["k"][at, h]
                v = s["v"][:, h].view(torch.uint8)[at].view(s["v"].dtype) if c["cache"] == "e4m3" else s["v"][at, h]
                k, v = k.double() * s["scales"][0], v.double() * s["scales"][1]
                mine = slice(h * (nq // nkv), (h + 1) * (nq // nkv))
                x = (s["q"][b, mine].double() @ k.T) * hd ** -0.5
                lse[b, mine] = torch.logsumexp(x, -1)
                out[b, mine] = torch.softmax(x, -1) @ v
        return {"out": out, "lse": lse}
    if c["op"] == "select":
        B, W, V = s["logits"].shape
        best = np.full((B, W), -np.inf)
        for b in range(B):
            found = []
            for j in range(W):
                if not np.isfinite(float(s["score"][b, j])):
                    continue
                if int(s["done"][b, j]):
                    found.append(np.array([float(s["score"][b, j])]))
                    continue
                x = s["logits"][b, j].double()
                x = x[torch.isfinite(x)]
                if x.numel():
                    top = torch.sort(x, descending=True).values[:W] - torch.logsumexp(x, 0)
                    found.append(top.cpu().numpy() + float(s["score"][b, j]))
            if found:
                v = np.sort(np.concatenate(found))[::-1][:W]
                best[b, :len(v)] = v
        return {"parent": None, "tok": None, "score": torch.from_numpy(best), "done": None}
    return None                                                    # indices, and rows that are moved as they are
