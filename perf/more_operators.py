"""Prompts and samples over the paged K/V cache: attention of a chunk of new tokens, log-probabilities of given tokens,
and the blocks of requests that are forked, released and compacted -- each in its plain form and as the library's call.

A case names its operator ("op") and its sizes.  Lengths are a fixed multiset of the case, dealt to the requests in an
order that the seed makes, so that the work of a case is known without its inputs; everything else of the inputs comes
from the seed.
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
    layer = dict(nkv=8, hd=128, type="bf16", block=16)
    return [
        # the target's pass over a verified chain: four requests, 8 new tokens each; latency counts
        dict(name="chunk_small", op="chunk", B=4, rlo=8, rhi=8, lo=200, hi=256, none=0, dead=0, type="bf16", cache="bf16",
             window=0, **heads),
        # a scheduler's tick of prompts: chunks of 100 to 2048 tokens behind contexts of nothing to 6000
        dict(name="chunk_batch", op="chunk", B=16, rlo=100, rhi=2048, lo=0, hi=6000, none=1, dead=0, type="bf16",
             cache="bf16", window=0, **heads),
        # one chunk of a long document: few rows, a 128K context
        dict(name="chunk_long", op="chunk", B=1, rlo=500, rhi=500, lo=130571, hi=130571, none=0, dead=0, type="f16",
             cache="f16", window=0, **heads),
        # prompts and single new tokens in one batch, 8-bit cache, sliding window, requests that were stopped
        dict(name="chunk_e4m3_window", op="chunk", B=24, rlo=1, rhi=701, lo=1, hi=4001, none=1, dead=2, type="bf16",
             cache="e4m3", window=1024, **heads),
        # what a serving step answers with beside its tokens
        dict(name="logprobs_step", op="logprobs", n=64, V=128256, k=5, type="bf16"),
        # the scores of a prompt's tokens, 32-bit logits
        dict(name="logprobs_prompt", op="logprobs", n=2048, V=151936, k=20, type="f32"),
        # four samples of one prompt, the draft layer's cache
        dict(name="fork_one", op="fork", live=1, fan=3, lo=700, hi=700, short=0, layers=1, **layer),
        # a batch of prompts, five samples each, a 32-layer cache
        dict(name="fork_batch", op="fork", live=32, fan=4, lo=300, hi=1600, short=0, layers=32, **layer),
        # one tick: some samples have ended
        dict(name="release_step", op="release", live=8, fan=4, lo=300, hi=2000, grow=200, block=16),
        # a large batch's
        dict(name="release_batch", op="release", live=128, fan=4, lo=256, hi=7000, grow=500, block=16),
        # the draft layer's cache after a while of serving
        dict(name="compact_draft", op="compact", live=4, fan=2, lo=200, hi=900, grow=100, full=0.7, layers=1, **layer),
        # a 32-layer cache
        dict(name="compact_batch", op="compact", live=24, fan=2, lo=200, hi=1500, grow=200, full=0.6, layers=32, **layer),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "logprobs", "logprobs", "fork", "release", "compact"])
    if op == "chunk":
        typ = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
        cache = typ if typ == "f32" or rng.random() < 0.75 else "e4m3"
        nkv, group = rng.choice([1, 2, 3, 4, 8, 8, 16]), rng.choice([1, 2, 4, 4, 5, 8, 16])
        hd = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
        B = _log(rng, 1, 64)
        rhi, hi = _log(rng, 1, 4000), _log(rng, 1, 60000)
        c = dict(op=op, B=B, rlo=rng.randint(1, rhi), rhi=rhi, lo=rng.randint(0, hi), hi=hi, none=rng.randint(0, B // 4),
                 dead=rng.randint(0, B // 6), type=typ, cache=cache, window=rng.choice([0, 0, 0, 64, 300, 1024]), nq=nkv * group,
                 nkv=nkv, hd=hd, block=rng.choice([1, 8, 16, 16, 16, 24, 32, 64, 128]))
        most = 1e11 if typ == "f32" else 6e11
        while work(c)["flops"] > most or (c["hi"] + c["rhi"]) * B * nkv * hd > 4e8:
            at = "hi" if c["hi"] > 4 * c["rhi"] else "rhi"
            c[at] = c[at] * 2 // 3
            low = "lo" if at == "hi" else "rlo"
            c[low] = min(c[low], c[at])
        return c
    if op == "logprobs":
        V = _log(rng, 500, 152000)
        return dict(op=op, n=min(_log(rng, 1, 2048), 300000000 // V), V=V, k=rng.choice([0, 1, 5, 5, 20, 32]),
                    type=rng.choice(["f32", "bf16", "bf16", "f16"]))
    block = rng.choice([1, 8, 16, 16, 24, 32, 64])
    hi = _log(rng, 16, 2000)
    layer = dict(layers=rng.choice([1, 1, 2, 12, 24, 36]), nkv=rng.choice([1, 2, 4, 8]), hd=rng.choice([64, 80, 128]),
                 type=rng.choice(["bf16", "f16", "f32", "e4m3"]), block=block)
    row = 2 * layer["layers"] * layer["nkv"] * layer["hd"] * BYTES[layer["type"]]
    if op == "fork":
        fan = rng.randint(1, 8)
        live = max(1, min(_log(rng, 1, 64), int(3.5e9 // (row * (hi + (fan + 1) * block)))))
        return dict(op=op, live=live, fan=fan, lo=rng.randint(1, hi), hi=hi, short=rng.choice([0, 0, 1, live * fan // 3]), **layer)
    if op == "release":
        hi, fan = _log(rng, 16, 7000), rng.randint(1, 8)
        return dict(op=op, live=_log(rng, 1, 500 // fan), fan=fan, lo=rng.randint(1, hi), hi=hi, grow=rng.randint(1, 500),
                    block=block)
    fan, grow = rng.randint(1, 4), rng.randint(1, 200)
    live = max(1, min(_log(rng, 1, 60), int(2e9 // (row * (hi + fan * (grow + 2 * block))))))
    return dict(op=op, live=live, fan=fan, lo=rng.randint(1, hi), hi=hi, grow=grow, full=rng.choice([0.5, 0.6, 0.8, 0.95]), **layer)


def _spread(lo, hi, n):
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _chunks(c):
    """(new tokens, tokens in all) of the requests: "none" of them have no new tokens, "dead" ones have rows and no
    cache (stopped requests, which stay in a batch)."""
    B = c["B"]
    ctx = _spread(c["lo"], c["hi"], B)
    rows = _spread(c["rlo"], c["rhi"], B)
    out = []
    for i in range(B):
        n = 0 if i >= B - c["none"] else rows[(7 * i + 3) % B]
        out.append([n, ctx[i] + n])
    for i in range(c["dead"]):
        out[B - 1 - c["none"] - i][1] = 0
    return out


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _cuda(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a), dtype=dtype).to(DEV)


def _filled(shape, typ, scale, g):
    """Normal values of 1 / scale, in the type, made a piece at a time."""
    x = torch.empty(shape, device=DEV, dtype=TYPES[typ])
    for part in x.view(-1).split(1 << 27):
        part.copy_(torch.randn(part.shape, generator=g, device=DEV, dtype=torch.float32) / scale)
    return x


def prepare(case, seed):
    return {"chunk": _prepare_chunk, "logprobs": _prepare_logprobs, "fork": _prepare_fork, "release": _prepare_release,
            "compact": _prepare_compact}[case["op"]](case, seed)


def _prepare_chunk(c, seed):
    g, r = _gen(seed), np.random.RandomState(seed)
    B, nq, nkv, hd, bs = c["B"], c["nq"], c["nkv"], c["hd"], c["block"]
    chunks = np.array(_chunks(c))[r.permutation(B)]
    new, length = chunks[:, 0], chunks[:, 1]
    blocks = -(-length // bs)
    total = int(blocks.sum()) + 3
    ids = r.permutation(total)
    table = np.full((B, max(1, int(blocks.max()) + 1)), -1)
    ends = np.cumsum(blocks)
    for b in range(B):
        table[b, :blocks[b]] = ids[ends[b] - blocks[b]:ends[b]]
    cu = np.concatenate([[0], np.cumsum(new)])
    n = int(cu[-1]) + 5                                            # the batch's buffers are longer than its tokens
    scales = (K_SCALE, V_SCALE) if c["cache"] == "e4m3" else (1.0, 1.0)
    qkv = _filled((n, (nq + 2 * nkv) * hd), c["type"], 1.0, g)
    k, v = (_filled((total * bs, nkv, hd), c["cache"], s, g) for s in scales)
    return dict(c=c, q=qkv[:, :nq * hd], k=k, v=v, table=_cuda(table), length=_cuda(length), cu=_cuda(cu), scales=scales,
                chunks=[(int(a), int(b)) for a, b in zip(new, length)], out=torch.zeros(n, nq, hd, device=DEV,
                                                                                        dtype=TYPES[c["type"]]),
                lse=torch.zeros(n, nq, device=DEV))


def _prepare_logprobs(c, seed):
    g, r = _gen(seed), np.random.RandomState(seed)
    n, V = c["n"], c["V"]
    logits = _filled((n, V), c["type"], 0.4, g)
    tok = r.randint(0, V, n)
    for i in range(n):
        what = r.rand()
        if what < 0.05:                                            # constrained decoding: some ids are masked
            logits[i, torch.rand(V, generator=g, device=DEV) < 0.4] = -math.inf
        elif what < 0.08:
            tok[i] = -1                                            # a padded row
        elif what < 0.5:
            tok[i] = -2                                            # the best token, as most answers are
    if n > 3:
        logits[n // 2] = -math.inf                                 # a row that its mask leaves empty
    tok = _cuda(tok, torch.int64)
    best = torch.cat([x.argmax(-1) for x in logits.split(64)])
    return dict(c=c, logits=logits, tok=torch.where(tok == -2, best, tok).int())


def _rows(c):
    """Tokens of the rows: family by family, `fan` rows that share the family's full blocks."""
    fan = c["fan"]
    return [(p, [p + 1 + (5 * j + 3 * i) % c["grow"] for i in range(fan)])
            for j, p in enumerate(_spread(c["lo"], c["hi"], c["live"]))]


def _blocks(c):
    """Blocks in use, each counted once."""
    bs = c["block"]
    return sum(p // bs + sum(-(-n // bs) - p // bs for n in rows) for p, rows in _rows(c))


def _pool(rows, bs, num_blocks, r, empty=0):
    """Block tables of families of rows (their order dealt), holders beyond the first by block, and the free ids."""
    ids = r.permutation(num_blocks)
    B = sum(len(x) for _, x in rows) + empty
    place = r.permutation(B)
    mb = max(-(-n // bs) for _, x in rows for n in x) + 1
    table, length, shared = np.full((B, mb), -1), np.zeros(B, dtype=np.int64), np.zeros(num_blocks, dtype=np.int64)
    at, row, families = 0, 0, []
    for p, x in rows:
        whole = p // bs
        mine = ids[at:at + whole]
        at += whole
        shared[mine] = len(x) - 1
        families.append([])
        for n in x:
            b, more = place[row], -(-n // bs) - whole
            table[b, :whole] = mine
            table[b, whole:whole + more] = ids[at:at + more]
            length[b] = n
            at, row = at + more, row + 1
            families[-1].append(b)
    free = np.full(num_blocks, -1)
    free[:num_blocks - at] = ids[at:]
    return dict(table=_cuda(table), length=_cuda(length), shared=_cuda(shared), free=_cuda(free), n_free=_cuda([num_blocks - at]),
                num_blocks=num_blocks), families, place[row:]


def _cache(c, num_blocks, g):
    return _filled((2, c["layers"], num_blocks * c["block"], c["nkv"], c["hd"]), c["type"], 1.0, g)


def _prepare_fork(c, seed):
    g, r = _gen(seed), np.random.RandomState(seed)
    bs, n = c["block"], c["live"] * c["fan"]
    rows = [(0, [p]) for p in _spread(c["lo"], c["hi"], c["live"])]
    used = sum(-(-x[0] // bs) for _, x in rows)
    need = c["fan"] * sum(x[0] % bs > 0 for _, x in rows)
    num_blocks = used + max(0, need - c["short"]) + (0 if c["short"] else 7)
    pool, families, empty = _pool(rows, bs, num_blocks, r, empty=n)
    src = np.repeat(np.array([f[0] for f in families]), c["fan"])[r.permutation(n)]
    kv = _cache(c, num_blocks, g)
    return dict(pool, c=c, src=_cuda(src), dst=_cuda(empty), n=n, k=kv[0], v=kv[1])


def _prepare_release(c, seed):
    r = np.random.RandomState(seed)
    rows = _rows(c)
    pool, families, _ = _pool(rows, c["block"], _blocks(c) + 40, r)
    drop = np.zeros(pool["length"].numel())
    for j, f in enumerate(families):
        drop[f[:(j + 1) % (c["fan"] + 1)]] = 1                     # one of a family's rows, ..., all of them, none
    return dict(pool, c=c, drop=_cuda(drop))


def _num_blocks(c):
    return int(_blocks(c) / c["full"]) + 1


def _prepare_compact(c, seed):
    g, r = _gen(seed), np.random.RandomState(seed)
    pool, _, _ = _pool(_rows(c), c["block"], _num_blocks(c), r)
    kv = _cache(c, _num_blocks(c), g)
    return dict(pool, c=c, k=kv[0], v=kv[1])


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["c"]["op"]
    if own:
        return {"chunk": _own_chunk, "logprobs": _own_logprobs, "fork": _own_fork, "release": _own_release,
                "compact": _own_compact}[op](state)
    return {"chunk": _plain_chunk, "logprobs": _plain_logprobs, "fork": _plain_fork, "release": _plain_release,
            "compact": _plain_compact}[op](state)


def _plain_chunk(s):
    c = s["c"]
    nq, nkv, hd, bs = c["nq"], c["nkv"], c["hd"], c["block"]
    G, at = nq // nkv, 0
    for b, (n, length) in enumerate(s["chunks"]):
        first = length - n                                         # cache index of the first new token
        lo = max(0, first - c["window"] + 1) if c["window"] else 0
        if length == 0:
            s["out"][at:at + n] = 0
            s["lse"][at:at + n] = -math.inf
            at += n
            continue
        if n == 0:
            continue
        t = torch.arange(lo, length, device=DEV)
        slot = s["table"][b].long()[t // bs] * bs + t % bs
        kv = []
        for x, scale in zip((s["k"], s["v"]), s["scales"]):
            x = x.view(torch.uint8)[slot].view(x.dtype) if c["cache"] == "e4m3" else x[slot]
            kv.append((x.float() * scale).transpose(0, 1))         # [nkv, T, hd]
        step = max(1, int(2.5e8) // (nq * len(t)))
        for i in range(0, n, step):
            m = min(step, n - i)
            q = s["q"][at + i:at + i + m].float().view(m, nkv, G, hd).transpose(0, 1).reshape(nkv, m * G, hd) / math.sqrt(hd)
            x = (q @ kv[0].transpose(1, 2)).view(nkv, m, G, len(t))
            pos = torch.arange(first + i, first + i + m, device=DEV)[:, None]
            seen = t <= pos
            if c["window"]:
                seen &= t > pos - c["window"]
            x = x.masked_fill_(~seen[:, None, :], -math.inf)
            top = x.amax(-1, keepdim=True)                         # every row has its own token at least
            x = x.sub_(top).exp_()
            total = x.sum(-1, keepdim=True)
            y = (x.view(nkv, m * G, len(t)) @ kv[1]).view(nkv, m, G, hd) / total
            s["out"][at + i:at + i + m] = y.transpose(0, 1).reshape(m, nq, hd).to(s["out"].dtype)
            s["lse"][at + i:at + i + m] = (top + total.log())[..., 0].transpose(0, 1).reshape(m, nq)
        at += n
    return {"out": s["out"], "lse": s["lse"]}


def _plain_logprobs(s):
    c = s["c"]
    k, parts = c["k"], []
    ids = torch.arange(c["V"], device=DEV)
    for x, tok in zip(s["logits"].split(256), s["tok"].long().split(256)):
        x = x.float()
        x = torch.where(x.isfinite(), x, -math.inf)
        m = x.amax(-1, keepdim=True)
        base = torch.where(m.isfinite(), m, 0)
        e = torch.exp(x - base)
        total = e.sum(-1, dtype=torch.float64)                     # a vocabulary's sums in 64 bits
        lse = base[:, 0].double() + torch.log(total)
        moment = (e * torch.where(e > 0, x - base, 0)).sum(-1, dtype=torch.float64)
        entropy = torch.where(total > 0, torch.log(total) - moment / total, 0)
        mine = x.gather(1, tok.clamp(min=0)[:, None])
        has = (tok >= 0) & mine[:, 0].isfinite()
        before = (x > mine) | ((x == mine) & (ids < tok[:, None]))
        rank = torch.where(has, before.sum(-1), -1)
        logprob = torch.where(has, mine[:, 0].double() - lse, -math.inf)
        val, at = torch.sort(x, dim=-1, descending=True, stable=True)
        val, at = val[:, :k], at[:, :k]
        some = val > -math.inf
        top = torch.where(some, val.double() - lse[:, None], -math.inf)
        parts.append((logprob.float(), rank.int(), entropy.float(), lse.float(), torch.where(some, at, -1).int(), top.float()))
    names = ("logprob", "rank", "entropy", "lse", "top_ids", "top_logprob")
    return {name: torch.cat(p) for name, p in zip(names, zip(*parts))}


def _copy(x, typ, to, frm):
    x = x.view(torch.uint8) if typ == "e4m3" else x
    x[:, to] = x[:, frm]


def _plain_fork(s):
    c = s["c"]
    bs, mb = c["block"], s["table"].shape[1]
    table, length, n_free = s["table"].long(), s["length"].long(), s["n_free"].long()[0]
    src, dst = s["src"].long(), s["dst"].long()
    n = length[src]
    whole, rest = n // bs, n % bs
    need = rest > 0
    nth = need.cumsum(0) - need.long()
    served = ~need | (nth < n_free)
    takes = need & served
    place = (n_free - 1 - nth).clamp(min=0)
    new = s["free"].long()[place]
    i = torch.arange(mb, device=DEV)
    full = i < whole[:, None]
    rows = torch.where(full, table[src], torch.where((i == whole[:, None]) & need[:, None], new[:, None], -1))
    table_out = table.clone()
    table_out[dst] = torch.where(served[:, None], rows, table[dst])
    length_out = length.clone()
    length_out[dst] = torch.where(served, n, length[dst])
    ids = table[src][full & served[:, None]]
    shared = s["shared"].long() + torch.bincount(ids, minlength=s["num_blocks"])
    free = s["free"].long().clone()
    free[place[takes]] = -1
    old = table[src, whole.clamp(max=mb - 1)]
    r = torch.arange(bs, device=DEV)
    pick = (takes[:, None] & (r < rest[:, None])).nonzero(as_tuple=True)
    to, frm = new[pick[0]] * bs + pick[1], old[pick[0]] * bs + pick[1]
    for x in (s["k"], s["v"]):
        _copy(x, c["type"], to, frm)
    out = dict(table=table_out, length=length_out, shared=shared, free=free, n_free=(n_free - takes.sum()).view(1))
    return {**{k: v.int() for k, v in out.items()}, "k": s["k"], "v": s["v"]}


def _plain_release(s):
    bs, (B, mb), N = s["c"]["block"], s["table"].shape, s["num_blocks"]
    table, length, shared, n = s["table"].long(), s["length"].long(), s["shared"].long(), s["n_free"].long()
    drop = s["drop"] != 0
    i = torch.arange(mb, device=DEV)
    held = (i * bs < length[:, None]) & drop[:, None]
    code = torch.arange(B, device=DEV)[:, None] * mb + i
    ids, code = table[held], code[held]                            # by row, then by place
    count = torch.bincount(ids, minlength=N)
    last = torch.full((N,), -1, device=DEV).scatter_reduce(0, ids, code, "amax")
    back = (count > shared).nonzero()[:, 0]                        # the last holder has let go
    back = back[torch.argsort(last[back])]
    j = torch.arange(N, device=DEV)
    free = torch.where(j < n, s["free"].long(), -1)
    free[n + torch.arange(len(back), device=DEV)] = back
    out = dict(table=torch.where(drop[:, None], -1, table), length=torch.where(drop, 0, length),
               shared=(shared - count).clamp(min=0), free=free, n_free=n + len(back))
    return {k: v.int() for k, v in out.items()}


def _plain_compact(s):
    c, N = s["c"], s["num_blocks"]
    bs, mb = c["block"], s["table"].shape[1]
    table, length = s["table"].long(), s["length"].long()
    held = torch.arange(mb, device=DEV) * bs < length[:, None]
    used = torch.zeros(N, dtype=torch.bool, device=DEV)
    used[table[held]] = True
    U = used.sum()
    ids = torch.arange(N, device=DEV)
    to, frm = (~used & (ids < U)).nonzero()[:, 0], (used & (ids >= U)).nonzero()[:, 0]
    where = ids.clone()
    where[frm] = to
    shared = s["shared"].long().clone()
    shared[to] = shared[frm]
    shared[frm] = 0
    out = dict(table=torch.where(held, where[table.clamp(min=0)], -1), shared=shared,
               free=torch.where(ids < N - U, N - 1 - ids, -1), n_free=(N - U).view(1))
    r = torch.arange(bs, device=DEV)
    to, frm = ((x[:, None] * bs + r).view(-1) for x in (to, frm))
    for x in (s["k"], s["v"]):
        _copy(x, c["type"], to, frm)
    return {**{k: v.int() for k, v in out.items()}, "k": s["k"], "v": s["v"]}


# ------------------------------------------------------------------ the library's calls
def _lib():
    from eagle_speculative_decoding_step_gb300 import binding
    return binding


def _kept(s, make):
    """What a program keeps between calls on the same buffers: descriptors, workspace, output buffers."""
    if "kept" not in s:
        s["kept"] = make(_lib())
    return s["kept"]


def _zeros(nbytes):
    return torch.zeros(nbytes, device=DEV, dtype=torch.uint8)


def _own_chunk(s):
    lib, c = _lib(), s["c"]
    n = s["out"].shape[0]

    def make(lib):
        desc = lib.make_attn_desc(c["nq"], c["nkv"], c["hd"], c["type"], c["cache"], window=c["window"], k_scale=K_SCALE,
                                  v_scale=V_SCALE)
        return dict(desc=desc, ws=_zeros(lib.spec_chunk_attention_workspace_bytes(desc, c["B"], n)),
                    kv=lib.make_kv(dict(k=s["k"], v=s["v"], block_table=s["table"], block_size=c["block"],
                                        max_blocks=s["table"].shape[1], num_slots=s["k"].shape[0])))
    k = _kept(s, make)
    lib.spec_chunk_attention(k["desc"], s["q"], k["kv"], s["cu"], s["length"], c["B"], n, s["out"], s["lse"], k["ws"],
                             max_chunk=max(a for a, _ in s["chunks"]), max_len=max(b for _, b in s["chunks"]),
                             q_ld=s["q"].stride(0))
    return {"out": s["out"], "lse": s["lse"]}


def _own_logprobs(s):
    lib, c = _lib(), s["c"]
    n, V, top = c["n"], c["V"], c["k"]

    def make(lib):
        f, i = (lambda *a: torch.empty(*a, device=DEV)), (lambda *a: torch.empty(*a, device=DEV, dtype=torch.int32))
        return dict(ws=_zeros(lib.spec_token_logprobs_workspace_bytes(n, V, top)),
                    out=dict(logprob=f(n), rank=i(n), entropy=f(n), lse=f(n), top_ids=i(n, top), top_logprob=f(n, top)))
    k = _kept(s, make)
    lib.spec_token_logprobs(n, V, c["type"], s["logits"], s["tok"], top, ws=k["ws"], **k["out"])
    return dict(k["out"])


def _block_state(lib, s):
    """The pool's state, updated into other buffers (a pass can be taken again)."""
    o = {name: torch.empty_like(s[name]) for name in ("table", "length", "shared", "free", "n_free")}
    st = lib.make_block_state(s["c"]["block"], s["table"], o["table"], s["length"], o["length"], s["shared"], o["shared"],
                              s["free"], o["free"], s["n_free"], o["n_free"])
    return dict(out=o, st=st, ws=_zeros(lib.spec_block_state_workspace_bytes(s["table"].shape[0], s["num_blocks"])))


def _layers(lib, s):
    c = s["c"]
    return lib.make_kv_layers([dict(k=s["k"][i], v=s["v"][i], block_table=None, block_size=c["block"], max_blocks=0,
                                    num_slots=s["k"].shape[1]) for i in range(c["layers"])])


def _row_bytes(c):
    return c["nkv"] * c["hd"] * BYTES[c["type"]]


def _own_fork(s):
    lib = _lib()
    k = _kept(s, lambda lib: dict(_block_state(lib, s), kvs=_layers(lib, s)))
    lib.spec_block_fork(k["st"], s["n"], s["src"], s["dst"], k["kvs"], _row_bytes(s["c"]), k["ws"])
    return {**k["out"], "k": s["k"], "v": s["v"]}


def _own_release(s):
    lib = _lib()
    k = _kept(s, lambda lib: _block_state(lib, s))
    lib.spec_block_release(k["st"], s["drop"], k["ws"])
    return dict(k["out"])


def _own_compact(s):
    lib = _lib()
    k = _kept(s, lambda lib: dict(_block_state(lib, s), kvs=_layers(lib, s)))
    lib.spec_block_compact(k["st"], k["kvs"], _row_bytes(s["c"]), k["ws"])
    out = {name: k["out"][name] for name in ("table", "shared", "free", "n_free")}
    return {**out, "k": s["k"], "v": s["v"]}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "chunk":
        W, keys, pairs, rows = c["window"], 0, 0, 0
        for n, length in _chunks(c):
            rows += n
            if n == 0 or length == 0:
                continue
            first = length - n
            keys += length - (max(0, first - W + 1) if W else 0)
            if W:
                short = min(n, max(0, W - 1 - first))              # rows that see fewer keys than the window
                pairs += short * (first + 1) + short * (short - 1) // 2 + (n - short) * W
            else:
                pairs += n * (first + 1) + n * (n - 1) // 2
        q = rows * c["nq"] * c["hd"]
        return {"bytes": keys * c["nkv"] * c["hd"] * 2 * BYTES[c["cache"]] + 2 * q * BYTES[c["type"]] + 4 * rows * c["nq"],
                "flops": 4 * pairs * c["nq"] * c["hd"]}
    if c["op"] == "logprobs":
        return {"bytes": c["n"] * (c["V"] * BYTES[c["type"]] + 20 + 8 * c["k"]), "flops": 5 * c["n"] * c["V"]}
    bs = c["block"]
    row = 2 * c.get("layers", 0) * c.get("nkv", 0) * c.get("hd", 0) * BYTES[c.get("type", "f32")]
    if c["op"] == "fork":
        length = _spread(c["lo"], c["hi"], c["live"])
        moved = sum(n % bs for n in length) * c["fan"] * (1 - c["short"] / (c["live"] * c["fan"]))
        entries = sum(n // bs + 1 for n in length)
        return {"bytes": 4 * entries * (1 + 3 * c["fan"]) + 2 * moved * row, "flops": 0}
    rows = _rows(c)
    if c["op"] == "release":
        entries = back = 0
        for j, (p, x) in enumerate(rows):
            gone = (j + 1) % (c["fan"] + 1)
            entries += sum(-(-n // bs) for n in x[:gone])
            back += sum(-(-n // bs) - p // bs for n in x[:gone]) + (p // bs if gone == c["fan"] else 0)
        return {"bytes": 4 * (4 * entries + back + 2 * len(rows) * c["fan"]), "flops": 0}
    used, N = _blocks(c), _num_blocks(c)
    entries = sum(-(-n // bs) for _, x in rows for n in x)
    return {"bytes": 4 * (2 * entries + 2 * N) + 2 * used * (N - used) / N * bs * row, "flops": 0}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    c = case
    if c["op"] not in ("chunk", "logprobs"):
        return None                                                # indices, and rows that are moved as they are
    s = prepare(case, seed)
    if c["op"] == "chunk":
        nkv, bs, G = c["nkv"], c["block"], c["nq"] // c["nkv"]
        n = s["out"].shape[0]
        out = torch.zeros(n, c["nq"], c["hd"], dtype=torch.float64, device=DEV)
        lse = torch.zeros(n, c["nq"], dtype=torch.float64, device=DEV)
        q = s["q"].unflatten(1, (c["nq"], c["hd"]))
        cu = s["cu"].tolist()
        for b, length in enumerate(s["length"].tolist()):
            new = cu[b + 1] - cu[b]
            if length == 0:
                lse[cu[b]:cu[b + 1]] = -math.inf
            if length == 0 or new == 0:
                continue
            key = torch.arange(length, device=DEV)
            at = s["table"][b].long()[key // bs] * bs + key % bs
            step = max(1, int(2e8) // (G * length))
            for h in range(nkv):
                k = s["k"][:, h].view(torch.uint8)[at].view(s["k"].dtype) if c["cache"] == "e4m3" else s["k"][at, h]
                v = s["v"][:, h].view(torch.uint8)[at].view(s["v"].dtype) if c["cache"] == "e4m3" else s["v"][at, h]
                k, v = k.double() * s["scales"][0], v.double() * s["scales"][1]
                heads = slice(h * G, (h + 1) * G)
                for i in range(cu[b], cu[b + 1], step):
                    rows = slice(i, min(i + step, cu[b + 1]))
                    back = (length - new + torch.arange(i - cu[b], rows.stop - cu[b], device=DEV))[:, None] - key
                    hide = back < 0
                    if c["window"]:
                        hide |= back >= c["window"]
                    x = torch.einsum("mgd,td->mgt", q[rows, heads].double(), k) * c["hd"] ** -0.5
                    x.masked_fill_(hide[:, None], -math.inf)
                    lse[rows, heads] = torch.logsumexp(x, -1)
                    out[rows, heads] = torch.softmax(x, -1) @ v
        return {"out": out, "lse": lse}
    n, k = c["n"], c["k"]
    res = dict(logprob=torch.full((n,), -math.inf, dtype=torch.float64, device=DEV), rank=None,
               entropy=torch.zeros(n, dtype=torch.float64, device=DEV),
               lse=torch.full((n,), -math.inf, dtype=torch.float64, device=DEV), top_ids=None,
               top_logprob=torch.full((n, k), -math.inf, dtype=torch.float64, device=DEV))
    for i, tok in enumerate(s["tok"].tolist()):
        x = s["logits"][i].double()
        ok = x[torch.isfinite(x)]
        if not ok.numel():
            continue
        lp = torch.log_softmax(ok, 0)
        res["lse"][i] = torch.logsumexp(ok, 0)
        res["entropy"][i] = -(lp.exp() * lp).sum()
        best = lp.topk(min(k, len(lp))).values
        res["top_logprob"][i, :len(best)] = best
        if tok >= 0 and torch.isfinite(x[tok]):
            res["logprob"][i] = x[tok] - res["lse"][i]
    return res
