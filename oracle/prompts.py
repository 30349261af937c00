"""fp64 oracle of prompts and samples over the paged cache: attention of a chunk of new tokens,
log-probabilities of given tokens, and blocks that several requests share (fork, release, compact).
Plain loops over requests, from the definitions of include/eaglespec.h."""
import numpy as np


def chunk_attention(q, k, v, table, block_size, cu, seq_len, window=0, scale=0.0, spread=False):
    """q [n_rows, nq, hd]; k, v [slots, nkv, hd] (as the stored values stand for); out [n_rows, nq, hd] and lse [n_rows, nq]
    with NaN in rows of no request.  spread: also sum_j p_j |v_j| (as out) and max_j sum_c |q_c k_jc| * scale (as lse), what
    roundings of the weights and of the scores are relative to."""
    n_rows, nq, hd = q.shape
    nkv = k.shape[1]
    G = nq // nkv
    scale = scale or 1.0 / np.sqrt(hd)
    out, lse = np.full((n_rows, nq, hd), np.nan), np.full((n_rows, nq), np.nan)
    mass, size = np.zeros_like(out), np.zeros_like(lse)
    for b in range(len(seq_len)):
        lo, hi, length = int(cu[b]), int(cu[b + 1]), int(seq_len[b])
        if hi <= lo:
            continue
        pos = length - (hi - lo) + np.arange(hi - lo)
        t = np.arange(length)
        slots = table[b, t // block_size].astype(np.int64) * block_size + t % block_size
        there = (table[b, t // block_size] >= 0) & (slots < k.shape[0])
        seen = (t <= pos[:, None]) & there
        if window:
            seen &= t > pos[:, None] - window
        slots = np.where(there, slots, 0)
        for h in range(nkv):
            kk, vv = k[slots, h].astype(np.float64), v[slots, h].astype(np.float64)
            qq = q[lo:hi, h * G:(h + 1) * G].astype(np.float64)
            with np.errstate(invalid="ignore", over="ignore"):
                s = np.where(seen[:, None], np.einsum("mgd,td->mgt", qq, kk) * scale, -np.inf)
                m = s.max(-1, initial=-np.inf)
                base = np.where(np.isneginf(m), 0.0, m)
                e = np.where(np.isneginf(s), 0.0, np.exp(s - base[..., None]))
                l = e.sum(-1)
                p = e / np.where(l == 0, 1.0, l)[..., None]
                odd = ~np.isfinite(vv)
                o = np.einsum("mgt,td->mgd", p, np.where(odd, 0.0, vv))
                if odd.any():                              # on the rows that attend to the key
                    o[(np.einsum("mt,td->md", seen.astype(float), odd.astype(float)) > 0)[:, None].repeat(G, 1)] = np.nan
                out[lo:hi, h * G:(h + 1) * G] = o
                lse[lo:hi, h * G:(h + 1) * G] = np.where(l == 0, -np.inf, base + np.log(np.where(l == 0, 1.0, l)))
                if spread:
                    mass[lo:hi, h * G:(h + 1) * G] = np.einsum("mgt,td->mgd", p, np.abs(np.where(odd, 0.0, vv)))
                    a = np.where(seen[:, None], np.einsum("mgd,td->mgt", np.abs(qq), np.abs(kk)) * scale, 0.0)
                    size[lo:hi, h * G:(h + 1) * G] = a.max(-1, initial=0.0)
    return (out, lse, mass, size) if spread else (out, lse)


def token_logprobs(logits, tok, k):
    """logits [n, V], tok [n]: logprob, rank, entropy, lse [n], top_ids and top_logprob [n, k]."""
    n, V = logits.shape
    r = dict(logprob=np.full(n, -np.inf), rank=np.full(n, -1), entropy=np.zeros(n), lse=np.full(n, -np.inf),
             top_ids=np.full((n, k), -1), top_logprob=np.full((n, k), -np.inf))
    for i in range(n):
        x = logits[i].astype(np.float64)
        x = np.where(np.isfinite(x), x, -np.inf)
        if np.isneginf(x).all():
            continue
        m = x.max()
        e = np.exp(x - m)
        log_s = np.log(e.sum())
        r["lse"][i] = m + log_s
        p = e / e.sum()
        r["entropy"][i] = log_s - (p * np.where(p > 0, x - m, 0.0)).sum()
        order = np.lexsort((np.arange(V), -x))
        order = order[np.isfinite(x[order])]
        best = order[:k]
        r["top_ids"][i, :len(best)], r["top_logprob"][i, :len(best)] = best, x[best] - m - log_s
        t = int(tok[i])
        if 0 <= t < V and np.isfinite(x[t]):
            r["logprob"][i], r["rank"][i] = x[t] - m - log_s, int(np.where(order == t)[0][0])
    return r


# ------------------------------------------------------------------ blocks that several requests share
def _state(table, length, shared, free, n_free):
    return dict(table=np.array(table), length=np.array(length), shared=np.array(shared), free=np.array(free),
                n_free=int(n_free))


def block_fork(block_size, table, length, shared, free, n_free, src, dst):
    """The state after, "copies" [(from block, to block, slots)], "short" and "bad"."""
    r = _state(table, length, shared, free, n_free)
    B, mb = r["table"].shape
    N, cap = len(r["shared"]), mb * block_size
    old, named, need = np.array(length), set(), 0
    r.update(copies=[], short=False, bad=False)
    for a, d in zip(map(int, src), map(int, dst)):
        first = 0 <= d < B and d not in named
        if 0 <= d < B:
            named.add(d)
        if not (first and 0 <= a < B and old[d] == 0 and 0 <= old[a] <= cap):
            r["bad"] = True
            continue
        whole, rest = divmod(int(old[a]), block_size)
        nth = need
        need += rest > 0
        if rest and nth >= n_free:
            r["short"] = True
            continue
        row = np.full(mb, -1)
        for j in range(whole):
            i = int(table[a][j])
            if 0 <= i < N:
                row[j] = i
                r["shared"][i] += 1
            else:
                r["bad"] = True
        if rest:
            at = n_free - 1 - nth
            fresh, i = int(free[at]), int(table[a][whole])
            r["free"][at] = -1
            if 0 <= fresh < N:
                row[whole] = fresh
                if 0 <= i < N:
                    r["copies"].append((i, fresh, rest))
            r["bad"] |= not (0 <= fresh < N and 0 <= i < N)
        r["table"][d], r["length"][d] = row, old[a]
    r["n_free"] = n_free - min(need, n_free)
    return r


def block_release(block_size, table, length, shared, free, n_free, drop):
    r = _state(table, length, shared, free, n_free)
    B, mb = r["table"].shape
    N = len(r["shared"])
    gone, last, bad = np.zeros(N, dtype=int), {}, False
    for b in range(B):
        if not drop[b]:
            continue
        if not 0 <= length[b] <= mb * block_size:
            bad = True
            continue
        for j in range(-(-int(length[b]) // block_size)):
            i = int(table[b][j])
            if not 0 <= i < N:
                bad = True
                continue
            gone[i] += 1
            last.pop(i, None)
            last[i] = True                                 # dicts keep the order of insertion
        r["table"][b], r["length"][b] = -1, 0
    for i in last:
        bad |= gone[i] > shared[i] + 1
        if gone[i] > shared[i]:
            r["free"][r["n_free"]] = i
            r["n_free"] += 1
        r["shared"][i] = max(0, shared[i] - gone[i])
    r["bad"] = bad
    return r


def block_compact(block_size, table, length, shared, free, n_free):
    r = _state(table, length, shared, free, n_free)
    r.update(copies=[], refused=False)
    N = len(r["shared"])
    used = set()
    for b in range(len(r["table"])):
        if not 0 <= length[b] <= r["table"].shape[1] * block_size:
            r["refused"] = True
            return r
        used |= set(int(i) for i in table[b][:-(-int(length[b]) // block_size)])
    U = len(used)
    if U + n_free != N or any(not 0 <= i < N for i in used):
        r["refused"] = True
        return r
    to = [i for i in range(U) if i not in used]
    frm = sorted(i for i in used if i >= U)
    where = dict(zip(frm, to))
    r["copies"] = [(f, t, block_size) for f, t in zip(frm, to)]
    for f, t in zip(frm, to):
        r["shared"][t], r["shared"][f] = shared[f], 0
    for b in range(len(r["table"])):
        have = -(-int(length[b]) // block_size)
        r["table"][b] = [where.get(int(i), int(i)) if j < have else -1 for j, i in enumerate(table[b])]
    r["free"] = np.array([N - 1 - i if i < N - U else -1 for i in range(N)])
    r["n_free"] = N - U
    return r
