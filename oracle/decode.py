"""fp64 / integer oracle of decoding without speculation over the paged cache:
block tables and slot maps, K/V append, attention of one new token, beam
selection and reordering.  Plain loops over requests, from the definitions."""
import math

import numpy as np


def block_tables(block_size, num_blocks, len_old, len_new, table, free, n_free, cap):
    """Returns dict(table, free, n_free, length, cu, slots, pos, short): `free` is
    [num_blocks] padded with -1; `short` = some request was not served."""
    table = np.array(table, dtype=np.int64)
    B, mb = table.shape
    pool = [int(x) for x in free[:n_free]]
    have = [-(-int(o) // block_size) for o in len_old]
    want = [-(-int(n) // block_size) for n in len_new]
    for b in range(B):
        for i in range(want[b], have[b]):
            pool.append(int(table[b, i]))
            table[b, i] = -1
    avail, asked = len(pool), 0
    length, slots, pos, cu = [], [], [], [0]
    for b in range(B):
        need = max(want[b] - have[b], 0)
        asked += need
        ok = need == 0 or asked <= avail
        if ok:
            for i in range(have[b], want[b]):
                table[b, i] = pool.pop()
        length.append(int(len_new[b]) if ok else int(len_old[b]))
        for t in range(int(len_old[b]), int(len_new[b])):
            slots.append(int(table[b, t // block_size]) * block_size + t % block_size if ok else -1)
            pos.append(t)
        cu.append(len(slots))
    pad = lambda a, n, v: np.array(list(a[:n]) + [v] * (n - len(a)))  # noqa: E731
    return dict(table=table, free=pad(pool, num_blocks, -1), n_free=len(pool), length=np.array(length), cu=np.array(cu),
                slots=pad(slots, cap, -1), pos=pad(pos, cap, 0), short=asked > avail)


def e4m3_values():
    """The 256 values of the 8-bit type (NaN at 127 and 255)."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = -1.0 if c & 128 else 1.0, (c >> 3) & 15, c & 7
        out[c] = s * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    out[127] = out[255] = math.nan
    return out


def e4m3_round(x):
    """Nearest 8-bit value (ties to the even code), saturated at +-448; NaN stays."""
    grid = e4m3_values()[:127]                       # ascending, codes 0..126
    a = np.abs(np.asarray(x, dtype=np.float64))
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    r = np.where(a >= 448, 448.0, grid[code])
    return np.where(np.isnan(x), math.nan, np.copysign(r, x))


def slots_of(table_row, block_size, idx):
    return np.array([int(table_row[i // block_size]) * block_size + i % block_size for i in idx], dtype=np.int64)


def paged_attention(q, k, v, table, block_size, seq_len, window=0, scale=0.0, num_slots=None):
    """q [B, nq, hd], k / v [slots, nkv, hd] (values), table [B, blocks].  Keys whose
    block id is outside the cache are left out.  Returns out [B, nq, hd], lse [B, nq]."""
    B, nq, hd = q.shape
    nkv = k.shape[1]
    G = nq // nkv
    scale = scale or 1.0 / math.sqrt(hd)
    out, lse = np.zeros((B, nq, hd)), np.full((B, nq), -math.inf)
    for b in range(B):
        n = int(seq_len[b])
        idx = [i for i in range(max(0, n - window) if window else 0, n)
               if 0 <= int(table[b][i // block_size]) and int(table[b][i // block_size]) * block_size + i % block_size < k.shape[0]]
        if not idx:
            continue
        s = slots_of(table[b], block_size, idx)
        for h in range(nq):
            with np.errstate(invalid="ignore", over="ignore"):
                x = scale * (k[s, h // G].astype(np.float64) @ q[b, h].astype(np.float64))
                m = x.max()
                p = np.exp(x - m)
                lse[b, h] = m + math.log(p.sum()) if not math.isnan(p.sum()) else math.nan
                out[b, h] = (p / p.sum()) @ v[s, h // G].astype(np.float64)
    return out, lse


def beam_select(logits, score, done, eos):
    """logits [B, W, V], score / done [B, W]: (parent, tok, score, done) [B, W]."""
    B, W, V = logits.shape
    parent = np.tile(np.arange(W), (B, 1))
    tok, out, fin = np.full((B, W), -1), np.full((B, W), -math.inf), np.ones((B, W), dtype=int)
    for b in range(B):
        cand = []                                     # (-score, place, beam, token, finished)
        for j in range(W):
            s = float(score[b, j])
            if not math.isfinite(s):
                continue
            if done[b, j]:
                cand.append((-s, j * V + max(eos, 0), j, eos, True))
                continue
            x = logits[b, j].astype(np.float64)
            ok = np.nonzero(np.isfinite(x))[0]
            if len(ok) == 0:
                continue
            m = x[ok].max()
            lse = m + math.log(np.exp(x[ok] - m).sum())
            best = ok[np.lexsort((ok, -x[ok]))][:W]
            cand += [(-(s + (x[t] - lse)), j * V + int(t), j, int(t), False) for t in best]
        for r, (ns, _, j, t, f) in enumerate(sorted(cand)[:W]):
            parent[b, r], tok[b, r], out[b, r], fin[b, r] = j, t, -ns, f or t == eos
    return parent, tok, out, fin


def beam_reorder(block_size, parent, tok, seq_len, prompt_blocks, owned, table, spare, hist=None):
    """table [B, W, blocks], spare [B, W], hist [B, W, n] or None.  Returns dict(table,
    spare, slots, hist, copies); copies = [(from block, to block, slots)]."""
    B, W, mb = table.shape
    out, sp = np.full_like(table, -1), np.array(spare)
    slots, copies = np.full((B, W), -1), []
    ho = None if hist is None else np.full_like(hist, -1)
    for b in range(B):
        n = int(seq_len[b])
        i, r, P = n // block_size, n % block_size, int(prompt_blocks[b])
        for j in range(W):
            p = int(parent[b, j])
            out[b, j, :i] = table[b, p, :i]
            if r == 0:
                out[b, j, i] = owned[b, P + W + (i - P) * W + j]
            elif p == j:
                out[b, j, i] = table[b, j, i]
            else:
                out[b, j, i] = spare[b, j]
                sp[b, j] = table[b, j, i]
                copies.append((int(table[b, p, i]), int(spare[b, j]), r))
            slots[b, j] = out[b, j, i] * block_size + r
            if hist is not None:
                ho[b, j, :n] = hist[b, p, :n]
                ho[b, j, n] = tok[b, j]
    return dict(table=out, spare=sp, slots=slots, hist=ho, copies=copies)
