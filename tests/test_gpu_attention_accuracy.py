"""Attention of one new token against a bound that is worked out key by key (attention_bound): short rows, where a
weight's own bits show, and rows in which one key holds nearly all of the weight and has no value, so that the small
weights make the output."""
import numpy as np
import pytest
import torch

import attention_bound as ab
from eagle_speculative_decoding_step_gb300 import binding as lib

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
PAIRS = [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "e4m3"), ("f16", "e4m3")]


def stored(x, t, scale):
    """Rows as the cache holds them, and the values that they stand for."""
    y = torch.from_numpy(np.asarray(x) / scale).float()
    y = (y.clamp(-448, 448) if t == "e4m3" else y).to(TYPES[t])
    return y, y.double().numpy() * scale


def check(t, ct, bs, q, ks, vs, k_scale=1.0, v_scale=1.0, window=0, seed=0):
    """q [B, nq, hd]; ks, vs: of each request [n, nkv, hd]."""
    g = np.random.default_rng(seed)
    B, nq, hd = q.shape
    nkv, G = ks[0].shape[1], nq // ks[0].shape[1]
    lens = [len(k) for k in ks]
    blocks = [-(-n // bs) for n in lens]
    at = np.split(g.permutation(sum(blocks) + 2)[:sum(blocks)], np.cumsum(blocks)[:-1])
    table = np.full((B, max(blocks) + 1), -1)
    slots = (sum(blocks) + 2) * bs
    cache = [torch.full((slots, nkv, hd), float("nan")).to(TYPES[ct]) for _ in range(2)]
    values = [[], []]
    for b in range(B):
        table[b, :blocks[b]] = at[b]
        i = np.arange(lens[b])
        s = torch.from_numpy(table[b][i // bs] * bs + i % bs)
        for j, (x, scale) in enumerate(((ks[b], k_scale), (vs[b], v_scale))):
            y, val = stored(x, ct, scale)
            bits = torch.uint8 if ct == "e4m3" else TYPES[ct]
            cache[j].view(bits)[s] = y.view(bits)
            values[j].append(val)
    qt = torch.from_numpy(np.asarray(q)).to(TYPES[t])
    qv, qt = qt.double().numpy(), qt.cuda()
    table = torch.from_numpy(table).int().cuda()
    k, v = (x.cuda() for x in cache)
    kv = lib.make_kv(dict(k=k, v=v, block_table=table, block_size=bs, max_blocks=table.shape[1], num_slots=slots))
    desc = lib.make_attn_desc(nq, nkv, hd, t, ct, window=window, k_scale=k_scale, v_scale=v_scale)
    ws = torch.zeros(lib.spec_attention_workspace_bytes(desc, B), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(qt), torch.empty(B, nq, device="cuda")
    lib.spec_paged_attention(desc, qt, kv, torch.tensor(lens, dtype=torch.int32, device="cuda"), B, out, lse, ws)
    assert lib.spec_get_device_error(ws) == 0
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(B):
        lo = max(0, lens[b] - window) if window else 0
        for h in range(nq):
            kk, vv = (values[j][b][lo:, h // G] for j in range(2))
            o, tol, l, l_tol = ab.bound(qv[b, h], kk, vv, hd ** -0.5, t, ct)
            off = np.abs(out[b, h] - o)
            assert (off <= tol).all(), (b, h, lens[b], (off / tol).max(), int((off > tol).sum()))
            assert abs(lse[b, h] - l) <= l_tol, (b, h, lens[b], lse[b, h], l, l_tol)


def scales(ct):
    return (0.0625, 0.03125) if ct == "e4m3" else (1.0, 1.0)


@pytest.mark.parametrize("t,ct", PAIRS)
@pytest.mark.parametrize("nq,nkv,hd,bs", [(8, 2, 64, 16), (16, 2, 128, 16), (6, 3, 80, 24), (4, 2, 256, 16), (10, 1, 192, 8),
                                          (12, 1, 64, 1), (2, 2, 16, 32)])
def test_short_rows(t, ct, nq, nkv, hd, bs):
    g = np.random.default_rng(nq * hd)
    lens = [1, 2, 3, 5, 8, 15, 16, 17, 31, 33, 40, 64, 100]
    q = g.standard_normal((len(lens), nq, hd))
    check(t, ct, bs, q, *([g.standard_normal((n, nkv, hd)) for n in lens] for _ in range(2)), *scales(ct))


@pytest.mark.parametrize("t,ct", PAIRS)
@pytest.mark.parametrize("nq,nkv,hd,bs", [(4, 1, 64, 16), (16, 1, 128, 16), (4, 4, 80, 1), (8, 2, 256, 16)])
@pytest.mark.parametrize("first", [True, False])
def test_a_key_without_value_that_holds_nearly_all_of_the_weight(t, ct, nq, nkv, hd, bs, first):
    """The first key of the row, as a model's attention has it, or the last, after which all is scaled anew."""
    g = np.random.default_rng(hd + nq)
    lens, above = [1000, 300, 1000, 7000], [14.0, 22.0, 17.0, 16.0]
    q = ab.rounded(g.standard_normal((len(lens), nq, hd)), "bf16")
    ks, vs = [], []
    for b, n in enumerate(lens):
        x = [ab.sink(g, n, hd, above[b], q[b, h * (nq // nkv):(h + 1) * (nq // nkv)], hd ** -0.5) for h in range(nkv)]
        k, v = (np.stack([y[i] for y in x], 1) for i in range(2))
        ks.append(k if first else k[::-1])
        vs.append((v if first else v[::-1]) * 64)
    check(t, ct, bs, q, ks, vs, *((0.5, 2.0) if ct == "e4m3" else (1.0, 1.0)))


# ------------------------------------------------------------------ values that are not finite
def plain_call(t, q, k, v, bs=16):
    """One request of len(k) keys, blocks in order."""
    nq, hd = q.shape
    n, nkv = k.shape[:2]
    table = torch.arange(-(-n // bs), dtype=torch.int32, device="cuda")[None]
    pad = torch.zeros(table.numel() * bs - n, nkv, hd)
    k, v = (torch.cat([x, pad]).to(TYPES[t]).cuda() for x in (k, v))
    kv = lib.make_kv(dict(k=k, v=v, block_table=table, block_size=bs, max_blocks=table.numel(), num_slots=k.shape[0]))
    desc = lib.make_attn_desc(nq, nkv, hd, t)
    ws = torch.zeros(lib.spec_attention_workspace_bytes(desc, 1), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(1, nq, hd, dtype=TYPES[t], device="cuda"), torch.empty(1, nq, device="cuda")
    lib.spec_paged_attention(desc, q.to(TYPES[t]).cuda(), kv, torch.tensor([n], dtype=torch.int32, device="cuda"), 1, out, lse, ws)
    return out[0].float().cpu(), lse[0].cpu()


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", [1, 40, 700])
def test_scores_that_are_not_finite(t, n):
    g = torch.Generator().manual_seed(n)
    q, k, v = torch.randn(4, 64, generator=g), torch.randn(n, 2, 64, generator=g), torch.randn(n, 2, 64, generator=g)
    q[0, 3], q[1, 3], q[2:, 3] = 1.0, -1.0, 0.0               # of head 0: scores of +infinity, -infinity; of head 1: NaN
    i = n // 2
    k[i, :, 3] = float("inf")
    out, lse = plain_call(t, q, k, v)
    assert not torch.isfinite(out[0]).any() and not torch.isfinite(lse[0])
    assert not torch.isfinite(out[2:]).any() and not torch.isfinite(lse[2:]).any()
    if n == 1:                                                # no score but -infinity: as without keys
        assert (out[1] == 0).all() and lse[1] == -float("inf")
        return
    keep = torch.arange(n) != i
    rest, rest_lse = plain_call(t, q, k[keep], v[keep])
    assert torch.isfinite(out[1]).all()
    eps = torch.finfo(TYPES[t]).eps                           # the same sum in another order, rounded once each
    assert (out[1] - rest[1]).abs().max() <= eps * rest[1].abs().max() + 1e-5 and abs(lse[1] - rest_lse[1]) < 1e-5


# ------------------------------------------------------------------ forms that few calls take
def run_lens(t, ct, nq, nkv, hd, bs, lens, window=0):
    g = np.random.default_rng(nq + hd + bs + window)
    q = g.standard_normal((len(lens), nq, hd))
    check(t, ct, bs, q, *([g.standard_normal((n, nkv, hd)) for n in lens] for _ in range(2)), *scales(ct), window=window)


@pytest.mark.parametrize("t,ct", PAIRS)
@pytest.mark.parametrize("nq,nkv,hd,bs", [(128, 1, 256, 16), (80, 1, 192, 16), (136, 2, 256, 1), (100, 1, 144, 24), (128, 1, 128, 16)])
def test_more_query_tiles_than_warps(t, ct, nq, nkv, hd, bs):
    """Over 64 queries a K/V head above 128 components (fp32: over 32, and over 64 below that): K and V are read once for
    each split."""
    run_lens(t, ct, nq, nkv, hd, bs, [1, 17, 40, 200])


@pytest.mark.parametrize("t,ct", PAIRS)
@pytest.mark.parametrize("bs", [1, 2, 3, 4, 12, 20, 100])
def test_blocks_that_are_no_multiple_of_eight(t, ct, bs):
    """A key a copy; block and slot of a key by shifts or by divisions."""
    run_lens(t, ct, 8, 2, 64, bs, [1, 2, 13, 64, 129, 700])
    run_lens(t, ct, 4, 4, 128, bs, [5, 33, 300])


@pytest.mark.parametrize("t,ct", PAIRS)
@pytest.mark.parametrize("bs", [1, 2, 4, 12, 8, 24, 16])
@pytest.mark.parametrize("window", [1, 7, 50, 300])
def test_windows_on_any_block_size(t, ct, bs, window):
    run_lens(t, ct, 8, 2, 64, bs, [1, 6, 7, 8, 51, 299, 301, 900], window)
