"""GPU parity of decoding without speculation (block tables, K/V append, attention of one
new token, beam selection and reordering) against the fp64 oracle."""
import math

import numpy as np
import pytest
import torch

from eagle_speculative_decoding_step_gb300 import binding as lib
from oracle import decode as oracle

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
ERR_DEVICE, ERR_CAPACITY = -6, -4


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def zeros(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def error(ws):
    return lib.spec_get_device_error(ws)


# ------------------------------------------------------------------ block tables
def tables_case(seed, B, bs, spare):
    g = np.random.default_rng(seed)
    most = max(3 * bs, 40)
    old = g.integers(0, most, B) * (g.random(B) < 0.7)
    new = np.where(g.random(B) < 0.6, old + g.integers(0, 9, B), g.integers(0, most + 8, B)) * (g.random(B) < 0.85)
    mb = -(-(most + 8) // bs) + 1
    have = -(-old // bs)
    nb = int(have.sum()) + spare
    ids = g.permutation(nb)
    table, at = np.full((B, mb), -1), 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    free = np.full(nb, -1)
    free[:nb - at] = ids[at:]
    return old, new, table, free, nb - at, nb


def run_tables(bs, old, new, table, free, n_free, nb, cap, in_place, pos=True):
    B, mb = table.shape
    o, n, t, f, nf = i32(old), i32(new), i32(table), i32(free), i32([n_free])
    ws = zeros(lib.spec_block_tables_workspace_bytes(B))
    e = lambda *s: torch.full(s, -77, dtype=torch.int32, device="cuda")  # noqa: E731
    t2, f2, nf2, l2 = (t, f, nf, o) if in_place else (e(B, mb), e(len(free)), e(1), e(B))
    cu, slots, p = e(B + 1), e(cap), e(cap) if pos else None
    lib.spec_block_tables(B, bs, mb, nb, o, n, t, t2, f, nf, f2, nf2, l2, cu, slots, p, cap, ws)
    err = error(ws)
    assert int(ws[256:260].view(torch.int32)[0]) == 0              # the counter is left at zero
    r = dict(table=t2, free=f2, length=l2, cu=cu, slots=slots)
    r = {k: v.cpu().numpy() for k, v in r.items()}
    return dict(r, n_free=int(nf2[0]), pos=p.cpu().numpy() if pos else None), err


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,bs,spare", [(1, 16, 5), (7, 1, 60), (64, 16, 200), (65, 24, 3), (600, 16, 700), (1500, 8, 100),
                                        (8192, 32, 9000), (40, 128, 0)])
def test_block_tables(B, bs, spare, in_place):
    old, new, table, free, n_free, nb = tables_case(B + bs, B, bs, spare)
    total = int(np.maximum(new - old, 0).sum())
    cap = total + 7
    ref = oracle.block_tables(bs, nb, old, new, table, free, n_free, cap)
    got, err = run_tables(bs, old, new, table, free, n_free, nb, cap, in_place)
    assert err == (ERR_CAPACITY if ref["short"] else 0)
    for k in ("table", "length", "cu", "slots", "pos"):
        np.testing.assert_array_equal(got[k], ref[k], err_msg=k)
    assert got["n_free"] == ref["n_free"]
    n = ref["n_free"] if in_place else nb
    np.testing.assert_array_equal(got["free"][:n], ref["free"][:n])


def test_block_tables_short_slot_map_and_bad_inputs():
    old, new, table = np.array([4, 0]), np.array([10, 5]), np.array([[3, -1, -1], [-1, -1, -1]])
    free = np.array([0, 1, 2, 4, 5, -1])
    ref = oracle.block_tables(4, 6, old, new, table, free, 5, 20)
    got, err = run_tables(4, old, new, table, free, 5, 6, 8, False, pos=False)      # 11 tokens, room for 8
    assert err == ERR_CAPACITY
    np.testing.assert_array_equal(got["slots"], ref["slots"][:8])
    np.testing.assert_array_equal(got["table"], ref["table"])
    # a length over the table's end: that request stays as it is, the other one is served
    got, err = run_tables(4, old, np.array([13, 5]), table, free, 5, 6, 20, False)
    assert err == ERR_DEVICE and got["length"].tolist() == [4, 5]
    assert got["table"].tolist() == [[3, -1, -1], [5, 4, -1]] and got["cu"].tolist() == [0, 0, 5]
    got, err = run_tables(4, np.array([-3, 0]), new, table, free, 5, 6, 20, False)
    assert err == ERR_DEVICE and got["length"].tolist() == [0, 5]
    # an id out of range in the pool reaches no table
    got, err = run_tables(4, old, np.array([4, 5]), table, np.array([0, 1, 2, 99, 5, -1]), 5, 6, 20, False)
    assert err == ERR_DEVICE and got["table"][1].tolist() == [5, -1, -1] and got["slots"][:5].tolist() == [20, 21, 22, 23, -1]
    # a pool count out of range
    _, err = run_tables(4, old, np.array([4, 5]), table, free, 70, 6, 20, False)
    assert err == ERR_DEVICE


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("t,c", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("nkv,hd,n,ld,off", [(8, 128, 37, 0, 0), (1, 16, 1, 0, 0), (3, 80, 130, 777, 3), (2, 256, 64, 2048, 512),
                                             (16, 64, 9, 0, 0)])
def test_cache_append(t, c, nkv, hd, n, ld, off):
    g = torch.Generator(device="cuda").manual_seed(n)
    w, slots = nkv * hd, n + 20
    ld = ld or 2 * w
    x = (torch.randn(n, ld + w + off, generator=g, device="cuda") * 3).to(TYPES[t])
    k, v = x[:, off:off + w], x[:, off + 5:off + 5 + w] if off % 8 else x[:, off + w // 2:off + w // 2 + w]
    k.view(torch.int32 if t == "f32" else torch.int16)[0, 0] = torch.tensor(float("nan"), dtype=TYPES[t]).view(
        torch.int32 if t == "f32" else torch.int16)
    k[0, 1], v[0, 2] = 1e4, -1e4
    at = np.random.default_rng(n).permutation(slots)[:n]
    if n > 8:
        at[3] = -1
    ck = torch.full((slots, nkv, hd), 2.0, device="cuda").to(TYPES[c])
    cv = ck.clone()
    ks, vs = 0.37, 0.11
    ws = zeros(256)
    kv = lib.make_kv(dict(k=ck, v=cv, block_table=None, block_size=1, max_blocks=0, num_slots=slots))
    lib.spec_cache_append(lib.make_attn_desc(nkv, nkv, hd, t, c, k_scale=ks, v_scale=vs), k, v, x.stride(0), i32(at), n, kv, ws)
    assert error(ws) == 0
    for cache, rows, s in ((ck, k, ks), (cv, v, vs)):
        rows = rows.float().cpu().numpy()
        if c == "e4m3":                                   # the quotient is taken in fp32 (the definition's rounding)
            rows = oracle.e4m3_round(np.float32(rows) / np.float32(s))
        ref = np.full((slots, w), 2.0)
        ref[at[at >= 0]] = rows[at >= 0]
        np.testing.assert_array_equal(cache.float().cpu().numpy().reshape(slots, w), ref.astype(np.float32))


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("ks,vs", [(0.0625, 1.0), (0.3, 1.7e-3), (7.1, 3e4)])
def test_cache_append_every_value_to_eight_bits(t, ks, vs):
    """All 65536 bit patterns: the quotient in fp32, then one rounding to nearest even, whatever the scale."""
    x = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(TYPES[t]).reshape(64, 1024)
    ck, cv = torch.zeros(2, 64, 8, 128, device="cuda").to(TYPES["e4m3"]).unbind(0)
    ws = zeros(256)
    kv = lib.make_kv(dict(k=ck, v=cv, block_table=None, block_size=1, max_blocks=0, num_slots=64))
    lib.spec_cache_append(lib.make_attn_desc(8, 8, 128, t, "e4m3", k_scale=ks, v_scale=vs), x, x, 0, i32(np.arange(64)), 64, kv,
                          ws)
    assert error(ws) == 0
    with np.errstate(over="ignore"):
        for cache, s in ((ck, ks), (cv, vs)):
            ref = oracle.e4m3_round(x.float().cpu().numpy() / np.float32(s))
            np.testing.assert_array_equal(cache.float().cpu().numpy().reshape(64, 1024), ref.astype(np.float32))


def test_cache_append_skips_slots_out_of_range():
    ck, cv = torch.zeros(2, 8, 1, 16, device="cuda").unbind(0)
    x = torch.ones(4, 16, device="cuda")
    ws = zeros(256)
    kv = lib.make_kv(dict(k=ck, v=cv, block_table=None, block_size=1, max_blocks=0, num_slots=8))
    lib.spec_cache_append(lib.make_attn_desc(1, 1, 16, "f32"), x, x, 0, i32([2, 8, -5, 7]), 4, kv, ws)
    assert error(ws) == ERR_DEVICE
    assert ck[:, 0, 0].tolist() == [0, 0, 1, 0, 0, 0, 0, 1] == cv[:, 0, 15].tolist()


# ------------------------------------------------------------------ attention
class Cache:
    """A paged cache whose slots outside the allowed keys hold NaN."""

    def __init__(self, seed, lens, nkv, hd, bs, t, window=0, ks=1.0, vs=1.0, spread=1.0, first_block=0):
        g = np.random.default_rng(seed)
        B = len(lens)
        blocks = [-(-n // bs) for n in lens]
        total = sum(blocks) + 3
        ids = g.permutation(total) + first_block
        mb = max(blocks) + 2
        self.table = np.full((B, mb), -1)
        self.bs, self.slots, self.lens = bs, (total + first_block) * bs, np.array(lens)
        self.k = torch.full((self.slots, nkv, hd), float("nan"), device="cuda").to(TYPES[t]) if first_block == 0 else \
            torch.empty(self.slots, nkv, hd, device="cuda", dtype=TYPES[t])
        self.v = self.k.clone() if first_block == 0 else torch.empty_like(self.k)
        at = 0
        for b, n in enumerate(lens):
            self.table[b, :blocks[b]] = ids[at:at + blocks[b]]
            at += blocks[b]
            idx = np.arange(max(0, n - window) if window else 0, n)
            if len(idx):
                s = torch.from_numpy(oracle.slots_of(self.table[b], bs, idx)).cuda()
                for x, scale in ((self.k, ks), (self.v, vs)):
                    r = torch.from_numpy(g.standard_normal((len(idx), nkv, hd)) * spread / scale).float().cuda()
                    r = (r.clamp(-448, 448) if t == "e4m3" else r).to(TYPES[t])       # stored saturated, as the append does
                    bits = torch.uint8 if t == "e4m3" else x.dtype
                    x.view(bits)[s] = r.view(bits)
        self.ttable = i32(self.table)

    def kv(self):
        return lib.make_kv(dict(k=self.k, v=self.v, block_table=self.ttable, block_size=self.bs,
                                max_blocks=self.table.shape[1], num_slots=self.slots))


def check_attention(c, desc, q, t, window, scale, ks, vs, out, lse, hd):
    """The kernel's sums are fp32: a score is off by E <= (hd + 4) 2^-24 scale sum|q k|, a weight by
    a factor exp(2 E) and what exp and the rescalings add, (n + 16) 2^-24 with n terms summed; a
    weight enters the second product as two 16-bit parts, 2^-17 of it at most is lost; the output is
    rounded once to its type."""
    k, v = c.k.double().cpu().numpy() * ks, c.v.double().cpu().numpy() * vs
    k, v = np.nan_to_num(k), np.nan_to_num(v)
    qd = q.double().cpu().numpy()
    ref, ref_lse = oracle.paged_attention(qd, k, v, c.table, c.bs, c.lens, window, scale)
    mass, _ = oracle.paged_attention(qd, k, np.abs(v), c.table, c.bs, c.lens, window, scale)
    sc = scale or hd ** -0.5
    E = (hd + 4) * 2.0 ** -24 * sc * np.abs(qd).max(-1) * np.abs(k).max() * hd
    rel = 2 * E + (c.lens.max() + 16) * 2.0 ** -24 + (0 if t == "f32" else 2.0 ** -17)
    tol = torch.finfo(TYPES[t]).eps / 2 * np.abs(ref) + 2 * rel[..., None] * mass + 1e-30
    got = out.double().cpu().numpy().reshape(ref.shape)
    bad = np.abs(got - ref) > tol
    assert not bad.any() and np.isfinite(got).all(), (np.argwhere(bad)[:5], (np.abs(got - ref) - tol).max())
    if lse is not None:
        gl = lse.double().cpu().numpy()
        live = np.isfinite(ref_lse)
        assert (gl[~live] == -math.inf).all()
        tl = E + (c.lens.max() + 16) * 2.0 ** -24 + 2.0 ** -23 * np.abs(np.where(live, ref_lse, 0))
        assert (np.abs(gl - ref_lse)[live] <= tl[live]).all()


def attend(seed, t, ct, lens, nq, nkv, hd, bs, window=0, scale=0.0, pad=0, max_len=0, with_lse=True, spread=1.0):
    ks, vs = (0.05, 0.02) if ct == "e4m3" else (1.0, 1.0)
    c = Cache(seed, lens, nkv, hd, bs, ct, window, ks, vs, spread)
    B = len(lens)
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn(B, nq * hd + pad, generator=g, device="cuda").to(TYPES[t])
    out = torch.full((B, nq * hd + pad), 7.0, device="cuda").to(TYPES[t])
    lse = torch.full((B, nq), 7.0, device="cuda") if with_lse else None
    desc = lib.make_attn_desc(nq, nkv, hd, t, ct, window=window, scale=scale, k_scale=ks, v_scale=vs)
    ws = zeros(lib.spec_attention_workspace_bytes(desc, B))
    for _ in range(2):                                     # the second call finds the counters as the first left them
        lib.spec_paged_attention(desc, q, c.kv(), i32(lens), B, out, lse, ws, max_len=max_len, q_ld=nq * hd + pad,
                                 out_ld=nq * hd + pad)
    assert error(ws) == 0
    if pad:
        assert (out[:, nq * hd:].float() == 7.0).all()
    check_attention(c, desc, q[:, :nq * hd].reshape(B, nq, hd), t, window, scale, ks, vs, out[:, :nq * hd], lse, hd)


PAIRS = [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "e4m3"), ("f16", "e4m3")]


@pytest.mark.parametrize("t,ct", PAIRS)
@pytest.mark.parametrize("nq,nkv,hd,bs", [(32, 8, 128, 16), (4, 4, 64, 16), (6, 2, 80, 24), (16, 1, 128, 8), (8, 8, 256, 32),
                                          (5, 1, 96, 1), (64, 4, 128, 128), (40, 8, 64, 16), (128, 1, 64, 16), (2, 1, 16, 16),
                                          (48, 16, 128, 16), (32, 1, 256, 16), (36, 3, 112, 16)])
def test_attention_shapes(t, ct, nq, nkv, hd, bs):
    attend(hd + nq, t, ct, [0, 1, 15, 16, 17, 129, 300, 2], nq, nkv, hd, bs)


@pytest.mark.parametrize("t,ct", PAIRS)
@pytest.mark.parametrize("nkv,hd,bs", [(8, 16, 16), (8, 32, 8), (4, 32, 16), (2, 64, 32), (6, 64, 16), (16, 48, 16), (3, 64, 8),
                                       (2, 144, 16), (2, 160, 24), (4, 192, 16), (1, 208, 1), (2, 224, 16)])
def test_attention_head_sizes(t, ct, nkv, hd, bs):
    """Heads that share 128 bytes, heads that fill no whole 128 bytes, and those above 128 components."""
    for group in (1, 5, 12):
        attend(hd + group, t, ct, [0, 1, 31, 33, 260, 700], group * nkv, nkv, hd, bs)


@pytest.mark.parametrize("t,ct", PAIRS)
@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 0], [4097], [33, 0, 5000, 1, 64, 65, 127, 128], [2] * 300])
def test_attention_lengths(t, ct, lens):
    attend(len(lens) + sum(lens), t, ct, lens, 8, 2, 64, 16)
    attend(len(lens) + sum(lens), t, ct, lens, 8, 4, 128, 16, max_len=max(lens))


@pytest.mark.parametrize("t,ct", PAIRS)
@pytest.mark.parametrize("window", [1, 16, 100, 1000])
def test_attention_window(t, ct, window):
    attend(window, t, ct, [0, 1, 99, 100, 101, 999, 1500], 16, 4, 128, 16, window=window)


@pytest.mark.parametrize("t,ct", PAIRS)
def test_attention_strides_scale_and_no_lse(t, ct):
    attend(5, t, ct, [40, 700], 8, 2, 64, 16, scale=0.3, pad=64, with_lse=False)
    attend(6, t, ct, [40, 700], 8, 2, 64, 16, spread=6.0)          # sharp rows: scores of tens


def test_attention_more_requests_than_a_launch_plans():
    g = np.random.default_rng(1)
    attend(9, "bf16", "bf16", [int(x) for x in g.integers(0, 40, 5000)], 2, 1, 64, 16)


def test_attention_unused_layout_hint_gives_the_same():
    """max_len only lays out work: with and without it, results agree to the tolerance."""
    for m in (0, 700, 8, 1 << 20):
        attend(11, "bf16", "bf16", [700, 3, 512], 32, 8, 128, 16, max_len=m)


def test_attention_is_deterministic():
    c = Cache(3, [5000, 17, 1200], 8, 128, 16, "bf16")
    q = torch.randn(3, 32, 128, device="cuda").bfloat16()
    desc = lib.make_attn_desc(32, 8, 128, "bf16")
    ws = zeros(lib.spec_attention_workspace_bytes(desc, 3))
    outs = []
    for _ in range(5):
        o = torch.empty_like(q)
        lib.spec_paged_attention(desc, q, c.kv(), i32(c.lens), 3, o, None, ws)
        outs.append(o)
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_attention_calls_of_all_shapes_share_a_workspace():
    """One workspace, calls of other shapes in between: the same bits as with a workspace of its own."""
    cases = [("bf16", "bf16", [30000], 32, 8, 128, 16), ("f32", "f32", [900, 0, 77], 16, 2, 64, 8),
             ("f16", "e4m3", [3000, 5, 2500, 1], 32, 2, 256, 16), ("bf16", "bf16", [40] * 200, 4, 4, 80, 24),
             ("bf16", "e4m3", [12345], 6, 3, 128, 32), ("f32", "f32", [5000, 4000], 8, 1, 256, 1)]
    calls, size = [], 0
    for i, (t, ct, lens, nq, nkv, hd, bs) in enumerate(cases):
        c = Cache(i, lens, nkv, hd, bs, ct, 0, 0.05, 0.02) if ct == "e4m3" else Cache(i, lens, nkv, hd, bs, ct)
        desc = lib.make_attn_desc(nq, nkv, hd, t, ct, k_scale=0.05, v_scale=0.02)
        q = torch.randn(len(lens), nq, hd, device="cuda").to(TYPES[t])
        own = zeros(lib.spec_attention_workspace_bytes(desc, len(lens)))
        size = max(size, own.numel())
        ref, lse = torch.empty_like(q), torch.empty(len(lens), nq, device="cuda")
        lib.spec_paged_attention(desc, q, c.kv(), i32(lens), len(lens), ref, lse, own)
        calls.append((desc, q, c, lens, ref, lse))
    shared = zeros(size)
    for _ in range(2):
        for desc, q, c, lens, ref, ref_lse in calls:
            out, lse = torch.empty_like(q), torch.empty_like(ref_lse)
            lib.spec_paged_attention(desc, q, c.kv(), i32(lens), len(lens), out, lse, shared)
            assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    assert error(shared) == 0


def test_attention_leaves_out_bad_blocks_and_clamps_lengths():
    c = Cache(4, [100, 64, 70], 2, 64, 16, "bf16")
    c.table[0, 2] = 10 ** 6                                         # its 16 keys are left out
    c.table[1, :] = -1                                              # nothing left
    c.ttable = i32(c.table)
    q = torch.randn(3, 8, 64, device="cuda").bfloat16()
    desc = lib.make_attn_desc(8, 2, 64, "bf16")
    ws = zeros(lib.spec_attention_workspace_bytes(desc, 3))
    out, lse = torch.empty_like(q), torch.empty(3, 8, device="cuda")
    lib.spec_paged_attention(desc, q, c.kv(), i32(c.lens), 3, out, lse, ws)
    assert error(ws) == ERR_DEVICE
    check_attention(c, desc, q, "bf16", 0, 0.0, 1.0, 1.0, out, lse, 64)
    ws.zero_()
    lib.spec_paged_attention(desc, q, c.kv(), i32([0, -4, 70]), 3, out, lse, ws)
    assert error(ws) == ERR_DEVICE and (out[:2] == 0).all() and out[2].abs().sum() > 0


def test_attention_values_that_are_not_finite_reach_their_own_rows_only():
    c = Cache(8, [50, 50], 2, 64, 16, "f16")
    s = int(oracle.slots_of(c.table[0], 16, [20])[0])
    c.v[s, 1, 5] = float("inf")
    q = torch.randn(2, 4, 64, device="cuda").half()
    desc = lib.make_attn_desc(4, 2, 64, "f16")
    ws = zeros(lib.spec_attention_workspace_bytes(desc, 2))
    out = torch.empty_like(q)
    lib.spec_paged_attention(desc, q, c.kv(), i32(c.lens), 2, out, None, ws)
    hit = ~torch.isfinite(out)
    assert hit[0, 2:, 5].all() and int(hit.sum()) == 2


def test_attention_offsets_past_32_bits():
    """A cache of more than 2^31 elements whose used blocks are the last ones."""
    c = Cache(12, [200, 33], 8, 128, 16, "bf16", first_block=132000)
    assert c.k.numel() > 2 ** 31
    q = torch.randn(2, 32, 128, device="cuda").bfloat16()
    desc = lib.make_attn_desc(32, 8, 128, "bf16")
    ws = zeros(lib.spec_attention_workspace_bytes(desc, 2))
    out = torch.empty_like(q)
    lib.spec_paged_attention(desc, q, c.kv(), i32(c.lens), 2, out, None, ws)
    assert error(ws) == 0
    base = 132000 * 16
    small = Cache.__new__(Cache)
    small.k, small.v, small.table, small.bs, small.lens = c.k[base:], c.v[base:], np.where(c.table >= 0, c.table - 132000, -1), 16, c.lens
    used = torch.zeros(small.k.shape[0], dtype=torch.bool)
    for b, n in enumerate(c.lens):
        used[oracle.slots_of(small.table[b], 16, np.arange(n))] = True
    small.k, small.v = (torch.where(used.cuda()[:, None, None], x, 0) for x in (small.k, small.v))
    check_attention(small, desc, q, "bf16", 0, 0.0, 1.0, 1.0, out, None, 128)


# ------------------------------------------------------------------ beam selection
def run_select(x, score, done, eos, t, ld=None):
    B, W, V = x.shape
    ld = ld or V
    buf = torch.zeros(B * W * ld + 3, device="cuda", dtype=TYPES[t])
    for r in range(B * W):
        buf[r * ld:r * ld + V] = x.reshape(B * W, V)[r].to(TYPES[t])
    ws = zeros(lib.spec_beam_workspace_bytes(B, W, V))
    e = lambda: torch.full((B, W), -77, dtype=torch.int32, device="cuda")  # noqa: E731
    p, tok, d, s = e(), e(), e(), torch.zeros(B, W, device="cuda")
    for _ in range(2):
        lib.spec_beam_select(B, W, V, t, buf, torch.as_tensor(score, dtype=torch.float32).cuda(), i32(done), eos, p, tok, s, d,
                             ws, ld=ld)
    assert error(ws) == 0
    vals = torch.stack([buf[r * ld:r * ld + V] for r in range(B * W)]).view(B, W, V)
    ref = oracle.beam_select(vals.double().cpu().numpy(), np.float32(score), np.asarray(done), eos)
    np.testing.assert_array_equal(p.cpu().numpy(), ref[0])
    np.testing.assert_array_equal(tok.cpu().numpy(), ref[1])
    np.testing.assert_array_equal(d.cpu().numpy(), ref[3])
    got, want = s.double().cpu().numpy(), ref[2]
    assert (np.isfinite(got) == np.isfinite(want)).all()
    f = np.isfinite(want)
    # an fp32 sum of exponentials (each 2^-21 off at most) is within 2^-20 of it, so is the lse; one rounding at the end
    assert (np.abs(got - want)[f] <= 2.0 ** -20 + 2.0 ** -24 * np.abs(want[f])).all()


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,W,V,ld", [(1, 4, 1000, None), (3, 1, 8192, None), (2, 8, 8193, 8197), (5, 5, 33, None),
                                      (2, 16, 40001, 40001), (1, 32, 20000, 20002), (2, 3, 2, None), (1, 2, 1, None)])
def test_beam_select(t, B, W, V, ld):
    g = np.random.default_rng(B * V + W)
    x = torch.from_numpy(g.standard_normal((B, W, V)) * 3).float().cuda()
    score = -g.random((B, W)) * 5 - 3
    done = (g.random((B, W)) < 0.2).astype(int)
    score[0, 1:] = -np.inf
    run_select(x, score, done, min(2, V - 1), t, ld)


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_beam_select_masks(t):
    g = np.random.default_rng(7)
    x = torch.from_numpy(g.standard_normal((6, 4, 9000)) * 3).float().cuda()
    x[0, 0] = -math.inf                                        # nothing left
    x[1] = -math.inf
    x[2, 1, ::2] = -math.inf
    x[3, 2, 10:] = torch.finfo(TYPES[t]).min                   # the type's lowest value is a logit like any other
    x[4, 0, 5], x[4, 0, 6] = math.nan, math.inf                # not finite: no candidates
    x[5, :, 8] = -math.inf
    score = -g.random((6, 4)) * 5
    score[5, 0], score[5, 1], score[5, 2] = math.nan, math.inf, -math.inf
    done = np.zeros((6, 4), dtype=int)
    done[1, 3] = 1
    run_select(x, score, done, 8, t)
    run_select(x, score, np.ones((6, 4), dtype=int), 8, t)     # all finished
    run_select(x, score, done, -1, t)


@pytest.mark.parametrize("W", [1, 8, 32])
def test_beam_select_ties_go_to_the_first(W):
    for V in (40, 8192, 30000):
        x = torch.zeros(2, W, V, device="cuda")                # every candidate ties: lists overflow
        run_select(x, np.zeros((2, W)), np.zeros((2, W), dtype=int), 0, "f32")
        g = np.random.default_rng(V)
        x = torch.from_numpy(np.round(g.standard_normal((2, 1, V)) * 2)).float().cuda().repeat(1, W, 1)
        run_select(x, np.full((2, W), -1.5), np.zeros((2, W), dtype=int), 3, "bf16", V + 1)


@pytest.mark.parametrize("W", [1, 5, 32])
@pytest.mark.parametrize("t", ["f32", "f16"])
def test_beam_select_rows_that_keep_rising(t, W):
    """Every later logit beats the best so far: the running candidate list overflows again and again."""
    V = 30011
    up = torch.arange(V, device="cuda") / V * 20 - 10
    x = torch.stack([up, up.flip(0), torch.where(torch.arange(V, device="cuda") % 5000 == 4999, up, -math.inf)])
    x = x.repeat(1, W).view(3, W, V) + torch.arange(W, device="cuda")[:, None] * 0.25
    run_select(x, -np.arange(3 * W).reshape(3, W) * 0.125, np.zeros((3, W), dtype=int), 7, t, V + 3)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_beam_select_rows_of_the_lowest_value_are_uniform(t):
    x = torch.full((2, 2, 9001), torch.finfo(TYPES[t]).min, device="cuda")
    x[1, 0, 17] = 3.0
    x[1, 1, 5] = -0.0
    x[1, 1, 6] = 0.0
    run_select(x, np.array([[-1.0, -2.0], [-1.0, -1.0]]), np.zeros((2, 2), dtype=int), 3, t)


# ------------------------------------------------------------------ reordering
@pytest.mark.parametrize("t", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("B,W,bs,layers,nkv,hd", [(1, 4, 16, 1, 8, 128), (5, 3, 4, 3, 1, 16), (3, 8, 1, 2, 2, 64), (9, 2, 24, 2, 1, 80),
                                                  (2, 32, 8, 64, 1, 16), (4, 1, 16, 1, 1, 64)])
def test_beam_reorder(t, B, W, bs, layers, nkv, hd):
    g = np.random.default_rng(B * W + bs)
    prompt = g.integers(0, 5 * bs + 3, B)
    n = prompt + g.integers(0, 3 * bs, B)
    n[0] = 3 * bs                                               # a block border
    prompt[0] = min(prompt[0], n[0])
    P, at = prompt // bs, n // bs
    mb, old = int(at.max()) + 3, int((P + W + (at - P + 1) * W).max())
    ids = g.permutation(B * old)
    owned = ids.reshape(B, old)
    table, spare = np.full((B, W, mb), -1), np.zeros((B, W), dtype=int)
    for b in range(B):
        table[b, :, :P[b]] = owned[b, :P[b]]
        spare[b] = owned[b, P[b]:P[b] + W]
        for i in range(P[b], at[b]):
            table[b, :, i] = owned[b, P[b] + W + (i - P[b]) * W + g.integers(0, W, W)]
        if n[b] % bs:
            table[b, :, at[b]] = owned[b, P[b] + W + (at[b] - P[b]) * W + np.arange(W)]
    hist = g.integers(0, 1000, (B, W, int(n.max()) + 2))
    parent, tok = g.integers(0, W, (B, W)), g.integers(0, 1000, (B, W))
    ref = oracle.beam_reorder(bs, parent, tok, n, P, owned, table, spare, hist)
    slots = B * old * bs
    k = (torch.randn(layers, slots, nkv, hd, device="cuda") * 4).to(TYPES[t])
    v = (torch.randn(layers, slots, nkv, hd, device="cuda") * 4).to(TYPES[t])
    k0, v0 = k.float().cpu(), v.float().cpu()
    e = lambda a: torch.full(np.shape(a), -77, dtype=torch.int32, device="cuda")  # noqa: E731
    to, so, sl, ho = e(table), e(spare), e(spare), e(hist)
    st = lib.make_beam_state(B, W, bs, mb, i32(parent), i32(tok), i32(n), i32(P), i32(owned), i32(table), to, i32(spare), so,
                             sl, i32(hist), ho)
    kvs = lib.make_kv_layers([dict(k=k[i], v=v[i], block_table=None, block_size=bs, max_blocks=0, num_slots=slots)
                              for i in range(layers)])
    ws = zeros(256)
    lib.spec_beam_reorder(st, kvs, nkv * hd * k.element_size(), ws)
    assert error(ws) == 0
    for got, name in ((to, "table"), (so, "spare"), (sl, "slots"), (ho, "hist")):
        np.testing.assert_array_equal(got.cpu().numpy(), ref[name], err_msg=name)
    for f, d, r in ref["copies"]:
        for x in (k0, v0):
            x[:, d * bs:d * bs + r] = x[:, f * bs:f * bs + r]
    assert torch.equal(k.float().cpu(), k0) and torch.equal(v.float().cpu(), v0)


def test_beam_reorder_bad_inputs_copy_nothing():
    def run(parent=(1, 0), n=3, P=1, owned=(4, 8, 9, 10, 11, 12, 13), table=((4, 10, -1), (4, 11, -1)), spare=(8, 9), mb=3):
        k = torch.arange(32.0, device="cuda").view(32, 1, 1).repeat(1, 1, 4)
        kv = lib.make_kv_layers([dict(k=k, v=k.clone(), block_table=None, block_size=2, max_blocks=0, num_slots=32)])
        e = lambda *s: torch.full(s, -77, dtype=torch.int32, device="cuda")  # noqa: E731
        to, so, sl = e(2, mb), e(2), e(2)
        st = lib.make_beam_state(1, 2, 2, mb, i32([parent]), i32([[5, 6]]), i32([n]), i32([P]), i32([owned]),
                                 i32(np.array(table)[:, :mb]), to, i32([spare]), so, sl)
        ws = zeros(256)
        lib.spec_beam_reorder(st, kv, 16, ws)
        return error(ws), to.tolist(), so.tolist(), sl.tolist(), k[:, 0, 0].tolist()
    same = list(map(float, range(32)))
    e, to, so, sl, k = run()
    assert e == 0 and sl == [17, 19] and k[16] == 22 and k[18] == 20 and so == [10, 11]
    e, to, so, sl, k = run(parent=(7, 0))
    assert e == ERR_DEVICE and to[0] == [4, 10, -1] and k[18] == 20 and k[16] == 16
    e, to, so, sl, k = run(spare=(99, -1))
    assert e == ERR_DEVICE and sl == [-1, -1] and k == same
    e, to, so, sl, k = run(n=4, owned=(4, 8, 9, 10, 11))
    assert e == ERR_CAPACITY and sl == [-1, -1] and k == same
    e, to, so, sl, k = run(n=9)
    assert e == ERR_CAPACITY and sl == [-1, -1] and k == same
    e, to, so, sl, k = run(n=-1)
    assert e == ERR_DEVICE and sl == [-1, -1] and k == same
    e, to, so, sl, k = run(P=5)
    assert e == ERR_DEVICE and sl == [-1, -1] and k == same


# ------------------------------------------------------------------ streams and graphs
def test_calls_follow_the_current_stream_and_can_be_captured():
    c = Cache(2, [300, 20], 2, 64, 16, "bf16")
    q = torch.randn(2, 8, 64, device="cuda").bfloat16()
    desc = lib.make_attn_desc(8, 2, 64, "bf16")
    ws, lens, kv = zeros(lib.spec_attention_workspace_bytes(desc, 2)), i32(c.lens), c.kv()
    a, b = torch.empty_like(q), torch.zeros_like(q)
    lib.spec_paged_attention(desc, q, kv, lens, 2, a, None, ws)
    x = torch.randn(2, 4, 5000, device="cuda")
    sws = zeros(lib.spec_beam_workspace_bytes(2, 4, 5000))
    sc, dn = torch.zeros(2, 4, device="cuda"), i32(np.zeros((2, 4)))
    o1 = [torch.zeros(2, 4, dtype=d, device="cuda") for d in (torch.int32, torch.int32, torch.float32, torch.int32)]
    o2 = [y.clone() for y in o1]
    lib.spec_beam_select(2, 4, 5000, "f32", x, sc, dn, 2, *o1, sws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        lib.spec_paged_attention(desc, q, kv, lens, 2, b, None, ws)
        lib.spec_beam_select(2, 4, 5000, "f32", x, sc, dn, 2, *o2, sws)
    for _ in range(3):
        b.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b) and all(torch.equal(p, r) for p, r in zip(o1, o2)) and error(ws) == 0
