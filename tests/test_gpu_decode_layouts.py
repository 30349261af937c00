"""GPU parity of the decoding calls at layouts and shapes that a model's rows can have, against the fp64 oracle."""
import numpy as np
import pytest
import torch

from eagle_speculative_decoding_step_gb300 import binding as lib
from eagle_speculative_decoding_step_gb300 import decode
from oracle import decode as oracle

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


# ------------------------------------------------------------------ strides of K and V
@pytest.mark.parametrize("t,c", [("bf16", "bf16"), ("f32", "f32"), ("f16", "e4m3")])
@pytest.mark.parametrize("nkv,hd,k_ld,v_ld,off", [(2, 64, 0, 512, 256), (2, 64, 512, 0, 256), (3, 80, 240, 777, 3), (3, 80, 777, 0, 3),
                                                  (8, 128, 1024, 6144, 5120)])
def test_cache_append_takes_k_and_v_of_other_strides(t, c, nkv, hd, k_ld, v_ld, off):
    """Values are small integers, which every type holds."""
    n, w = 37, nkv * hd
    g = torch.Generator(device="cuda").manual_seed(w + k_ld)

    def rows(ld, off):
        x = torch.randint(-8, 9, (n, ld or w), generator=g, device="cuda").to(TYPES[t])
        return x[:, off:off + w] if ld > w else x
    k, v = rows(k_ld, off), rows(v_ld, off)
    at = np.random.default_rng(n).permutation(n + 9)[:n]
    ck = torch.zeros(n + 9, nkv, hd, device="cuda").to(TYPES[c])
    cv = torch.zeros(n + 9, nkv, hd, device="cuda").to(TYPES[c])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    kv = lib.make_kv(dict(k=ck, v=cv, block_table=None, block_size=1, max_blocks=0, num_slots=n + 9))
    lib.spec_cache_append(lib.make_attn_desc(nkv, nkv, hd, t, c), k, v, k_ld, i32(at), n, kv, ws, v_ld=v_ld)
    assert lib.spec_get_device_error(ws) == 0
    for cache, x in ((ck, k), (cv, v)):
        ref = torch.zeros(n + 9, w)
        ref[torch.from_numpy(at)] = x.float().cpu()
        assert torch.equal(cache.float().cpu().view(n + 9, w), ref)


class Layouts(decode.RandomModel):
    def __init__(self, lay, **kw):
        super().__init__(**kw)
        self.lay = lay

    def __call__(self, tok, pos, attend):
        return super().__call__(tok, pos, lambda i, q, k, v: attend(i, *self.lay(q, k, v)))


def by_heads(x):
    return x.transpose(0, 1).contiguous().transpose(0, 1)


@pytest.mark.parametrize("kv_dtype", [None, "e4m3"])
def test_decoding_does_not_depend_on_the_layout_of_the_rows(kv_dtype):
    got = []
    for lay in (lambda q, k, v: (q, k, v), lambda q, k, v: (q, k.contiguous(), v), lambda q, k, v: (q, k, v.contiguous()),
                lambda q, k, v: (by_heads(q), by_heads(k), by_heads(v))):
        m = Layouts(lay, seed=1)
        c = decode.PagedCache(2, 64, 16, m.nq, m.nkv, m.hd, kv_dtype=kv_dtype, k_scale=0.02, v_scale=0.02)
        b = decode.Batch(m, c, 5, 64, m.vocab)
        logits = [b.feed(i32([3, 50, 7, 9, 1000 + t])) for t in range(20)]
        assert b.error() == 0
        got.append(torch.stack(logits))
    assert all(torch.equal(x, got[0]) for x in got[1:])


# ------------------------------------------------------------------ memory
@pytest.mark.parametrize("dtype,kv_dtype,es", [("bf16", None, 2), ("bf16", "e4m3", 1)])
def test_making_a_cache_takes_no_more_than_the_cache(dtype, kv_dtype, es):
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    c = decode.PagedCache(4, 4096, 16, 32, 8, 128, dtype=dtype, kv_dtype=kv_dtype)
    size = 2 * 4 * 4096 * 16 * 8 * 128 * es
    assert torch.cuda.max_memory_allocated() - before < size + c.ws.numel() + (1 << 22)


# ------------------------------------------------------------------ scales
@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("ks,vs", [(1e-39, 3e38), (2.9e-39, 1.1e38), (1.2e-38, 8.4e37), (1e-45, 1.9e38), (2.0 ** -127, 2.0 ** 127)])
def test_cache_append_to_eight_bits_with_scales_at_the_ends_of_their_type(t, ks, vs):
    """All 65536 bit patterns: the quotient in fp32, whatever the reciprocal of the scale is in that type."""
    x = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(TYPES[t]).reshape(64, 1024)
    ck, cv = torch.zeros(2, 64, 8, 128, device="cuda").to(TYPES["e4m3"]).unbind(0)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    kv = lib.make_kv(dict(k=ck, v=cv, block_table=None, block_size=1, max_blocks=0, num_slots=64))
    lib.spec_cache_append(lib.make_attn_desc(8, 8, 128, t, "e4m3", k_scale=ks, v_scale=vs), x, x, 0, i32(np.arange(64)), 64, kv,
                          ws)
    assert lib.spec_get_device_error(ws) == 0
    with np.errstate(all="ignore"):
        for cache, s in ((ck, ks), (cv, vs)):
            ref = oracle.e4m3_round(x.float().cpu().numpy() / np.float32(s))
            np.testing.assert_array_equal(cache.float().cpu().numpy().reshape(64, 1024), ref.astype(np.float32))


# ------------------------------------------------------------------ a cache that ends inside a block
@pytest.mark.parametrize("bs", [16, 8, 24, 12, 1])
@pytest.mark.parametrize("t,ct", [("bf16", "bf16"), ("f32", "f32"), ("f16", "e4m3")])
def test_keys_past_the_caches_end_are_left_out_and_told(bs, t, ct):
    """Block 3 lies partly in the cache; its other slots are out of range as a block id past the end is."""
    there = bs // 2
    slots = 3 * bs + there
    g = torch.Generator(device="cuda").manual_seed(bs)
    k, v = (torch.randn(slots, 2, 64, generator=g, device="cuda").to(TYPES[ct]) for _ in range(2))
    q = torch.randn(2, 4, 64, generator=g, device="cuda").to(TYPES[t])
    table = i32([[0, 1, 3, -1], [2, 0, 1, -1]])
    desc = lib.make_attn_desc(4, 2, 64, t, ct)
    ws = torch.zeros(lib.spec_attention_workspace_bytes(desc, 2), dtype=torch.uint8, device="cuda")
    kv = lib.make_kv(dict(k=k, v=v, block_table=table, block_size=bs, max_blocks=4, num_slots=slots))
    for lens, code in (([2 * bs + there, 3 * bs], 0), ([3 * bs, 3 * bs], -6), ([2 * bs + there + 1, 1], -6)):
        ws.zero_()
        out = torch.empty_like(q)
        lib.spec_paged_attention(desc, q, kv, i32(lens), 2, out, None, ws)
        assert lib.spec_get_device_error(ws) == code, lens
        ref, _ = oracle.paged_attention(q.double().cpu().numpy(), k.double().cpu().numpy(), v.double().cpu().numpy(),
                                        table.cpu().numpy(), bs, lens)
        assert np.abs(out.double().cpu().numpy() - ref).max() <= torch.finfo(TYPES[t]).eps * np.abs(ref).max() + 1e-5


def test_tables_of_half_a_billion_tokens_a_request():
    """Blocks of 2^20 slots: a call's requests go in launches of 31 or 127, whose tiles 32 bits count at any lengths."""
    B, bs, mb, slots = 200, 1 << 20, 512, 5000
    g = torch.Generator(device="cuda").manual_seed(0)
    for t in ("bf16", "f32"):
        k, v = (torch.randn(slots, 2, 64, generator=g, device="cuda").to(TYPES[t]) for _ in range(2))
        q = torch.randn(B, 4, 64, generator=g, device="cuda").to(TYPES[t])
        lens = i32((np.arange(B) * 37) % slots)
        desc = lib.make_attn_desc(4, 2, 64, t)
        ws = torch.zeros(lib.spec_attention_workspace_bytes(desc, B), dtype=torch.uint8, device="cuda")
        got = []
        for size, n in ((bs, mb), (8192, 1)):
            table = torch.full((B, n), -1, dtype=torch.int32, device="cuda")
            table[:, 0] = 0
            kv = lib.make_kv(dict(k=k, v=v, block_table=table, block_size=size, max_blocks=n, num_slots=slots))
            out, lse = torch.empty_like(q), torch.empty(B, 4, device="cuda")
            lib.spec_paged_attention(desc, q, kv, lens, B, out, lse, ws, max_len=slots)
            assert lib.spec_get_device_error(ws) == 0
            got.append((out, lse))
        (a, x), (b, y) = got                                  # cut in other places: the same but for the order of the sums
        eps = torch.finfo(TYPES[t]).eps
        assert (a.float() - b.float()).abs().max() <= 2 * eps * b.abs().max().float() + 1e-5
        assert torch.equal(torch.isfinite(x), torch.isfinite(y)) and (x - y).nan_to_num(0.0).abs().max() < 1e-5
