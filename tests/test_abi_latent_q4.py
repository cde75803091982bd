"""Host-side argument checks of the latent-cache and block entry points: bad
calls are refused before anything is launched (no GPU needed)."""
import ctypes

import pytest

NULL = None
FAKE = ctypes.c_void_p(1 << 20)        # aligned, never dereferenced: checks fail first
ODD = ctypes.c_void_p((1 << 20) + 4)
F32, BF16, FP8, Q4 = 0, 1, 2, 3
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 6


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__
    __graft_entry__._builder().build()
    import top_kv_selection_b200 as m
    return m


def test_row_bytes(dsa):
    assert dsa.dsa_latent_q4_row_bytes(512, 64) == 416
    for dc in (128, 256, 384, 512):
        for dr in range(0, 65, 8):
            rb = dsa.dsa_latent_q4_row_bytes(dc, dr)
            assert rb % 16 == 0 and 0 <= rb - (dc // 2 + 2 * dr + dc // 16) < 16
            assert rb != dsa.dsa_latent_row_bytes(dc, dr)      # the binding tells them apart


def prologue(L, **kw):
    a = dict(kv=FAKE, dt=BF16, bs=8 * 576, ts=576, B=2, S=8, dc=512, dr=64, w=FAKE, eps=1e-6, cs=FAKE,
             il=1, sp=0, t_max=8, cache=FAKE, fmt=Q4)
    a.update(kw)
    return L.dsa_latent_prologue(a["kv"], a["dt"], a["bs"], a["ts"], a["B"], a["S"], a["dc"], a["dr"], a["w"],
                                 a["eps"], a["cs"], a["il"], a["sp"], a["t_max"], a["cache"], a["fmt"], NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(dc=500), UNSUPPORTED), (dict(dr=72), UNSUPPORTED), (dict(dr=4), UNSUPPORTED),
    (dict(dc=640, ts=704), UNSUPPORTED),
    (dict(dt=2), INVALID), (dict(fmt=F32), INVALID), (dict(fmt=4), INVALID),
    (dict(kv=NULL), INVALID), (dict(cache=NULL), INVALID), (dict(kv=ODD), INVALID), (dict(cache=ODD), INVALID),
    (dict(w=ODD), INVALID), (dict(cs=ODD), INVALID),
    (dict(sp=1), INVALID),                                     # row 8 past the cache
    (dict(sp=-1), INVALID), (dict(B=-1), INVALID), (dict(S=-1), INVALID),
    (dict(ts=568), INVALID),                                   # tokens would overlap
    (dict(ts=580), INVALID), (dict(bs=8 * 576 + 4), INVALID),  # not multiples of 16 bytes
    (dict(dt=F32, ts=578), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(B=0, kv=NULL, cache=NULL), OK), (dict(S=0, kv=NULL, cache=NULL), OK),
])
def test_prologue_checks(dsa, kw, status):
    assert prologue(dsa._lib, **kw) == status


def read(L, **kw):
    a = dict(cache=FAKE, fmt=Q4, t_max=100, idx=NULL, sp=0, B=2, n=100, dc=512, dr=64, out=FAKE, dt=BF16)
    a.update(kw)
    return L.dsa_latent_read(a["cache"], a["fmt"], a["t_max"], a["idx"], a["sp"], a["B"], a["n"], a["dc"],
                             a["dr"], a["out"], a["dt"], NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(dc=96), UNSUPPORTED), (dict(dr=65), UNSUPPORTED), (dict(fmt=F32), INVALID), (dict(dt=Q4), INVALID),
    (dict(sp=1), INVALID), (dict(sp=-1), INVALID), (dict(n=-1), INVALID), (dict(B=-1), INVALID),
    (dict(cache=NULL), INVALID), (dict(out=NULL), INVALID), (dict(out=ODD), INVALID), (dict(cache=ODD), INVALID),
    (dict(idx=ctypes.c_void_p((1 << 20) + 2)), INVALID),
    (dict(idx=FAKE, t_max=0), INVALID),
    (dict(n=0, cache=NULL, out=NULL), OK), (dict(B=0, cache=NULL, out=NULL), OK),
])
def test_read_checks(dsa, kw, status):
    assert read(dsa._lib, **kw) == status


def keys(L, **kw):
    a = dict(k=FAKE, ks=FAKE, t_max=128, B=2, sp=0, S=128, D=128, m=64, bk=FAKE, bs=FAKE, n_max=2)
    a.update(kw)
    return L.dsa_block_keys(a["k"], a["ks"], a["t_max"], a["B"], a["sp"], a["S"], a["D"], a["m"], a["bk"],
                            a["bs"], a["n_max"], NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(D=96), UNSUPPORTED), (dict(m=0), INVALID), (dict(n_max=1), INVALID), (dict(sp=1), INVALID),
    (dict(sp=-1), INVALID), (dict(k=NULL), INVALID), (dict(bk=ODD), INVALID), (dict(k=ODD), INVALID),
    (dict(B=0, k=NULL), OK),
    (dict(S=63, k=NULL), OK),                                  # no block is finished: nothing to write
    (dict(sp=64, S=0, k=NULL), OK),
])
def test_block_keys_checks(dsa, kw, status):
    assert keys(dsa._lib, **kw) == status


def attn(dsa, blocks, **kw):
    L = dsa._lib
    a = dict(q=FAKE, kv=FAKE, fmt=Q4, t_max=4096, sel=FAKE, B=1, S=1, Hq=128, dc=512, dr=64, k=2048, m=64,
             sp=4095, out=FAKE, lse=FAKE, ws=FAKE, wsb=1 << 30)
    if blocks:
        a["k"] = 32
    a.update(kw)
    head = (a["q"], a["kv"]) + ((a["fmt"],) if blocks else ())
    mid = (a["t_max"], a["sel"], a["B"], a["S"], a["Hq"], a["dc"], a["dr"], a["k"])
    mid += (a["m"],) if blocks else ()
    fn = L.dsa_block_mla_attn if blocks else L.dsa_sparse_mla_attn_q4
    return fn(*head, *mid, a["sp"], 0.04, a["out"], a["lse"], a["ws"], a["wsb"], NULL)


@pytest.mark.parametrize("blocks", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(dc=500), UNSUPPORTED), (dict(dr=72), UNSUPPORTED), (dict(Hq=1025), UNSUPPORTED),
    (dict(sp=4096), INVALID), (dict(sp=-1), INVALID), (dict(k=-1), INVALID), (dict(B=-1), INVALID),
    (dict(q=ODD), INVALID), (dict(kv=ODD), INVALID), (dict(out=ODD), INVALID), (dict(q=NULL), INVALID),
    (dict(sel=NULL), INVALID), (dict(out=NULL), INVALID), (dict(lse=ctypes.c_void_p((1 << 20) + 2)), INVALID),
    (dict(t_max=1 << 32), INVALID),
    (dict(B=1 << 20, S=1 << 12, sp=0), UNSUPPORTED),
    (dict(B=0, q=NULL), OK), (dict(S=0, q=NULL), OK), (dict(Hq=0, q=NULL), OK),
])
def test_attention_checks(dsa, blocks, kw, status):
    assert attn(dsa, blocks, **kw) == status


def test_block_attention_checks(dsa):
    assert attn(dsa, False, k=0) == INVALID           # a list of positions is not empty
    assert attn(dsa, True, k=1, sel=NULL) == INVALID
    assert attn(dsa, True, k=0, sel=NULL, B=0) == OK
    assert attn(dsa, True, m=0) == INVALID
    assert attn(dsa, True, fmt=F32) == INVALID
    assert attn(dsa, True, k=1 << 20, m=1 << 20) == UNSUPPORTED
    assert attn(dsa, True, m=(1 << 20) + 1) == UNSUPPORTED


def test_workspace_checks(dsa):
    L = dsa._lib
    need = L.dsa_sparse_mla_attn_q4_workspace_size(1, 1, 128, 512, 64, 2048)
    assert attn(dsa, False, wsb=need - 1) == WORKSPACE
    assert attn(dsa, False, ws=NULL) == WORKSPACE
    assert attn(dsa, False, ws=ODD) == WORKSPACE
    assert attn(dsa, False, k=0x7FFFFFFF) == UNSUPPORTED
    assert attn(dsa, True, k=0x7FFFFFFF, m=1) == UNSUPPORTED
    assert L.dsa_sparse_mla_attn_q4_workspace_size(1, 1, 128, 500, 64, 2048) == 0
    assert L.dsa_block_mla_attn_workspace_size(1, 1, 128, 512, 64, 32, 0) == 0
    assert L.dsa_block_mla_attn_workspace_size(1, 1, 128, 512, 64, 1 << 20, 1 << 20) == 0
    assert L.dsa_block_mla_attn_workspace_size(1, 1, 128, 512, 64, 0x7FFFFFFF, 1) == 0
    # partials for the splits of few rows, none once every SM has a row
    assert 0 < need <= 20 << 20
    assert L.dsa_sparse_mla_attn_q4_workspace_size(1, 4096, 128, 512, 64, 2048) == 0
    assert L.dsa_sparse_mla_attn_q4_workspace_size(0, 1, 128, 512, 64, 2048) == 0


def test_decode_step_takes_the_4_bit_cache(dsa):
    L = dsa._lib
    need = L.dsa_decode_step_workspace_size(8, 64, 128, 131072, 2048, 128, 512, 64, Q4)
    assert need >= 8 * 131072 * 4

    def call(dt=Q4, dc=512, ws_bytes=need, Hq=128):
        return L.dsa_decode_step(FAKE, FAKE, FAKE, FAKE, FAKE, 131072, FAKE, FAKE, 8, 64, 128, Hq, dc, 64,
                                 131072, 2048, 0.088, 0.041, dt, FAKE, FAKE, NULL, FAKE, ws_bytes, NULL)
    assert call(dt=4) == INVALID
    assert call(dc=96) == UNSUPPORTED                 # a bf16 shape, not a 4-bit one
    assert call(Hq=1025) == UNSUPPORTED
    assert call(ws_bytes=need - 1) == WORKSPACE


@pytest.mark.parametrize("sp", [(1 << 63) - 1, (1 << 63) - 4])
def test_a_position_near_the_end_of_64_bits_is_refused(dsa, sp):
    """Its sum with the number of tokens does not fit 64 bits."""
    L = dsa._lib
    assert prologue(L, sp=sp) == INVALID
    assert read(L, sp=sp) == INVALID
    assert keys(L, sp=sp) == INVALID
    for blocks in (False, True):
        assert attn(dsa, blocks, sp=sp, S=8) == INVALID


def test_row_counts_past_64_bits_are_refused(dsa):
    L = dsa._lib
    for blocks in (False, True):          # B * S * Hq = 2^64
        assert attn(dsa, blocks, B=1 << 30, S=1 << 30, Hq=16, sp=0, t_max=(1 << 31) - 1, k=16) == UNSUPPORTED
    assert read(L, idx=FAKE, B=4, n=1 << 61) == INVALID
    assert keys(L, B=1 << 30, S=(1 << 34), t_max=1 << 34, n_max=1 << 34, m=1) == UNSUPPORTED


def test_block_keys_refuse_blocks_past_their_counters(dsa):
    """A block near 2^31 tokens would take the kernel's token counter past 32 bits."""
    for m in ((1 << 20) + 1, (1 << 31) - 1, (1 << 31) - 100):
        assert keys(dsa._lib, m=m, t_max=1 << 32, S=1 << 32) == UNSUPPORTED
        assert keys(dsa._lib, m=m, t_max=1 << 32, S=1, D=64) == UNSUPPORTED
    assert keys(dsa._lib, m=1 << 20, k=NULL, S=(1 << 20) - 1, t_max=1 << 20) == OK      # finishes no block


def test_decode_step_refuses_selections_past_the_attentions(dsa):
    """2^30 rows and more, which dsa_sparse_mla_attn_q4 refuses too (its slot numbers are 32-bit)."""
    L = dsa._lib
    T = (1 << 31) - 1

    def size(T, topk, dt=Q4):
        return L.dsa_decode_step_workspace_size(1, 1, 64, T, topk, 1, 128, 0, dt)

    def call(T, topk):
        return L.dsa_decode_step(FAKE, FAKE, FAKE, FAKE, FAKE, T, FAKE, FAKE, 1, 1, 64, 1, 128, 0, T, topk, 0.1,
                                 0.1, Q4, FAKE, FAKE, NULL, FAKE, 0, NULL)
    for K in (1 << 30, T - 100, T):
        assert size(T, K) == 0 and call(T, K) == UNSUPPORTED
        assert L.dsa_decode_step_noalloc(FAKE, FAKE, FAKE, FAKE, FAKE, T, FAKE, FAKE, 1, 1, 64, 1, 128, 0, T, K,
                                         0.1, 0.1, Q4, FAKE, FAKE, NULL, NULL) in (UNSUPPORTED, 3)   # (3: no device)
    # min(index_topk, T) counts, and the largest selection is taken (its scores alone are T floats)
    assert size(T, (1 << 30) - 1) >= 4 * T and call(T, (1 << 30) - 1) == WORKSPACE
    assert size(1000, T) >= 4000 and call(1000, T) == WORKSPACE


@pytest.mark.parametrize("blocks", [False, True])
def test_selections_of_more_entries_than_31_bits_are_taken(dsa, blocks):
    """2^20 query rows of 2048 entries: no documented limit refuses them (the misaligned query
    is what this call stops at)."""
    kw = dict(S=1 << 20, t_max=1 << 21, sp=0, Hq=16, k=2048, q=ODD)
    assert attn(dsa, blocks, **kw, **(dict(m=16) if blocks else {})) == INVALID
    assert attn(dsa, blocks, **{**kw, "Hq": 1024, "S": 1 << 21}) == UNSUPPORTED       # B * S * Hq = 2^31


def test_binding_refuses_other_types_than_bf16_over_the_4_bit_cache(dsa):
    """The kernel reads q_mla and writes out as bf16 whatever the tensors hold."""
    import torch
    cache = torch.zeros(1, 4, 416, dtype=torch.uint8)
    q, out = torch.zeros(1, 2, 576, dtype=torch.bfloat16), torch.zeros(1, 2, 512, dtype=torch.bfloat16)
    assert dsa._kv_dtype(cache, q, out, 512) == Q4
    for bad in ((q.float(), out), (q, out.float()), (q.half(), out)):
        with pytest.raises(ValueError):
            dsa._kv_dtype(cache, *bad, 512)
    assert dsa._kv_dtype(torch.zeros(1, 4, 656, dtype=torch.uint8), q, out, 512) == FP8
    assert dsa._kv_dtype(q, q, out, 512) == BF16
