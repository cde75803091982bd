"""dsa_sparse_mla_attn_q4, dsa_block_mla_attn, dsa_block_keys and the decode step
over the 4-bit cache against 64-bit references.

Attention tolerance, per output element: the weights enter the value mix as
bf16 (half a step, 2^-8 of each term, so 2^-8 sum_j p_j |c_j|), the result is
rounded to bf16 (2^-8 |out|), and the fp32 logits are off by at most
dz = 2 sm_scale d 2^-24 max_j sum_i |q_i c_ji| (d products summed, truncating
adders allowed for), which moves each weight by 2 dz at most.  lse: dz, and
2^-18 for the exponentials, the sum and the logarithm."""
import numpy as np
import pytest
import torch

import latent_reference as R
import workloads

pytestmark = pytest.mark.gpu
FORMATS = [R.BF16, R.FP8, R.Q4]


@pytest.fixture(scope="module")
def dsa():
    import top_kv_selection_b200 as m
    return m


def make_cache(dsa, B, t_max, fmt, dc, dr, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    kv = (torch.randn(B, t_max, dc + dr, generator=g) * scale).cuda()
    raw = torch.zeros(B, t_max, R.row_bytes(fmt, dc, dr), dtype=torch.uint8, device="cuda")
    cache = raw.view(torch.bfloat16) if fmt == R.BF16 else raw
    dsa.dsa_latent_prologue(kv, None, 0.0, None, False, 0, cache, fmt, dc)
    return cache, R.decode_rows(raw.cpu().numpy(), fmt, dc, dr)


def make_q(B, S, Hq, d, seed):
    return torch.randn(B, S, Hq, d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def run_attn(dsa, q, cache, fmt, sel, block, sp, sm, dc, ws=None, lse=True):
    B, S, Hq, d = q.shape
    args = (B, S, Hq, dc, d - dc, sel.shape[-1])
    need = dsa.dsa_block_mla_attn_workspace_size(*args, block) if block else \
        dsa.dsa_sparse_mla_attn_q4_workspace_size(*args)
    if ws is None:
        ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((B, S, Hq, dc), float("nan"), dtype=torch.bfloat16, device="cuda")
    l = torch.full((B, S, Hq), float("nan"), device="cuda") if lse else None
    if block:
        dsa.dsa_block_mla_attn(q, cache, fmt, sel, block, sp, sm, dc, out, l, ws)
    else:
        dsa.dsa_sparse_mla_attn_q4(q, cache, sel, sp, sm, dc, out, l, ws)
    return out, l


def positions(sel, block, i):
    if block:
        return R.block_positions(sel, block, i)
    return [int(t) for t in sel if 0 <= t <= i]


def check(q, rows, sel, block, sp, sm, dc, out, lse):
    B, S, Hq, d = q.shape
    qd, o = q.double().cpu().numpy(), out.double().cpu().numpy()
    l = None if lse is None else lse.double().cpu().numpy()
    sel = sel.cpu().numpy()
    for b in range(B):
        for s in range(S):
            pos = positions(sel[b, s], block, sp + s)
            ro, rl = R.attend(qd[b, s], rows[b], pos, sm, dc)
            if not pos:
                assert not o[b, s].any(), (b, s)
                assert l is None or np.all(l[b, s] == -np.inf)
                continue
            c = rows[b][np.asarray(pos)]
            p = np.exp(sm * qd[b, s] @ c.T - rl[:, None])
            dz = 2 * abs(sm) * d * 2.0 ** -24 * (np.abs(qd[b, s]) @ np.abs(c).T).max(-1, keepdims=True)
            tol = (p @ np.abs(c[:, :dc])) * (2.0 ** -8 + 2 * dz + 2.0 ** -16) + np.abs(ro) * 2.0 ** -8
            err = np.abs(o[b, s] - ro)
            assert np.all(err <= tol), f"({b},{s}): {np.nanmax(err / np.maximum(tol, 1e-30)):.3g} x tolerance"
            if l is not None:
                assert np.all(np.abs(l[b, s] - rl) <= dz[:, 0] + 2.0 ** -18 + np.abs(rl) * 2.0 ** -23)


@pytest.mark.parametrize("B,S,Hq,dc,dr,t_max,k,sp,fill", [
    (2, 1, 128, 512, 64, 3000, 2048, 2999, 1.0),    # decode at the V3.2 sizes
    (1, 1, 128, 512, 64, 5000, 2048, 4999, 0.6),    # unfilled slots in any place
    (3, 1, 128, 512, 64, 300, 2048, 299, 1.0),      # fewer cached rows than slots
    (1, 4, 128, 512, 64, 2000, 512, 1500, 1.0),     # query rows with their own causal limits
    (2, 3, 128, 512, 64, 40, 16, 0, 1.0),           # the first positions of a sequence
    (1, 1, 128, 512, 64, 5000, 1, 4999, 1.0),       # one selected row
    (2, 1, 1, 512, 64, 900, 129, 899, 1.0),         # one head, one slot past a tile
    (2, 1, 16, 512, 64, 900, 127, 899, 1.0),
    (1, 2, 40, 512, 64, 900, 300, 800, 0.9),        # heads that fill no tile
    (1, 1, 80, 256, 32, 900, 256, 899, 1.0),
    (2, 1, 200, 128, 8, 500, 200, 499, 1.0),
    (1, 2, 64, 384, 40, 500, 200, 480, 1.0),
    (2, 1, 24, 128, 0, 500, 64, 499, 1.0),          # no rotary part
    (40, 1, 128, 512, 64, 500, 256, 499, 1.0),
    (1, 200, 16, 256, 64, 600, 150, 380, 1.0),      # more query rows than SMs
])
def test_q4_attention(dsa, B, S, Hq, dc, dr, t_max, k, sp, fill):
    q = make_q(B, S, Hq, dc + dr, B + S + k)
    cache, rows = make_cache(dsa, B, t_max, R.Q4, dc, dr, seed=k)
    idx = workloads.random_indices(B, S, k, t_max, sp, seed=k + Hq, fill=fill)
    sm = (dc + dr) ** -0.5
    out, lse = run_attn(dsa, q.cuda(), cache, R.Q4, idx.cuda(), 0, sp, sm, dc)
    assert dsa.dsa_get_device_error() == dsa.DSA_OK
    check(q, rows, idx, 0, sp, sm, dc, out, lse)


def block_lists(B, S, kb, block, sp, seed, fill=1.0):
    g = torch.Generator().manual_seed(seed)
    out = torch.full((B, S, kb), -1, dtype=torch.int32)
    for b in range(B):
        for s in range(S):
            avail = (sp + s + 1) // block
            m = int(round(fill * min(kb, avail)))
            out[b, s, torch.randperm(kb, generator=g)[:m]] = torch.randperm(avail, generator=g)[:m].int()
    return out


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B,S,Hq,dc,dr,t_max,kb,block,sp,fill", [
    (2, 1, 128, 512, 64, 3000, 16, 64, 2990, 1.0),
    (2, 1, 128, 512, 64, 3000, 32, 64, 2943, 1.0),      # the last token finishes a block: no tail
    (1, 1, 16, 512, 64, 3000, 16, 128, 2900, 0.5),      # unfilled slots in any place
    (1, 5, 128, 512, 64, 700, 4, 50, 640, 1.0),         # blocks that end inside a tile
    (2, 4, 24, 256, 32, 300, 40, 7, 290, 1.0),
    (1, 9, 64, 128, 8, 64, 3, 16, 0, 1.0),              # from the first token on
    (1, 3, 8, 384, 40, 300, 5, 1, 200, 1.0),            # blocks of one token: no tail ever
    (1, 2, 128, 512, 64, 4200, 1, 2048, 4100, 1.0),     # blocks longer than a tile
    (1, 1, 128, 512, 64, 300, 4, 1000, 299, 1.0),       # one unfinished block longer than the context
    (1, 160, 32, 128, 64, 800, 4, 32, 600, 1.0),        # more query rows than SMs
])
def test_block_attention(dsa, fmt, B, S, Hq, dc, dr, t_max, kb, block, sp, fill):
    q = make_q(B, S, Hq, dc + dr, B + S + kb)
    cache, rows = make_cache(dsa, B, t_max, fmt, dc, dr, seed=kb)
    blk = block_lists(B, S, kb, block, sp, seed=kb + Hq, fill=fill)
    sm = (dc + dr) ** -0.5
    out, lse = run_attn(dsa, q.cuda(), cache, fmt, blk.cuda(), block, sp, sm, dc)
    assert dsa.dsa_get_device_error() == dsa.DSA_OK
    check(q, rows, blk, block, sp, sm, dc, out, lse)


@pytest.mark.parametrize("fmt", FORMATS)
def test_block_lists_skip_unfinished_and_future_blocks(dsa, fmt):
    """Entries that are not finished for the query count as empty (its own block
    is attended once, as the tail); every query sees only its own past."""
    B, S, Hq, dc, dr, t_max, block, sp = 1, 20, 16, 512, 64, 200, 16, 60
    q = make_q(B, S, Hq, dc + dr, 5)
    cache, rows = make_cache(dsa, B, t_max, fmt, dc, dr, seed=6)
    blk = torch.arange(12, dtype=torch.int32).repeat(B, S, 1)         # every block of the cache
    blk[0, ::2, 3] = -1
    blk[0, 1::3, 11] = 1 << 27                                        # far past the cache
    out, lse = run_attn(dsa, q.cuda(), cache, fmt, blk.cuda(), block, sp, 0.04, dc)
    assert dsa.dsa_get_device_error() == dsa.DSA_OK
    check(q, rows, blk, block, sp, 0.04, dc, out, lse)


def test_no_finished_block_to_list(dsa):
    """The first tokens of a sequence: no block is finished, the list has no columns."""
    q = make_q(2, 5, 16, 576, 5)
    cache, rows = make_cache(dsa, 2, 40, R.Q4, 512, 64, seed=6)
    blk = torch.empty(2, 5, 0, dtype=torch.int32)
    out, lse = run_attn(dsa, q.cuda(), cache, R.Q4, blk.cuda(), 64, 3, 0.04, 512)
    check(q, rows, blk, 64, 3, 0.04, 512, out, lse)


def test_offsets_beyond_32_bits(dsa):
    """A 5 GB cache: rows, blocks and keys whose byte offsets pass 2^32, written, read and
    attended; the rows between are left alone."""
    B, dc, dr, t_max, S = 2, 512, 64, 6_000_000, 3
    cache = torch.empty(B, t_max, 416, dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(3)
    near = list(range(40)) + list(range(t_max - 200, t_max))
    kv = torch.randn(B, len(near), dc + dr, generator=g).to(torch.bfloat16).cuda()
    dsa.dsa_latent_prologue(kv[:, :40], None, 0.0, None, False, 0, cache, R.Q4, dc)
    dsa.dsa_latent_prologue(kv[:, 40:], None, 0.0, None, False, t_max - 200, cache, R.Q4, dc)
    rows = R.decode_rows(cache[:, near].cpu().numpy(), R.Q4, dc, dr)
    n, s = R.q4_groups(kv[..., :dc].double().cpu().numpy())
    assert np.array_equal(rows[..., :dc], R.bf16(n * np.repeat(s, 32, -1)))
    out = torch.empty(B, 200, dc + dr, device="cuda")
    dsa.dsa_latent_read(cache, R.Q4, t_max - 200, out, dc)
    assert np.array_equal(out.double().cpu().numpy(), rows[:, 40:])
    # positions: the last ones and the first ones, a sequence's rows renumbered for the check
    q = make_q(B, S, 32, dc + dr, 4)
    idx = torch.tensor([t_max - 1, t_max - 2, t_max - 3, 5, -1, t_max - 150, 39], dtype=torch.int32).repeat(B, S, 1)
    sp = t_max - S
    o, lse = run_attn(dsa, q.cuda(), cache, R.Q4, idx.cuda(), 0, sp, 0.04, dc)
    place = {t: i for i, t in enumerate(near)}
    local = torch.tensor([[[place[t] if 0 <= t <= sp + s else -1 for t in idx[b, s].tolist()] for s in range(S)]
                          for b in range(B)], dtype=torch.int32)
    check(q, rows, local, 0, 10 ** 6, 0.04, dc, o, lse)
    # blocks of 16: the last finished one and the second, and the unfinished one
    blk = torch.tensor([(t_max - S) // 16 - 1, 1], dtype=torch.int32).repeat(B, S, 1)
    o, lse = run_attn(dsa, q.cuda(), cache, R.Q4, blk.cuda(), 16, sp, 0.04, dc)
    local = torch.full((B, S, 64), -1, dtype=torch.int32)
    for b in range(B):
        for s in range(S):
            pos = R.block_positions(blk[b, s].tolist(), 16, sp + s)
            local[b, s, :len(pos)] = torch.tensor([place[t] for t in pos], dtype=torch.int32)
    check(q, rows, local, 0, 10 ** 6, 0.04, dc, o, lse)
    del cache
    # block keys at the end of a 4.4 GB key cache
    T, D, m = 17_200_000, 128, 64
    kc = torch.zeros(2, T, D, dtype=torch.uint8, device="cuda")
    ks = torch.zeros(2, T, device="cuda")
    kc[:, -128:] = torch.randint(0, 120, (2, 128, D), generator=g, dtype=torch.uint8).cuda()
    ks[:, -128:] = 0.01
    bc, bs = torch.zeros(2, T // m, D, dtype=torch.uint8, device="cuda"), torch.zeros(2, T // m, device="cuda")
    dsa.dsa_block_keys(kc, ks, T - 128, 128, m, bc, bs)
    want = np.stack([R.block_keys(kc[b, -128:].cpu().numpy(), ks[b, -128:].cpu().numpy(), m, D) for b in range(2)])
    got = R.E4M3[bc[:, -2:].cpu().numpy()] * bs[:, -2:, None].double().cpu().numpy()
    assert np.all(np.abs(got - want) <= np.abs(want) * 2.0 ** -4 + np.abs(want).max(-1, keepdims=True) * 2.0 ** -14)
    assert not bs[:, :-2].any()


def test_selections_of_more_entries_than_31_bits(dsa):
    """2^20 query rows of 2049 slots, a few of them filled, in the last ones too: the lists'
    offsets pass 2^31 entries."""
    S, k, dc, dr, sp = 1 << 20, 2049, 128, 0, 5000
    small, rows = make_cache(dsa, 1, 4096, R.Q4, dc, dr, seed=2)
    cache = torch.zeros(1, sp + S, small.shape[-1], dtype=torch.uint8, device="cuda")
    cache[:, :4096] = small
    q = torch.randn(1, S, 2, dc, dtype=torch.bfloat16, device="cuda")
    idx = torch.full((1, S, k), -1, dtype=torch.int32, device="cuda")
    s = torch.arange(S, device="cuda", dtype=torch.int32)
    for j, slot in enumerate((0, 1, 700, 2048)):
        idx[0, :, slot] = (s * (j + 3) + 1000 * j) % 1000 + 1000 * j
    out, lse = run_attn(dsa, q, cache, R.Q4, idx, 0, sp, 0.1, dc)
    for at in (0, (1 << 31) // k - 1, (1 << 31) // k, S - 3):
        check(q[:, at:at + 3], rows, idx[:, at:at + 3], 0, sp + at, 0.1, dc, out[:, at:at + 3], lse[:, at:at + 3])
    del idx, cache, q, out, lse
    torch.cuda.empty_cache()


def test_empty_rows(dsa):
    B, S, Hq, dc, dr, t_max, k = 3, 2, 128, 512, 64, 300, 300
    q = make_q(B, S, Hq, dc + dr, 1)
    cache, rows = make_cache(dsa, B, t_max, R.Q4, dc, dr, seed=2)
    idx = workloads.random_indices(B, S, k, t_max, 290, seed=3)
    idx[1] = -1                                                        # a sequence with nothing selected
    idx[2, 0] = 295                                                    # only future positions
    idx[0, 1, :] = -1
    idx[0, 1, 299] = 7                                                 # the last slot alone
    out, lse = run_attn(dsa, q.cuda(), cache, R.Q4, idx.cuda(), 0, 290, 0.04, dc)
    idx[2, 0] = -1
    check(q, rows, idx, 0, 290, 0.04, dc, out, lse)


def test_positions_past_the_cache_are_recorded(dsa):
    q = make_q(1, 1, 16, 576, 1).cuda()
    cache, rows = make_cache(dsa, 1, 50, R.Q4, 512, 64, seed=2)
    # start_pos + S <= t_max is checked on the host, so t > start_pos + s is only a future position
    idx = torch.tensor([[[0, 49, 50, 1 << 30, -5]]], dtype=torch.int32, device="cuda")
    out, lse = run_attn(dsa, q, cache, R.Q4, idx, 0, 49, 0.04, 512)
    assert dsa.dsa_get_device_error() == dsa.DSA_OK
    check(q, rows, torch.tensor([[[0, 49]]], dtype=torch.int32), 0, 49, 0.04, 512, out, lse)


def test_rows_outside_the_selection_are_not_read(dsa):
    """NaN in every cache row that is not selected, scales and rotary part included."""
    dc, dr, t_max, sp = 512, 64, 600, 599
    q = make_q(1, 1, 32, dc + dr, 1).cuda()
    for fmt in FORMATS:
        cache, rows = make_cache(dsa, 1, t_max, fmt, dc, dr, seed=2)
        blk = torch.tensor([[[3, -1, 7, 20]]], dtype=torch.int32)
        keep = R.block_positions([3, 7, 20], 16, sp)
        mask = torch.ones(t_max, dtype=torch.bool, device="cuda")
        mask[keep] = False
        cache.view(torch.uint8)[0, mask] = 0xFF                        # bf16, e4m3 and fp32 NaN
        out, lse = run_attn(dsa, q, cache, fmt, blk.cuda(), 16, sp, 0.04, dc)
        check(q, rows, blk, 16, sp, 0.04, dc, out, lse)


@pytest.mark.parametrize("scale", [2.0 ** 20, 2.0 ** -12])
def test_latents_of_any_scale(dsa, scale):
    """Values far outside fp16's range, and logits whose maxima differ by tens
    between tiles (a sharp softmax)."""
    dc, dr, t_max, k = 512, 64, 2500, 2048
    q = make_q(2, 1, 128, dc + dr, 1)
    cache, rows = make_cache(dsa, 2, t_max, R.Q4, dc, dr, seed=2, scale=scale)
    idx = workloads.random_indices(2, 1, k, t_max, t_max - 1, seed=3)
    sm = (dc + dr) ** -0.5 / scale * 20
    out, lse = run_attn(dsa, q.cuda(), cache, R.Q4, idx.cuda(), 0, t_max - 1, sm, dc)
    check(q, rows, idx, 0, t_max - 1, sm, dc, out, lse)


def test_growing_logits_move_the_running_maximum(dsa):
    """Each tile's largest logit is far above the one before, then falls again."""
    dc, dr, t_max = 512, 64, 1024
    g = torch.Generator().manual_seed(8)
    dirn = torch.randn(dc + dr, generator=g)
    gain = torch.cat((torch.linspace(-3, 3, 768), torch.linspace(3, -3, 256)))
    kv = torch.randn(1, t_max, dc + dr, generator=g) * 0.3 + gain[:, None] * dirn
    raw = torch.zeros(1, t_max, 416, dtype=torch.uint8, device="cuda")
    dsa.dsa_latent_prologue(kv.cuda(), None, 0.0, None, False, 0, raw, R.Q4, dc)
    rows = R.decode_rows(raw.cpu().numpy(), R.Q4, dc, dr)
    q = (dirn + 0.5 * torch.randn(1, 300, 64, dc + dr, generator=g)).to(torch.bfloat16)
    q[:, :, ::2] *= -1
    idx = torch.arange(t_max, dtype=torch.int32).repeat(1, 300, 1)
    # 300 query rows: one CTA walks all eight tiles of a row
    out, lse = run_attn(dsa, q.cuda(), raw, R.Q4, idx.cuda(), 0, t_max - 300, 0.1, dc)
    sub = torch.arange(0, 300, 37)
    check(q[:, :1], rows, idx[:, :1], 0, t_max - 300, 0.1, dc, out[:, :1], lse[:, :1])
    for s in sub.tolist():
        check(q[:, s:s + 1], rows, idx[:, s:s + 1], 0, t_max - 300 + s, 0.1, dc, out[:, s:s + 1], lse[:, s:s + 1])


@pytest.mark.parametrize("shift", [-3000.0, -200.0, 200.0])
def test_first_tiles_with_nothing_selected_and_logits_far_from_zero(dsa, shift):
    """The first 128-slot tiles hold no valid slot; the logits that follow are far from zero, so
    a reference of zero would lose them all (or overflow)."""
    dc, dr, t_max, k = 512, 64, 600, 512
    g = torch.Generator().manual_seed(5)
    dirn = torch.randn(dc + dr, generator=g)
    kv = torch.randn(1, t_max, dc + dr, generator=g) * 0.2 + dirn
    raw = torch.zeros(1, t_max, 416, dtype=torch.uint8, device="cuda")
    dsa.dsa_latent_prologue(kv.cuda(), None, 0.0, None, False, 0, raw, R.Q4, dc)
    rows = R.decode_rows(raw.cpu().numpy(), R.Q4, dc, dr)
    for S in (1, 200):                                   # one tile a CTA, and every tile in one CTA
        q = (dirn + 0.05 * torch.randn(1, S, 64, dc + dr, generator=g)).to(torch.bfloat16)
        sm = shift / float(dirn @ dirn)
        idx = torch.full((1, S, k), -1, dtype=torch.int32)
        idx[:, :, 300:] = torch.arange(k - 300, dtype=torch.int32)
        out, lse = run_attn(dsa, q.cuda(), raw, R.Q4, idx.cuda(), 0, t_max - S, sm, dc)
        for s in range(0, S, 50):
            check(q[:, s:s + 1], rows, idx[:, s:s + 1], 0, t_max - S + s, sm, dc,
                  out[:, s:s + 1], lse[:, s:s + 1])


@pytest.mark.parametrize("power", [0, 10, 60, 110, 124])
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("S", [1, 200])                 # one tile a CTA, and every tile in one CTA
def test_equal_logits_as_far_from_zero_as_fp32_goes(dsa, S, sign, power):
    """Every selected row has the same logit, sign * 7 * 2^power, exactly (one nonzero column of
    q, a power of two, against a 4-bit value without rounding), after 128-slot tiles that hold
    no valid slot: the weights are equal whatever the logit is, the output is the mean.  Sums of
    up to 512 fp32 terms and the two roundings of the weights and the output."""
    dc, dr, t_max, k, n = 512, 64, 700, 512, 212
    kv = torch.randn(1, t_max, dc + dr, generator=torch.Generator().manual_seed(power))
    kv[..., :32] = 0
    kv[..., 5] = sign * 7 * 2.0 ** (power // 2)
    raw = torch.zeros(1, t_max, 416, dtype=torch.uint8, device="cuda")
    dsa.dsa_latent_prologue(kv.cuda(), None, 0.0, None, False, 0, raw, R.Q4, dc)
    rows = R.decode_rows(raw.cpu().numpy(), R.Q4, dc, dr)
    assert np.all(rows[..., 5] == sign * 7 * 2.0 ** (power // 2))
    q = torch.zeros(1, S, 24, dc + dr, dtype=torch.bfloat16, device="cuda")
    q[..., 5] = 2.0 ** (power - power // 2)
    idx = torch.full((1, S, k), -1, dtype=torch.int32)
    idx[:, :, k - n:] = torch.randperm(t_max - S, generator=torch.Generator().manual_seed(1))[:n].sort().values.int()
    out, lse = run_attn(dsa, q, raw, R.Q4, idx.cuda(), 0, t_max - S, 1.0, dc)
    sel = rows[0, idx[0, 0, k - n:].numpy()][:, 32:dc]
    got, want = out[..., 32:].double().cpu().numpy(), sel.mean(0)
    assert np.all(np.abs(got - want) <= np.abs(want) * 2.0 ** -8 + np.abs(sel).mean(0) * (512 * 2.0 ** -24))
    z = sign * 7 * 2.0 ** power
    assert np.all(np.abs(lse.double().cpu().numpy() - (z + np.log(n))) <= abs(z) * 2.0 ** -22 + 2.0 ** -18)


@pytest.mark.parametrize("sm", [0.0, 1e-30, 1e30, -1e30])
@pytest.mark.parametrize("S", [1, 200])
def test_scales_far_from_one(dsa, S, sm):
    """A scale of zero (or nothing) weighs all selected rows alike; a huge one leaves the row with
    the largest logit, or the smallest where it is negative (whole numbers, so that logits are
    exact and far apart once scaled), its share the other rows with that logit have too."""
    dc, dr, t_max, k = 256, 8, 700, 400
    g = torch.Generator().manual_seed(4)
    kv = torch.randint(-7, 8, (1, t_max, dc + dr), generator=g).float()
    kv[..., 0:dc:32] = 7                                 # (a 4-bit step of one)
    raw = torch.zeros(1, t_max, R.row_bytes(R.Q4, dc, dr), dtype=torch.uint8, device="cuda")
    dsa.dsa_latent_prologue(kv.cuda(), None, 0.0, None, False, 0, raw, R.Q4, dc)
    rows = R.decode_rows(raw.cpu().numpy(), R.Q4, dc, dr)
    assert np.array_equal(rows, kv.double().numpy())
    q = torch.randint(-3, 4, (1, S, 20, dc + dr), generator=g).to(torch.bfloat16)
    idx = torch.full((1, S, k), -1, dtype=torch.int32)
    idx[:, :, 140:] = torch.randperm(t_max - S, generator=g)[:k - 140].int()
    out, lse = run_attn(dsa, q.cuda(), raw, R.Q4, idx.cuda(), 0, t_max - S, sm, dc)
    z = np.einsum("shd,td->sht", q[0].double().numpy(), rows[0, idx[0, 0, 140:].numpy()])
    p = np.ones_like(z) if abs(sm) < 1 else (z == (z.max(-1, keepdims=True) if sm > 0 else z.min(-1, keepdims=True)))
    p = p / p.sum(-1, keepdims=True)
    sel = rows[0, idx[0, 0, 140:].numpy(), :dc]
    got, want = out[0].double().cpu().numpy(), p @ sel
    # the weights are 1 or 0: the rounding of the output, and the fp32 sums and quotient
    assert np.all(np.abs(got - want) <= np.abs(want) * 2.0 ** -8 + (p @ np.abs(sel)) * (400 * 2.0 ** -24))
    if abs(sm) < 1:
        assert np.all(np.abs(lse[0].double().cpu().numpy() - np.log(k - 140)) <= 2.0 ** -18)


@pytest.mark.parametrize("S", [1, 200])                 # split over CTAs, and one CTA a row
def test_nan_stays_where_it_belongs(dsa, S):
    """A NaN in one head's query makes that head NaN, in a selected row every head of that
    query; a NaN logit among finite ones is not lost in the merge of the splits."""
    t_max, k = 1200, 1000
    q = make_q(1, S, 32, 576, 1)
    cache, rows = make_cache(dsa, 1, t_max, R.BF16, 512, 64, seed=2)
    blk = torch.arange(60, dtype=torch.int32).repeat(1, S, 1)
    sp = t_max - S
    q[0, 0, 5, 17] = float("nan")
    out, lse = run_attn(dsa, q.cuda(), cache, R.BF16, blk.cuda(), 16, sp, 0.04, 512)
    assert out[0, 0, 5].isnan().all() and lse[0, 0, 5].isnan()
    keep = [h for h in range(32) if h != 5]
    assert not out[0, 0, keep].isnan().any() and not lse[0, 0, keep].isnan().any()
    check(q[:, -1:] if S > 1 else q[:, :, :5], rows, blk[:, -1:], 16, sp + S - 1, 0.04, 512,
          out[:, -1:] if S > 1 else out[:, :, :5], lse[:, -1:] if S > 1 else lse[:, :, :5])
    cache[0, 700, 3] = float("nan")                      # in one share only
    out, lse = run_attn(dsa, make_q(1, S, 32, 576, 1).cuda(), cache, R.BF16, blk.cuda(), 16, sp, 0.04, 512)
    assert out[..., 3].isnan().all() and lse.isnan().all()


def test_no_lse_and_repeat_is_bitwise_equal(dsa):
    q = make_q(4, 1, 128, 576, 1).cuda()
    cache, _ = make_cache(dsa, 4, 3000, R.Q4, 512, 64, seed=2)
    idx = workloads.random_indices(4, 1, 2048, 3000, 2999, seed=3).cuda()
    a, lse = run_attn(dsa, q, cache, R.Q4, idx, 0, 2999, 0.04, 512)
    for _ in range(5):
        b, none = run_attn(dsa, q, cache, R.Q4, idx, 0, 2999, 0.04, 512, lse=False)
        assert none is None and torch.equal(a, b)


def test_two_streams_with_their_own_workspaces_and_a_graph(dsa):
    cache, _ = make_cache(dsa, 4, 3000, R.Q4, 512, 64, seed=2)
    idx = workloads.random_indices(4, 1, 2048, 3000, 2999, seed=3).cuda()
    qs = [make_q(4, 1, 128, 576, 10 + i).cuda() for i in range(2)]
    want = [run_attn(dsa, q, cache, R.Q4, idx, 0, 2999, 0.04, 512)[0] for q in qs]
    need = max(1, dsa.dsa_sparse_mla_attn_q4_workspace_size(4, 1, 128, 512, 64, 2048))
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in qs]
    outs = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for q, w, o, st in zip(qs, ws, outs, streams):
            dsa.dsa_sparse_mla_attn_q4(q, cache, idx, 2999, 0.04, 512, o, None, w, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    o = torch.zeros_like(want[0])
    qg = qs[0].clone()
    with torch.cuda.graph(graph):
        dsa.dsa_sparse_mla_attn_q4(qg, cache, idx, 2999, 0.04, 512, o, None, ws[0])
    graph.replay()
    assert torch.equal(o, want[0])
    qg.copy_(qs[1])
    graph.replay()
    assert torch.equal(o, want[1])


def test_binding_refuses_wrong_tensors(dsa):
    q = make_q(2, 1, 16, 576, 1).cuda()
    cache, _ = make_cache(dsa, 2, 300, R.Q4, 512, 64, seed=2)
    idx = torch.zeros(2, 1, 8, dtype=torch.int32, device="cuda")
    out = torch.empty(2, 1, 16, 512, dtype=torch.bfloat16, device="cuda")
    ok = dict(q=q, kv_q4=cache, idx=idx, start_pos=299, sm_scale=0.04, dc=512, out=out, lse=None, workspace=None)
    for bad in (dict(q=q.float()), dict(kv_q4=cache[:1].contiguous()), dict(kv_q4=cache[..., :-16].contiguous()),
                dict(idx=idx.long()), dict(idx=idx[:1].contiguous()), dict(out=out.float()),
                dict(out=out[:, :, :8].contiguous()), dict(lse=torch.empty(2, 16, device="cuda")),
                dict(idx=idx.cpu()), dict(q=q.transpose(0, 2).contiguous().transpose(0, 2))):
        with pytest.raises(ValueError):
            dsa.dsa_sparse_mla_attn_q4(**{**ok, **bad})


# ------------------------------------------------------------------ block keys
@pytest.mark.parametrize("B,t_max,D,block,start,S", [
    (2, 1000, 128, 64, 0, 1000), (3, 1000, 64, 16, 5, 900), (2, 400, 128, 7, 13, 300), (1, 300, 128, 1, 0, 300),
    (4, 256, 128, 64, 191, 1),           # one token finishes a block
    (4, 256, 128, 64, 192, 1),           # one token finishes none
    (1, 5000, 64, 2048, 100, 4500), (2, 64, 128, 3, 0, 64),
])
def test_block_keys(dsa, B, t_max, D, block, start, S):
    """The mean's fp32 sum is off by block * 2^-24 of the mean magnitude; a code may then
    differ from the exact one's by one e4m3 step where that is at a border."""
    g = torch.Generator().manual_seed(D + block)
    keys = torch.randn(B, t_max, D, generator=g).cuda()
    kc = torch.empty(B, t_max, D, dtype=torch.uint8, device="cuda")
    ks = torch.empty(B, t_max, device="cuda")
    dsa.dsa_indexer_quant(keys, kc, ks)
    n_max = t_max // block + 2
    bc = torch.full((B, n_max, D), 0x5A, dtype=torch.uint8, device="cuda")
    bs = torch.full((B, n_max), -3.0, device="cuda")
    dsa.dsa_block_keys(kc, ks, start, S, block, bc, bs)
    first, last = start // block, (start + S) // block
    c, s = bc.cpu().numpy(), bs.cpu().numpy().astype(np.float64)
    assert np.all(c[:, :first] == 0x5A) and np.all(c[:, last:] == 0x5A)
    assert np.all(s[:, :first] == -3) and np.all(s[:, last:] == -3)
    for b in range(B):
        ref = R.block_keys(kc[b].cpu().numpy(), ks[b].cpu().numpy(), block, D)[first:last]
        if not len(ref):
            continue
        mag = R.block_keys(kc[b].cpu().numpy() & 0x7F, ks[b].cpu().numpy(), block, D)[first:last]
        amax = np.maximum(np.abs(ref).max(-1), 1e-4)
        off = (mag.max(-1) * (block + 2) * 2.0 ** -24)[:, None]
        assert np.all(np.abs(s[b, first:last] - amax / 448) <= amax / 448 * 2.0 ** -22 + off[:, 0] / 448)
        got = R.E4M3[c[b, first:last]] * s[b, first:last][:, None]
        tol = np.maximum(np.abs(ref) * 2.0 ** -4, (amax / 448)[:, None] * 2.0 ** -10) * (1 + 2.0 ** -10) + 2 * off
        assert np.all(np.abs(got - ref) <= tol)


def test_block_keys_do_not_depend_on_how_the_tokens_arrive(dsa):
    B, T, D, block = 2, 500, 128, 48
    kc = torch.randint(0, 127, (B, T, D), generator=torch.Generator().manual_seed(1), dtype=torch.uint8).cuda()
    ks = torch.rand(B, T, generator=torch.Generator().manual_seed(2)).cuda()
    def empty():
        return (torch.zeros(B, 11, D, dtype=torch.uint8, device="cuda"), torch.zeros(B, 11, device="cuda"))
    whole, steps = empty(), empty()
    dsa.dsa_block_keys(kc, ks, 0, T, block, *whole)
    t = 0
    for n in (100, 1, 1, 42, 1, 200, 155):
        dsa.dsa_block_keys(kc, ks, t, n, block, *steps)
        t += n
    assert t == T and torch.equal(whole[0], steps[0]) and torch.equal(whole[1], steps[1])


def exact_codes(mean, scale):
    """Values of the e4m3 codes nearest to mean / scale (ties to even), and which quotients lie
    within 2^-40 of a border between two codes (beyond what 64-bit sums can tell)."""
    q = mean / scale
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(q), 2.0 ** -30))), -6) - 3)
    n = q / step
    near = np.abs(np.abs(n - np.floor(n)) - 0.5) < np.maximum(np.abs(n), 1) * 2.0 ** -40
    return np.clip(np.rint(n) * step, -448, 448), near


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("block", [4, 16, 64, 130, 512])
@pytest.mark.parametrize("eps", [None, 1e-2, 1e-3, 1e-4, 0.0])
def test_block_keys_of_tokens_that_cancel(dsa, D, block, eps):
    """Pairs of tokens of opposite sign whose scales differ by a relative eps: the mean is eps of
    its terms (eps 0: none is left; None: ordinary keys).  Codes are those of the 64-bit mean; a
    term's product is exact in 64 bits and a sum of 512 off by at most 512 * 2^-53 of its
    largest terms, 2^-30 of the mean at eps 1e-4, so that far fewer dims than one in a run are
    within that of a border: a dim that is may differ."""
    n = 120 if block < 100 else 24
    g = torch.Generator().manual_seed(block + D)
    kc = torch.randint(0, 127, (1, n * block, D), generator=g, dtype=torch.uint8)
    ks = torch.rand(1, n * block, generator=g) + 0.5
    if eps is None:
        kc |= torch.randint(0, 2, kc.shape, generator=g, dtype=torch.uint8) << 7
    else:
        kc[:, 1::2] = kc[:, ::2] | 0x80
        ks[:, 1::2] = ks[:, ::2] * (1 + eps)
    kc[0, -block:] = 0                                   # a block of zeros
    kc[0, -3 * block:-2 * block] &= 0x80                 # and of zeros of either sign
    ks[0, -5 * block:-4 * block] *= 1e-9                 # and one under the scale's floor
    bc, bs = torch.zeros(1, n, D, dtype=torch.uint8, device="cuda"), torch.zeros(1, n, device="cuda")
    dsa.dsa_block_keys(kc.cuda(), ks.cuda(), 0, n * block, block, bc, bs)
    k = (R.E4M3[kc[0].numpy()] * ks[0].double().numpy()[:, None]).astype(np.longdouble)
    mean = k.reshape(n, block, D).sum(1).astype(np.float64) / block
    scale = np.maximum(np.abs(mean).max(-1), np.float64(np.float32(1e-4))) / 448
    got_s = bs[0].double().cpu().numpy()
    assert np.all(np.abs(got_s - scale) <= scale * 2.0 ** -14)
    want, near = exact_codes(mean, scale[:, None])
    if eps == 1e-4:
        near |= np.abs(exact_codes(mean * (1 + 2.0 ** -30), scale[:, None])[0] -
                       exact_codes(mean * (1 - 2.0 ** -30), scale[:, None])[0]) > 0
    assert near.mean() < 1e-3 or block <= 16
    assert np.all((R.E4M3[bc[0].cpu().numpy()] == want) | near)


def test_block_keys_keep_nan_and_sums_past_fp32(dsa):
    """A NaN code makes its dim NaN and no other; terms whose fp32 sum would pass the type's
    range keep their mean."""
    D, block = 128, 16
    kc = torch.randint(0, 126, (1, 3 * block, D), generator=torch.Generator().manual_seed(3), dtype=torch.uint8)
    ks = torch.full((1, 3 * block), 0.5)
    kc[0, 5, 77] = 0xFF
    ks[0, block:2 * block] = 7e35                        # 448 * 7e35 = 3.1e38, times 16
    bc, bs = torch.zeros(1, 3, D, dtype=torch.uint8, device="cuda"), torch.zeros(1, 3, device="cuda")
    dsa.dsa_block_keys(kc.cuda(), ks.cuda(), 0, 3 * block, block, bc, bs)
    got = R.E4M3[bc[0].cpu().numpy()]
    assert np.isnan(got[0, 77])
    mean = (R.E4M3[kc[0].numpy()] * ks[0].double().numpy()[:, None]).reshape(3, block, D).mean(1)
    scale = np.nanmax(np.abs(mean), -1) / 448
    assert np.all(np.abs(bs[0].double().cpu().numpy() - scale) <= scale * 2.0 ** -14)
    want, near = exact_codes(np.nan_to_num(mean), scale[:, None])
    ok = (got == want) | near
    ok[0, 77] = True
    assert ok.all()


# ------------------------------------------------------------ operators together
def test_decode_step_over_the_4_bit_cache(dsa):
    """dsa_decode_step with a 4-bit latent cache whose newest row the prologue wrote: the
    selection is that of the bf16 cache's step, the attention that of the rows."""
    wl = workloads.WORKLOADS[1]
    T, B, topk = 3000, 2, 512
    dc, dr = wl.dc, wl.dr
    seqs = [workloads.decode_sequence(wl, b, T=T) for b in range(B)]
    kv = torch.stack([s["kv"] for s in seqs]).cuda()
    cache = torch.zeros(B, T, dsa.dsa_latent_q4_row_bytes(dc, dr), dtype=torch.uint8, device="cuda")
    dsa.dsa_latent_prologue(kv[:, :T - 1], None, 0.0, None, False, 0, cache, R.Q4, dc)
    k_cache = torch.zeros(B, T, wl.D, dtype=torch.uint8, device="cuda")
    k_scale = torch.zeros(B, T, device="cuda")
    for b, s in enumerate(seqs):
        dsa.dsa_indexer_quant(s["keys"][:T - 1].cuda(), k_cache[b], k_scale[b])
    q_idx, w, q_mla = (torch.stack([s[n] for s in seqs]).cuda() for n in ("q_idx", "w", "q_mla"))
    k_new = torch.stack([s["keys"][T - 1] for s in seqs]).cuda()

    def step(rows, dt, fn=None):
        idx = torch.empty(B, topk, dtype=torch.int32, device="cuda")
        out = torch.empty(B, wl.Hq, dc, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(B, wl.Hq, device="cuda")
        args = (q_idx, w, k_new, k_cache, k_scale, rows, q_mla, T, topk, wl.softmax_scale_idx, wl.sm_scale,
                idx, out, lse)
        if fn:
            fn(*args)
            return idx, out, lse
        need = dsa.dsa_decode_step_workspace_size(B, wl.H, wl.D, T, topk, wl.Hq, dc, dr, dt)
        dsa.dsa_decode_step(*args, torch.empty(need, dtype=torch.uint8, device="cuda"))
        return idx, out, lse

    dsa.dsa_latent_prologue(kv[:, T - 1:], None, 0.0, None, False, T - 1, cache, R.Q4, dc)
    idx, out, lse = step(cache, dsa.DSA_Q4_LATENT)
    ref_idx = step(kv, dsa.DSA_BF16)[0]
    assert torch.equal(idx, ref_idx)
    rows = R.decode_rows(cache.cpu().numpy(), R.Q4, dc, dr)
    check(q_mla[:, None], rows, idx[:, None], 0, T - 1, wl.sm_scale, dc, out[:, None], lse[:, None])
    idx2, out2, lse2 = step(cache, dsa.DSA_Q4_LATENT, dsa.dsa_decode_step_noalloc)
    assert torch.equal(idx2, idx) and torch.equal(out2, out) and torch.equal(lse2, lse)
    assert dsa.dsa_get_device_error() == dsa.DSA_OK


@pytest.mark.parametrize("fmt", FORMATS)
def test_block_selected_chunk_and_decode(dsa, fmt):
    """The whole path as a server runs it, a prefill chunk and then single tokens: latents and
    indexer keys appended, block keys of the finished blocks, scores over block keys, top-k of
    blocks, attention over the selected blocks.  Each stage is checked from the values that the
    stage before left."""
    B, H, D, Hq, dc, dr, block, kb, t_max = 2, 8, 128, 16, 512, 64, 16, 5, 400
    g = torch.Generator().manual_seed(77)
    raw = torch.zeros(B, t_max, R.row_bytes(fmt, dc, dr), dtype=torch.uint8, device="cuda")
    cache = raw.view(torch.bfloat16) if fmt == R.BF16 else raw
    kc, ks = torch.zeros(B, t_max, D, dtype=torch.uint8, device="cuda"), torch.zeros(B, t_max, device="cuda")
    n_max = t_max // block
    bc, bs = torch.zeros(B, n_max, D, dtype=torch.uint8, device="cuda"), torch.zeros(B, n_max, device="cuda")
    w_norm = (1 + 0.1 * torch.randn(dc, generator=g)).cuda()
    sm = (dc + dr) ** -0.5
    pos = 0
    for S in (150, 1, 1, 9, 1, 1):
        cs = torch.randn(S, dr // 2, 2, generator=g)
        cs = (cs / cs.norm(dim=-1, keepdim=True)).cuda()
        ics = cs.clone()
        q_i = torch.randn(B, S, H, D, generator=g).cuda()
        k_i = torch.randn(B, S, D, generator=g).cuda()
        wts = torch.randn(B, S, H, generator=g).cuda()
        kv = torch.randn(B, S, dc + dr, generator=g).to(torch.bfloat16).cuda()
        q = make_q(B, S, Hq, dc + dr, S + pos).cuda()
        qf, qs = torch.empty(B, S, H, D, dtype=torch.uint8, device="cuda"), torch.empty(B, S, H, device="cuda")
        dsa.dsa_indexer_prologue(q_i, k_i, ics, pos, qf, qs, kc, ks)
        dsa.dsa_latent_prologue(kv, w_norm, 1e-6, cs, True, pos, cache, fmt, dc)
        dsa.dsa_block_keys(kc, ks, pos, S, block, bc, bs)
        T = (pos + S) // block
        scores = torch.empty(B, S, T, device="cuda")
        dsa.dsa_index_scores_csa(qf, qs, wts, bc, bs, pos, T, block, D ** -0.5, scores)
        K = min(kb, T)
        blk = torch.empty(B, S, K, dtype=torch.int32, device="cuda")
        ws = torch.empty(max(1, dsa.dsa_topk_select_workspace_size(B, S, T, kb)), dtype=torch.uint8, device="cuda")
        dsa.dsa_topk_select_csa(scores, pos, block, kb, blk, ws)
        out, lse = run_attn(dsa, q, cache, fmt, blk, block, pos, sm, dc)
        assert dsa.dsa_get_device_error() == dsa.DSA_OK
        # the selected blocks score highest among the query's finished ones
        sc, sel = scores.cpu().numpy(), blk.cpu().numpy()
        for b in range(B):
            for s in range(S):
                avail = (pos + s + 1) // block
                got = sel[b, s][sel[b, s] >= 0]
                assert len(got) == min(K, avail)
                rest = np.setdiff1d(np.arange(avail), got)
                assert not len(rest) or not len(got) or sc[b, s, got].min() >= sc[b, s, rest].max()
        rows = R.decode_rows(raw.cpu().numpy(), fmt, dc, dr)
        check(q, rows, blk, block, pos, sm, dc, out, lse)
        pos += S
    # the block keys are the means of all that was appended
    want = np.stack([R.block_keys(kc[b].cpu().numpy(), ks[b].cpu().numpy(), block, D) for b in range(B)])[:, :pos // block]
    got = (R.E4M3[bc.cpu().numpy()] * bs.cpu().numpy()[..., None])[:, :pos // block]
    amax = np.abs(want).max(-1, keepdims=True)
    assert np.all(np.abs(got - want) <= np.abs(want) * 2.0 ** -4 + amax * 2.0 ** -14)
