"""dsa_latent_prologue and dsa_latent_read against the 64-bit reference.

Tolerances.  Without a norm and without a rotation every step before the one
rounding is exact, so bytes must be equal (for an fp32 input the 4-bit quotient
is a single-precision one: a code may differ where the exact quotient lies
within 2^-22 of a border).  With a norm the fp32 chain (512 products summed,
square root, reciprocal, two products) is off by at most 2^-18 relative; with a
rotation by 2^-22 of the pair's length.  A code may then differ by one step only
where the exact quotient is that close to a border, a scale only where the exact
scale is that close to one; every decoded value must be within half a step of
the exact one, plus what the scale's own rounding moves the largest codes."""
import numpy as np
import pytest
import torch

import latent_reference as R

pytestmark = pytest.mark.gpu
SHAPES = [(512, 64), (256, 32), (128, 8), (384, 40), (128, 0)]


@pytest.fixture(scope="module")
def dsa():
    import top_kv_selection_b200 as m
    return m


def new_cache(B, t_max, fmt, dc, dr, fill=0x5A):
    rb = R.row_bytes(fmt, dc, dr)
    raw = torch.full((B, t_max, rb), fill, dtype=torch.uint8, device="cuda")
    return raw.view(torch.bfloat16) if fmt == R.BF16 else raw


def to_bytes(cache):
    return cache.view(torch.uint8).cpu().numpy()


def make_kv(B, S, dc, dr, dtype, seed, spread=True):
    g = torch.Generator().manual_seed(seed)
    kv = torch.randn(B, S, dc + dr, generator=g)
    if spread:
        kv = kv * torch.exp2(torch.randint(-8, 8, (B, S, 1), generator=g).float())
    return kv.to(dtype)


@pytest.mark.parametrize("fmt", [R.BF16, R.FP8, R.Q4])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dc,dr", SHAPES)
def test_append_without_norm_is_the_rounding_alone(dsa, fmt, dtype, dc, dr):
    B, S, t_max, start = 3, 37, 60, 11
    kv = make_kv(B, S, dc, dr, dtype, dc + dr + fmt)
    kv[0, 0] = 0                                        # a row of zeros: the smallest scale
    kv[1, 2, :32] = 0
    cache = new_cache(B, t_max, fmt, dc, dr)
    dsa.dsa_latent_prologue(kv.cuda(), None, 0.0, None, False, start, cache, fmt, dc)
    raw = to_bytes(cache)
    assert np.all(raw[:, :start] == 0x5A) and np.all(raw[:, start + S:] == 0x5A)
    rows = raw[:, start:start + S]
    x = kv.double().numpy()
    if fmt == R.BF16:
        assert np.array_equal(R.decode_rows(rows, fmt, dc, dr), R.bf16(x))
        return
    assert np.array_equal(R.decode_rows(rows, fmt, dc, dr)[..., dc:], R.bf16(x[..., dc:]))
    if fmt == R.FP8:                                    # the rounding of dsa_latent_quant, byte for byte
        ref = torch.empty(B, S, R.row_bytes(fmt, dc, dr), dtype=torch.uint8, device="cuda")
        dsa.dsa_latent_quant(kv.cuda(), ref, dc)
        assert np.array_equal(rows, ref.cpu().numpy())
        return
    n, s = R.q4_groups(x[..., :dc])
    at = dc // 2 + 2 * dr
    got_s = R._u16_as_bf16(rows[..., at:at + dc // 16:2], rows[..., at + 1:at + dc // 16:2])
    assert np.array_equal(got_s, s)
    assert not rows[..., at + dc // 16:].any()          # the row's end is zero
    got = R.decode_rows(rows, fmt, dc, dr)[..., :dc]
    step = np.repeat(s, 32, -1)
    bad = got != R.bf16(n * step)
    quot = x[..., :dc] / step
    near = np.abs(np.abs(quot - np.floor(quot)) - 0.5) < 2.0 ** -22
    assert not (bad & ~near).any()
    if dtype == torch.bfloat16:
        assert not bad.any()


@pytest.mark.parametrize("fmt", [R.BF16, R.FP8, R.Q4])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dc,dr,norm,rope", [(512, 64, True, "pairs"), (512, 64, True, "halves"),
                                             (512, 64, False, "pairs"), (256, 32, True, None),
                                             (384, 40, True, "halves"), (128, 8, True, "pairs")])
def test_append_with_norm_and_rotation(dsa, fmt, dtype, dc, dr, norm, rope):
    B, S, start = 2, 41, 5
    kv = make_kv(B, S, dc, dr, dtype, dc + fmt + S)
    g = torch.Generator().manual_seed(4)
    w = 1 + 0.2 * torch.randn(dc, generator=g) if norm else None
    cs = None
    if rope:
        a = torch.rand(S, dr // 2, generator=g, dtype=torch.float64) * 6.28
        cs = torch.stack((a.cos(), a.sin()), -1).float()
    cache = new_cache(B, S + start + 3, fmt, dc, dr)
    cuda = lambda t: None if t is None else t.cuda()
    dsa.dsa_latent_prologue(kv.cuda(), cuda(w), 1e-6, cuda(cs), rope == "pairs", start, cache, fmt, dc)
    raw = to_bytes(cache)
    assert np.all(raw[:, :start] == 0x5A) and np.all(raw[:, start + S:] == 0x5A)
    got = R.decode_rows(raw[:, start:start + S], fmt, dc, dr)
    ref = R.prologue(kv.double().numpy(), None if w is None else w.double().numpy(), 1e-6,
                     None if cs is None else cs.double().numpy(), rope == "pairs", dc)
    pe, rp = got[..., dc:], ref[..., dc:]
    length = np.abs(kv.double().numpy()[..., dc:]).max(-1, keepdims=True) * 2
    assert np.all(np.abs(pe - rp) <= np.abs(rp) * 2.0 ** -8 + length * 2.0 ** -22)
    c, rc = got[..., :dc], ref[..., :dc]
    rel = 2.0 ** -18
    if fmt == R.BF16:
        assert np.all(np.abs(c - rc) <= np.abs(rc) * (2.0 ** -8 + rel))
        return
    group = 32 if fmt == R.Q4 else 128
    amax = np.repeat(np.abs(rc.reshape(B, S, -1, group)).max(-1), group, -1)
    if fmt == R.Q4:
        # half a step, the scale's rounding on a code of up to 7 steps, the decoded value's rounding
        tol = amax / 7 * (0.5 + 7 * 2.0 ** -8 + 8 * rel) + np.abs(rc) * 2.0 ** -7
        n, s = R.q4_groups(rc)
        same = R.bf16(n * np.repeat(s, 32, -1)) == c
        assert same.mean() > 0.999                     # borders are that rare
    else:
        tol = np.maximum(np.abs(rc) * 2.0 ** -4, amax / 448 * 2.0 ** -10) * (1 + 2.0 ** -10) + \
            np.abs(rc) * 2.0 ** -7 + amax * rel
    assert np.all(np.abs(c - rc) <= tol)


@pytest.mark.parametrize("S", [1, 5])
def test_append_takes_strided_projections(dsa, S):
    """kv as a slice of a wider projection's output, batch-first or token-first."""
    B, dc, dr, t_max = 4, 512, 64, 9
    wide = torch.randn(B, S, 1536 + dc + dr, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    for kv in (wide[..., 1536:], wide.transpose(0, 1).contiguous().transpose(0, 1)[..., 1536:]):
        a, b = new_cache(B, t_max, R.Q4, dc, dr), new_cache(B, t_max, R.Q4, dc, dr)
        dsa.dsa_latent_prologue(kv, None, 0.0, None, False, 2, a, R.Q4, dc)
        dsa.dsa_latent_prologue(kv.contiguous(), None, 0.0, None, False, 2, b, R.Q4, dc)
        assert torch.equal(a, b)
    with pytest.raises(dsa.DSAError):                   # a slice that does not start on 16 bytes
        dsa.dsa_latent_prologue(wide[..., 1535:-1], None, 0.0, None, False, 2, a, R.Q4, dc)
    with pytest.raises(ValueError):
        dsa.dsa_latent_prologue(kv.transpose(1, 2).contiguous().transpose(1, 2), None, 0.0, None, False, 2, a, R.Q4, dc) \
            if S > 1 else dsa.dsa_latent_prologue(kv, None, 0.0, None, False, 2, a[:3], R.Q4, dc)


@pytest.mark.parametrize("fmt", [R.BF16, R.FP8, R.Q4])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dc,dr", SHAPES)
def test_read_back(dsa, fmt, dtype, dc, dr):
    B, t_max = 3, 71
    cache = new_cache(B, t_max, fmt, dc, dr)
    dsa.dsa_latent_prologue(make_kv(B, t_max, dc, dr, torch.float32, 9).cuda(), None, 0.0, None, False, 0,
                            cache, fmt, dc)
    ref = R.decode_rows(to_bytes(cache), fmt, dc, dr)
    for start, n in ((0, t_max), (13, 40), (70, 1)):
        out = torch.full((B, n, dc + dr), float("nan"), dtype=dtype, device="cuda")
        dsa.dsa_latent_read(cache, fmt, start, out, dc)
        assert np.array_equal(out.double().cpu().numpy(), ref[:, start:start + n])
    idx = torch.randint(-1, t_max, (B, 200), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    out = torch.full((B, 200, dc + dr), float("nan"), dtype=dtype, device="cuda")
    dsa.dsa_latent_read(cache, fmt, 0, out, dc, idx.cuda())
    want = np.stack([ref[b][idx[b].clamp_min(0)] for b in range(B)]) * (idx.numpy() >= 0)[..., None]
    assert np.array_equal(out.double().cpu().numpy(), want)
    assert dsa.dsa_get_device_error() == dsa.DSA_OK


def test_read_records_rows_past_the_cache(dsa):
    cache = new_cache(2, 5, R.Q4, 512, 64, fill=0x11)
    idx = torch.tensor([[0, 5], [4, 1 << 30]], dtype=torch.int32, device="cuda")
    out = torch.ones(2, 2, 576, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_latent_read(cache, R.Q4, 0, out, 512, idx)
    assert not out[0, 1].any() and not out[1, 1].any() and out[0, 0].any() and out[1, 0].any()
    assert dsa.dsa_get_device_error() == dsa.DSA_ERR_DEVICE
    assert dsa.dsa_get_device_error() == dsa.DSA_OK


@pytest.mark.parametrize("S", [1, 3, 64])
def test_append_rounds_from_the_exact_value(dsa, S):
    """Normed rows whose quotients and scales lie close to a border between two codes: the
    stored code is the one of the exact value wherever that is not itself within 2^-40 of the
    border (many rows, so that every near border is met)."""
    dc, dr, B = 512, 64, 4096 // S
    kv = make_kv(B, S, dc, dr, torch.bfloat16, 12 + S, spread=False)
    w = (1 + 0.3 * torch.randn(dc, generator=torch.Generator().manual_seed(1)))
    a = torch.rand(S, dr // 2, generator=torch.Generator().manual_seed(2), dtype=torch.float64) * 6.28
    cs = torch.stack((a.cos(), a.sin()), -1).float()
    ref = R.prologue(kv.double().numpy(), w.double().numpy(), 1e-6, cs.double().numpy(), True, dc)
    for fmt in (R.Q4, R.BF16):
        cache = new_cache(B, S, fmt, dc, dr)
        dsa.dsa_latent_prologue(kv.cuda(), w.cuda(), 1e-6, cs.cuda(), True, 0, cache, fmt, dc)
        got = R.decode_rows(to_bytes(cache), fmt, dc, dr)
        assert np.array_equal(got[..., dc:], R.bf16(ref[..., dc:].astype(np.float32)))
        if fmt == R.BF16:
            assert np.array_equal(got[..., :dc], R.bf16(ref[..., :dc].astype(np.float32)))
            continue
        n, s = R.q4_groups(ref[..., :dc])
        step = np.repeat(s, 32, -1)
        quot = ref[..., :dc] / step
        near = np.abs(np.abs(quot - np.floor(quot)) - 0.5) < 2.0 ** -40
        assert np.all((got[..., :dc] == R.bf16(n * step)) | near)


def q4_scales(y):
    """The 4-bit scales of y [..., dc] in 64 bits: amax / 7 rounded to fp32, then to bf16."""
    amax = np.abs(y.reshape(*y.shape[:-1], -1, 32)).max(-1)
    return R.bf16((np.maximum(amax, np.float64(np.float32(1e-4))) / 7).astype(np.float32))


def near_half(x):
    """Quotients within 2^-40 of a border between two codes."""
    return np.abs(np.abs(x - np.floor(x)) - 0.5) < 2.0 ** -40


@pytest.mark.parametrize("dc", [512, 384, 128])
def test_append_of_groups_next_to_a_border_of_their_scale(dsa, dc):
    """fp32 rows of one magnitude (the sum's roundings add up), each group's largest value moved
    to within six fp32 units of a border between two bf16 scales: the scale is the exact one."""
    rows = 512 * 65536 // dc // 8
    g = np.random.default_rng(dc)
    for it in range(4):
        x = (1 + 0.02 * g.random((rows, dc))) * g.choice([-1.0, 1.0], (rows, dc)) * g.uniform(0.5, 2, (rows, 1))
        w = (1 + 0.3 * g.random(dc)).astype(np.float32)
        at = np.arange(0, dc, 32) + g.integers(0, 32, dc // 32)
        w[at] *= 1.5                                     # each group's largest
        for _ in range(4):                               # (the norm moves a little with it)
            x = x.astype(np.float32).astype(np.float64)
            r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
            s = np.abs(x[:, at]) * r * w[at] / 7
            m, e = np.frexp(s)
            mid = np.ldexp((np.floor(m * 256) + 0.5) / 256, e)
            x[:, at] *= mid / s * (1 + g.uniform(-6, 6, s.shape) * 2.0 ** -23 / (2 * m))
        kv = torch.from_numpy(x.astype(np.float32))[None].contiguous()
        cache = new_cache(1, rows, R.Q4, dc, 0)
        dsa.dsa_latent_prologue(kv.cuda(), torch.from_numpy(w).cuda(), 1e-6, None, False, 0, cache, R.Q4, dc)
        raw = to_bytes(cache)[0]
        y = R.prologue(kv[0].double().numpy(), w.astype(np.float64), np.float64(np.float32(1e-6)), None, False, dc)
        s = q4_scales(y)
        lo = dc // 2
        got = R._u16_as_bf16(raw[:, lo:lo + dc // 16:2], raw[:, lo + 1:lo + dc // 16:2])
        assert np.array_equal(got, s), int((got != s).sum())
        quot = y / np.repeat(s, 32, -1)
        same = R.decode_rows(raw, R.Q4, dc, 0) == R.bf16(np.clip(np.rint(quot), -7, 7) * np.repeat(s, 32, -1))
        assert np.all(same | near_half(quot))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_append_of_values_next_to_a_border_of_bf16(dsa, dtype):
    """Every value of a normed row within six fp32 units of the middle between two bf16 numbers
    (by its weight; by itself too where the row is fp32), rows of one magnitude: the stored
    number is the exact value's."""
    dc, rows = 512, 1500
    g = np.random.default_rng(7)
    for it in range(8):
        x = torch.from_numpy((1 + 0.02 * g.random((rows, dc))) * g.choice([-1.0, 1.0], (rows, dc)) * g.uniform(0.5, 2, (rows, 1)))
        x = x.to(dtype)
        w = (1 + 0.3 * g.random(dc)).astype(np.float32)
        def middle(y):
            m, e = np.frexp(np.abs(y))
            return np.ldexp((np.floor(m * 256) + 0.5) / 256, e) * (1 + g.uniform(-6, 6, y.shape) * 2.0 ** -23 / (2 * m))
        for _ in range(4):
            xd = x.double().numpy()
            r = 1 / np.sqrt((xd * xd).mean(-1, keepdims=True) + 1e-6)
            y = xd * r * w
            if dtype == torch.float32:
                x = torch.from_numpy(xd * middle(y) / np.abs(y)).to(dtype)
            else:                                        # (each dim's weight by one of the rows)
                at = g.integers(0, rows, dc), np.arange(dc)
                w = (w * middle(y[at]) / np.abs(y[at])).astype(np.float32)
        cache = new_cache(1, rows, R.BF16, dc, 0)
        dsa.dsa_latent_prologue(x[None].contiguous().cuda(), torch.from_numpy(w).cuda(), 1e-6, None, False, 0, cache,
                                R.BF16, dc)
        y = R.prologue(x.double().numpy(), w.astype(np.float64), np.float64(np.float32(1e-6)), None, False, dc)
        got = R.decode_rows(to_bytes(cache)[0], R.BF16, dc, 0)
        assert np.array_equal(got, R.bf16(y.astype(np.float32))), int((got != R.bf16(y.astype(np.float32))).sum())


@pytest.mark.parametrize("fmt", [R.BF16, R.Q4])
def test_append_of_values_and_weights_far_apart(dsa, fmt):
    """Small values beside ordinary ones under weights far from one: no product on the way to
    the rounding loses its last bits (or all of them) to fp32's range."""
    dc, B, S = 256, 4, 8
    g = torch.Generator().manual_seed(9)
    kv = make_kv(B, S, dc, 0, torch.float32, 9, spread=False) * 2.0 ** -35
    kv[..., 1::4] *= 2.0 ** -50
    for lo, hi in ((2.0 ** -50, 2.0 ** 50), (2.0 ** -75, 2.0 ** 90), (1.0, 1.0)):
        w = 1 + 0.2 * torch.randn(dc, generator=g)
        w[1::4] *= lo
        w[2::4] *= hi
        cache = new_cache(B, S, fmt, dc, 0)
        dsa.dsa_latent_prologue(kv.cuda(), w.cuda(), 0.0, None, False, 0, cache, fmt, dc)
        got = R.decode_rows(to_bytes(cache), fmt, dc, 0)
        y = R.prologue(kv.double().numpy(), w.double().numpy(), 0.0, None, False, dc)
        if fmt == R.BF16:
            # (torch's cast: R.bf16 has no subnormal numbers, and some of these are)
            assert np.array_equal(got, torch.from_numpy(y).float().bfloat16().double().numpy())
        else:
            step = np.repeat(q4_scales(y), 32, -1)
            assert np.all((got == R.bf16(np.clip(np.rint(y / step), -7, 7) * step)) | near_half(y / step))


@pytest.mark.parametrize("fmt", [R.BF16, R.Q4])
def test_append_of_extreme_and_nan_rows(dsa, fmt):
    """Rows whose squares leave fp32's range (with and without eps) keep the exact norm; a NaN
    makes its row NaN under a norm, its 4-bit group (or itself, in bf16) without one, and no
    other row or group."""
    dc, dr = 256, 16
    kv = make_kv(4, 2, dc, dr, torch.float32, 5, spread=False)
    kv[0] *= 1e25
    kv[1] *= 1e-25
    kv[2, 0, 40] = float("nan")
    w = torch.ones(dc).cuda()
    for eps in (0.0, 1e-6):
        cache = new_cache(4, 2, fmt, dc, dr)
        dsa.dsa_latent_prologue(kv.cuda(), w, eps, None, False, 0, cache, fmt, dc)
        got = R.decode_rows(to_bytes(cache), fmt, dc, dr)[..., :dc]
        ref = R.prologue(kv.double().numpy(), np.ones(dc), eps, None, False, dc)[..., :dc]
        assert np.isnan(got[2, 0]).all()
        keep = np.ones((4, 2), bool)
        keep[2, 0] = False
        if fmt == R.BF16:
            want = R.bf16(ref.astype(np.float32))[keep]
        else:
            n, s = R.q4_groups(ref[keep])
            want = R.bf16(n * np.repeat(s, 32, -1))
        assert np.array_equal(got[keep], want)
    cache = new_cache(4, 2, fmt, dc, dr)
    dsa.dsa_latent_prologue(kv.cuda(), None, 0.0, None, False, 0, cache, fmt, dc)
    got = R.decode_rows(to_bytes(cache), fmt, dc, dr)[..., :dc]
    group = slice(32, 64) if fmt == R.Q4 else slice(40, 41)
    assert np.isnan(got[2, 0, group]).all()
    got[2, 0, group] = 0
    assert np.isfinite(got).all()


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("dc,dr", [(512, 64), (384, 40)])
def test_fp8_append_of_extreme_rows(dsa, dc, dr, eps):
    """Rows whose squares leave fp32's range, beside an ordinary one.  A code is off by half a
    step (2^-4, or 2^-10 scales below the normal codes), the decoded bf16 by 2^-8, the fp32
    chain with its scale by 2^-18 and a few roundings, 2^-17 together."""
    kv = make_kv(3, 4, dc, dr, torch.float32, 6, spread=False)
    for i, f in enumerate((1e25, 1e-25, 1e-18, 1.0, 5e37, 1e-30)):
        kv[i // 4, i % 4] *= f
    kv[2, 0, 7] = float("nan")
    kv[2, 1, 9] = float("inf")
    w = 1 + 0.2 * torch.randn(dc, generator=torch.Generator().manual_seed(8))
    cache = new_cache(3, 4, R.FP8, dc, dr)
    dsa.dsa_latent_prologue(kv.cuda(), w.cuda(), eps, None, False, 0, cache, R.FP8, dc)
    got = R.decode_rows(to_bytes(cache), R.FP8, dc, dr)[..., :dc]
    assert np.isnan(got[2, 0]).all()
    assert np.isnan(got[2, 1, 9]) and not np.delete(got[2, 1], 9).any()
    kv[2, :2] = 1
    got[2, :2] = 0
    ref = R.prologue(kv.double().numpy(), w.double().numpy(), eps, None, False, dc)[..., :dc]
    ref[2, :2] = 0
    scale = np.maximum(np.abs(ref).reshape(3, 4, -1, 128).max(-1), 1e-4) / 448
    tol = np.abs(ref) * (2.0 ** -4 + 2.0 ** -8 + 2.0 ** -12 + 2.0 ** -17)
    assert np.all(np.abs(got - ref) <= tol + np.repeat(scale, 128, -1) * 2.0 ** -10 * (1 + 2.0 ** -7))


def test_append_on_another_stream_and_in_a_graph(dsa):
    B, dc, dr = 4, 512, 64
    kv = make_kv(B, 1, dc, dr, torch.bfloat16, 3).cuda()
    a, b, c = (new_cache(B, 8, R.Q4, dc, dr) for _ in range(3))
    dsa.dsa_latent_prologue(kv, None, 0.0, None, False, 3, a, R.Q4, dc)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dsa.dsa_latent_prologue(kv, None, 0.0, None, False, 3, b, R.Q4, dc, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.dsa_latent_prologue(kv, None, 0.0, None, False, 3, c, R.Q4, dc)
    graph.replay()
    assert torch.equal(a, b) and torch.equal(a, c)
    kv.mul_(-1)                                          # a replay reads the inputs of its time
    graph.replay()
    assert not torch.equal(a, c)
