"""The 64-bit reference of the latent rows, pinned on the CPU against torch's own
casts and by hand-made rows."""
import numpy as np
import torch

import latent_reference as R


def test_bf16_rounding_is_torchs():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(20000, generator=g, dtype=torch.float32) * torch.exp2(torch.randint(-30, 30, (20000,), generator=g))
    assert np.array_equal(R.bf16(x.numpy()), x.to(torch.bfloat16).double().numpy())
    ties = torch.tensor([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, -1 - 2.0 ** -8])
    assert np.array_equal(R.bf16(ties.numpy()), ties.to(torch.bfloat16).double().numpy())


def test_e4m3_table_is_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.E4M3, t, equal_nan=True)


def test_q4_row_by_hand():
    dc, dr = 128, 8
    row = np.zeros(R.row_bytes(R.Q4, dc, dr), np.uint8)
    assert len(row) == 96
    # word 0: values 0..7 = -7, -5, -3, -1, 1, 3, 5, 7 -> codes 1, 3, 5, 7, 9, 11, 13, 15
    codes = [1, 3, 5, 7, 9, 11, 13, 15]
    word = 0
    for v, c in enumerate(codes):
        word |= c << (4 * (v // 2 + 4 * (v % 2)))
    row[:64] = 0x88
    row[:4] = np.frombuffer(np.uint32(word).tobytes(), np.uint8)
    row[64:80] = np.frombuffer(torch.arange(8).to(torch.bfloat16).view(torch.uint8).numpy().tobytes(), np.uint8)
    row[80:88] = torch.tensor([0.5, 1, 2, 4]).to(torch.bfloat16).view(torch.uint8).numpy()
    v = R.decode_rows(row[None], R.Q4, dc, dr)[0]
    assert np.array_equal(v[:8], 0.5 * (np.array(codes) - 8))
    assert not v[8:dc].any()
    assert np.array_equal(v[dc:], np.arange(8))


def test_q4_rounding_is_within_half_a_step():
    x = np.random.default_rng(1).standard_normal((50, 256))
    n, s = R.q4_groups(x)
    err = np.abs(x - n * np.repeat(s, 32, -1))
    # half a step, and what the scale's rounding takes off the largest value (7 steps of 2^-9)
    assert np.all(err <= np.repeat(s, 32, -1) * (0.5 + 7 * 2.0 ** -9) + 1e-12)


def test_block_positions_cover_the_causal_range_when_all_blocks_are_listed():
    for i in (0, 5, 15, 16, 40):
        for m in (1, 7, 16):
            got = R.block_positions(list(range(100)) + [-1], m, i)
            assert sorted(got) == list(range(i + 1))
