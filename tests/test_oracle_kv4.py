"""The 4-bit row format of the oracle, pinned by hand-worked rows and by its own bound:
|x - (code s + m)| <= s / 2, whatever the group."""
import numpy as np
import pytest

from oracle.sinkkv_oracle import kv4_pack, kv4_quantise, kv4_unpack, kv4_values


def test_a_worked_group():
    # 0, 1, .., 15, 15, 14, .., 0: m = 0, s = 1 and the codes are the values
    x = np.concatenate([np.arange(16.0), np.arange(15, -1, -1.0)])
    codes, mb, sb = kv4_quantise(x)
    assert mb.tolist() == [0x0000] and sb.tolist() == [0x3F80]      # bf16 0 and 1
    assert codes[0].tolist() == x.tolist()
    # ties go to even: 0.5 -> 0, 1.5 -> 2, 2.5 -> 2
    x = np.zeros(32)
    x[:4] = [0.5, 1.5, 2.5, 15.0]
    assert kv4_quantise(x)[0][0, :4].tolist() == [0, 2, 2, 15]


def test_a_worked_row():
    """Bytes of a 64-dim row: word (t, group) at 4 (2 t + group), nibble n = dim 32 group + 8 t + n."""
    k = np.zeros(64)
    k[0], k[15] = 15.0, 3.0          # group 0: t = 0 nibble 0; t = 1 nibble 7
    k[32 + 25] = -15.0               # group 1: m = -15, s = 1, t = 3 nibble 1 holds code 0, the others 15
    row = kv4_pack(k, np.full(64, 2.5))
    assert row.shape == (80,)
    assert row[:4].tolist() == [15, 0, 0, 0]
    assert row[8:12].tolist() == [0, 0, 0, 0x30]
    assert row[4:8].tolist() == [255] * 4 and row[28:32].tolist() == [0x0F, 255, 255, 255]
    assert row[32:40].view("<u2").tolist() == [0x0000, 0x3F80, 0xC170, 0x3F80]   # (0, 1), (-15, 1)
    assert row[40:72].tolist() == [0] * 32                                       # a constant half: s = 0
    assert row[72:80].view("<u2").tolist() == [0x4020, 0, 0x4020, 0]             # 2.5


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["normal", "offset", "tiny", "large", "mixed", "constant"])
def test_values_are_within_half_a_step(D, kind):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((40, D)).astype(np.float32)
    x = {"normal": x, "offset": x + np.float32(100), "tiny": x * np.float32(1e-30), "large": x * np.float32(1e30),
         "mixed": x * np.exp(rng.uniform(-20, 20, (40, D))).astype(np.float32),
         "constant": np.full_like(x, -3.3)}[kind]
    codes, mb, sb = kv4_quantise(x)
    got = kv4_values(codes, mb, sb)
    s = (sb.astype(np.uint32) << 16).view(np.float32).astype(np.float64).repeat(32, -1)
    # half a step, and the fp32 roundings of x - m and of the quotient (15 s 2^-23)
    assert np.all(np.abs(got - x) <= s / 2 + 16 * s * 2.0 ** -23)
    K, V = kv4_unpack(kv4_pack(x, x[::-1]))
    assert np.array_equal(K, got) and np.array_equal(V, got[::-1])


def test_bf16_minima_are_exact():
    """m is the group's minimum itself when the values are bf16, and the minimum gets code 0."""
    rng = np.random.default_rng(6)
    x = (rng.standard_normal((50, 128)).astype(np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32)
    codes, mb, sb = kv4_quantise(x)
    m = (mb.astype(np.uint32) << 16).view(np.float32)
    assert np.array_equal(m, x.reshape(50, 4, 32).min(-1))
    assert np.all(codes.min(-1) == 0)
