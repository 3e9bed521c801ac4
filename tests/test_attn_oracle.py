"""Pins of the attention oracle: the 8-bit format against torch's, the scale
rule and a block's growth worked by hand, the layout, attention against a
plain softmax."""
import sys
import os

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from oracle import attn_oracle as A  # noqa: E402


def test_format_equals_torch():
    codes = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(codes).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(A.e4m3_decode(codes), t, equal_nan=True)
    rng = np.random.default_rng(0)
    x = np.concatenate([np.clip(rng.standard_normal(20000) * s, -448, 448) for s in (1e-3, 0.1, 10, 200)])
    mags = A._MAG[:127]
    mids = (mags[1:] + mags[:-1]) / 2                      # ties, and their neighbours
    x = np.concatenate([x, mids, -mids, np.nextafter(mids, 0), np.nextafter(mids, 1e9), mags, -mags])
    x = x.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(x).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(A.e4m3_encode(x), want)
    assert A.e4m3_encode([np.nan])[0] & 0x7F == 0x7F and A.e4m3_encode([-np.inf])[0] == 0xFF


@pytest.mark.parametrize("amax,scale", [(448.0, 1.0), (448.0000001, 2.0), (449.0, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8),
                                        (1.75, 2.0 ** -8), (1.7500001, 2.0 ** -7), (0.0, 2.0 ** -64), (2.0 ** -80, 2.0 ** -64),
                                        (3.3e38, 2.0 ** 120)])
def test_least_scale(amax, scale):
    assert A.least_scale(amax) == scale


def test_layout_is_a_permutation():
    for D in (64, 128, 256):
        n, d = np.meshgrid(np.arange(16), np.arange(D), indexing="ij")
        for f in (A.k_offset, A.v_offset):
            assert sorted(f(n, d).reshape(-1)) == list(range(16 * D))
    # lane c = 16 g + n: K of token n, columns 8 g.. then 32 + 8 g..; V words of column n, tokens 4 g..
    assert A.k_offset(3, 0) == 48 and A.k_offset(3, 8) == 256 + 48 and A.k_offset(3, 33) == 48 + 9 and A.k_offset(0, 64) == 1024
    assert A.v_offset(0, 3) == 48 and A.v_offset(5, 0) == 256 + 1 and A.v_offset(0, 17) == 16 + 4 and A.v_offset(0, 64) == 1024


def test_append_by_hand():
    """One head, 64 columns: a token of ones, then one that doubles the scale, then a new block."""
    c = A.Cache(np.zeros((1, 1, 2, 2, 1024), np.uint8), np.full((1, 1, 2, 2), 7.0), 32, 1, 64)
    one = np.ones((1, 1, 64))
    c.append([0], 0, one, one * 448)                        # 1 = 256 * 2^-8, 448 = 448 * 1
    assert c.scales[0, 0, 0, 0] == 2.0 ** -8 and c.scales[0, 0, 0, 1] == 1.0
    assert A.e4m3_decode(c.codes[0, 0, 0, 0, A.k_offset(0, 5)]) == 256
    big = np.full((1, 1, 64), 3.0)
    big[0, 0, 1] = np.nan
    c.append([0], 1, big, one)                              # 3 = 384 * 2^-7; the ones become 128 * 2^-7
    assert c.scales[0, 0, 0, 0] == 2.0 ** -7 and c.scales[0, 0, 0, 1] == 1.0
    assert A.e4m3_decode(c.codes[0, 0, 0, 0, A.k_offset(0, 5)]) == 128
    assert A.e4m3_decode(c.codes[0, 0, 0, 0, A.k_offset(1, 5)]) == 384
    assert np.isnan(A.e4m3_decode(c.codes[0, 0, 0, 0, A.k_offset(1, 1)]))
    K, V, there = c.read([0], 0, 2)
    assert K[0, 0, 0] == 1 and K[1, 0, 0] == 3 and V[0, 0, 7] == 448 and V[1, 0, 7] == 1 and there.all()
    c.append([0], 16, one, one)
    assert c.scales[0, 0, 1, 0] == 2.0 ** -8
    assert c.block([3], 0) is None and c.block([-1], 0) is None


def test_rotate_by_hand():
    x = np.arange(1.0, 5.0).reshape(1, 1, 4)
    f = np.array([np.pi / 2, np.pi])
    assert np.allclose(A.rotate(x, [1], f), [[[-3, -2, 1, -4]]])            # pairs (0, 2), (1, 3)
    assert np.allclose(A.rotate(x, [1], f, True, 2.0), [[[-4, 2, -6, -8]]])  # pairs (0, 1), (2, 3)


def test_attention_against_a_plain_softmax():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((5, 4, 8)), rng.standard_normal((7, 2, 8)), rng.standard_normal((7, 2, 8))
    seen = np.arange(7)[None] <= np.arange(5)[:, None] - 1     # row 0 sees nothing, row i keys 0..i-1
    v[4:] = np.nan                                             # keys no row but none sees
    out, lse, _, _ = A.attention(q, k, v, seen, 0.3)
    assert np.all(out[0] == 0) and np.all(lse[0] == -np.inf)
    for i in range(1, 5):
        for h in range(4):
            s = torch.tensor(k[:i, h // 2] @ q[i, h] * 0.3)
            assert np.allclose(out[i, h], torch.softmax(s, 0).numpy() @ v[:i, h // 2])
            assert np.isclose(lse[i, h], torch.logsumexp(s, 0).item())
