"""Pins of the oracle of the norm, the 4-bit products and the page calls: values worked by hand."""
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from oracle import step_oracle as S  # noqa: E402


def test_norm_by_hand():
    # mean square of (3, -4, 0, 5) is 12.5
    y = S.rms_norm([3.0, -4.0, 0.0, 5.0], np.array([1.0, 2.0, 1.0, 0.5]), 0.0)
    assert np.allclose(y, np.array([3, -8, 0, 2.5]) / np.sqrt(12.5), rtol=1e-15)
    assert np.allclose(S.rms_norm([0.0, 0.0], 1.0, 0.25), [0, 0])


def test_codes_by_hand():
    y = np.array([127.0, -63.5, 0.5, -1.5, 2.5, 0, 0, 0] + [0.0] * 120 + [254.0, 1.0, 3.0, -5.0])
    codes, scales = S.codes8(y, 128)
    assert scales.tolist() == [1.0, 2.0]
    assert codes[:8].tolist() == [127, -64, 0, -2, 2, 0, 0, 0]         # ties to even
    assert codes[128:].tolist() == [127, 0, 2, -2]
    assert S.codes8(y, 0)[1].tolist() == [2.0]
    codes, scales = S.codes8(np.zeros(8), 0)
    assert not codes.any() and scales[0] == 0
    codes, scales = S.codes8(np.array([1.0, np.inf]), 0)
    assert not codes.any() and np.isnan(scales[0])


def test_quantizer_by_hand():
    w = np.zeros((2, 32))
    w[0, :4] = [-7.0, 3.4, 3.5, 7.0]
    w[1, :3] = [-1.0, 2.0, 0.1]
    q, s, z = S.quantize4(w, 32, False)
    assert s[0, 0] == 1 and q[0, :5].tolist() == [1, 11, 12, 15, 8] and (z == 8).all()
    q, s, z = S.quantize4(w, 32, True)
    step = float(np.float16(3 / 15))
    assert s[1, 0] == step and z[1, 0] == 5 and q[1, :4].tolist() == [0, 15, 6, 5]
    assert np.allclose(S.weights4(q, s, z, 32)[1, :3], [-5 * step, 10 * step, step])


def test_layout_by_hand():
    q = np.full((17, 136), 8, np.uint8)
    q[3, 41] = 1            # tile 0: word 1, lane 16 * 1 + 3, j = 1: bit 16
    q[16, 130] = 0xF        # the last tile: word 0, lane 0, j = 2: bit 4
    s = np.zeros((17, 3), np.float16)
    s[16, 2] = 1.0          # group 2 of 64: columns 128 and on, the last tile's first
    z = np.full((17, 3), 8, np.uint8)
    z[3, 1] = 7
    b = S.pack4(q, s, z, 64).reshape(4, -1)
    size = 1024 + 64 + 32
    assert b.shape == (4, size)
    at = 16 * 19 + 4 * 1 + 2
    assert b[0, at] == 1 ^ 8 and b[3, 0] == (0xF ^ 8) << 4
    assert b[3, 1024:1026].tolist() == [0x00, 0x3C] and b[0, 1024 + 64 + 2 * 3 + 1] == 255
    b[0, at], b[3, 0], b[3, 1025], b[0, 1024 + 64 + 7] = 0, 0, 0, 0
    assert not b.any()


def test_pages_by_hand():
    p = S.Pages([[4, 2, -1], [2, -1, -1], [-1] * 3], [33, 16, 0], [0, 0, 2, 0, 1, 0], 16)
    # row 0 holds 4, 2 and (for its 33rd position) an entry that names nothing
    assert p.resize([20, 0, 40]) == 0
    assert p.table == [[4, 2, -1], [-1] * 3, [0, 1, 3]] and p.refs == [1, 1, 1, 1, 1, 0] and p.lens == [20, 0, 40]
    assert p.fork([-1, 2, 5]) == 0                       # row 1 from row 2: two full pages shared, the third copied
    assert p.table[1] == [0, 1, 5] and p.refs == [2, 2, 1, 1, 1, 1] and p.copies == [(3, 5, 1)]
    assert p.resize([48, -1, -1]) == 1 and p.lens[0] == 20          # no page is free
    p.resize([0, -1, 17])
    assert p.refs == [2, 2, 0, 0, 0, 1] and p.lens == [0, 40, 17]
    assert p.fork([0, 1, 2]) == 0                        # row 2 ends inside page 1, which row 1 holds too
    assert p.table[2][:2] == [0, 2] and p.refs == [2, 1, 1, 0, 0, 1] and p.copies[-1] == (1, 2, 1)
    assert p.compact() == 4 and p.table[1] == [0, 1, 3] and p.refs == [2, 1, 1, 1, 0, 0] and p.copies[-1] == (5, 3, 1)
