"""GPU tests of calls to the attention entry points that their header allows: drafts that are cut back."""
import numpy as np
import pytest

from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch
    assert torch.cuda.is_available(), "GPU test needs a GPU"
    from bit_quantized_moe_02_amd import qmoe
    return qmoe


import torch  # noqa: E402

from attn_fixture import DT, f64, i32, page_table, random_cache, rows_in, to_device  # noqa: E402


def _same(dev, ref):
    got = A.Cache(dev.codes.cpu().numpy(), f64(dev.scales), ref.page, ref.heads, ref.dim)
    assert np.array_equal(got.scales, ref.scales)
    assert np.array_equal(got.codes[:, :, :, 1], ref.codes[:, :, :, 1]), "V codes differ"
    assert np.array_equal(got.codes[:, :, :, 0], ref.codes[:, :, :, 0]), "K codes differ"


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_append_after_a_draft_is_cut_back(q, dt):
    """A rejected draft's large values: the block keeps their scale, and its kept tokens the second rounding, until its
    first slot is written again; a block that only the draft was in starts anew."""
    dt = DT[dt]
    rng = np.random.default_rng(70)
    D, Hk, page = 64, 2, 16
    table, n_pages = page_table(rng, [64], page)
    codes, scales = random_cache(rng, n_pages, page, Hk, D)
    ref = A.Cache(codes, scales, page, Hk, D)
    dev = to_device(q, ref)

    def step(first, n, sigma):
        kt, kv = rows_in(rng, n, Hk, D, dt, sigma=sigma)
        vt, vv = rows_in(rng, n, Hk, D, dt, sigma=sigma)
        q.moe_kv_append(dev, q.KvBatch(i32(table), i32([first + n]), n), kt, vt)
        ref.append(table[0], first, kv, vv)
        _same(dev, ref)
        return np.abs(kv).max((0, 2))

    def scale(pos):
        page_, blk = ref.block(table[0], pos)
        return ref.scales[page_, :, blk, 0]

    small = step(0, 12, 2.0 ** -10)                     # a prompt of small values
    step(12, 8, 64.0)                                   # a draft over two blocks, rejected
    step(12, 2, 2.0 ** -10)
    assert np.all(scale(0) > 2.0 ** 10 * small / 448)   # the block's scale is still the draft's
    step(14, 6, 2.0 ** -10)
    assert np.all(scale(16) < 2.0 ** -10)               # the next block's first slot was written again
    step(0, 12, 2.0 ** -10)
    assert np.all(scale(0) < 2.0 ** -10)
