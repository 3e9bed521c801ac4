"""GPU checks of the norm, the 4-bit products and the page calls at the sizes where a call takes another way: every split of a
product over workgroups, pools on both sides of what is looked through at once, lists of pages longer than LDS; calls side
by side on two streams, and scales without room behind them."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

from attn_fixture import i32  # noqa: E402
from test_gpu_step_linear import matrix, rows16, run  # noqa: E402
from test_gpu_step_pages import Both  # noqa: E402


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU test needs a GPU"
    from bit_quantized_moe_02_amd import qmoe
    return qmoe


# What a workgroup takes (rows of x, tiles of 16 weight rows) follows from rows and n; these reach every one for 256 compute units.
SPLITS = [(3, 4001), (3, 7161), (4, 14321), (9, 1999), (16, 4096), (13, 7160), (60, 511), (16, 14330), (50, 1001), (64, 2040), (64, 4090),
          (33, 4799), (64, 7170), (70, 9600), (40, 14333), (130, 600), (64, 20000), (8, 28672)]


@pytest.mark.parametrize("rows,n", SPLITS)
@pytest.mark.parametrize("xt,group,zeros,x_group", [("bf16", 128, False, 0), ("fp16", 32, True, 0), ("bf16", 64, True, 0), ("int8", 128, True, 128),
                                                    ("int8", 64, False, 0), ("int8", 32, True, 0)])
def test_splits(q, rows, n, xt, group, zeros, x_group):
    run(q, np.random.default_rng(rows + n), n, 1160 if group == 128 else 328, rows, xt, group, zeros, "fp32", True, x_group, (8, 3))


def test_scales_need_room(q):
    """The last group's scales are read up to the next multiple of 4 rows."""
    rng = np.random.default_rng(0)
    m, _, _, _ = matrix(q, rng, 32, 256, 64, False)
    x, y = torch.zeros((5, 256), dtype=torch.int8, device="cuda"), torch.zeros((5, 32), device="cuda")
    room = torch.ones(16, device="cuda")
    q.moe_linear(m, x, y, room.as_strided((2, 5), (8, 1)), 128)
    tight = torch.ones(13, device="cuda")
    with pytest.raises(ValueError, match="room"):
        q.moe_linear(m, x, y, tight.as_strided((2, 5), (8, 1)), 128)


@pytest.mark.parametrize("n_pages", [4095, 4096, 4097, 16383, 16385, 65535, 65536, 65537, 131072])
def test_pools_of_every_size(q, n_pages):
    """All pages taken, some given back, taken again, moved: on both sides of what is looked through at once."""
    rng = np.random.default_rng(n_pages)
    seqs = 5
    per = -(-n_pages // seqs) + 3
    s = Both(q, rng, n_pages, seqs, per, 16, caches=())
    s.resize([16 * (n_pages // seqs)] * seqs)
    s.resize([16 * (n_pages // seqs) + 33] + [-1] * 4)
    s.resize([-1, 16 * 7, 5, -1, 0])
    s.resize([-1, 16 * 9, -1, 16 * per, 16 * 40])
    s.fork([-1, -1, 1, -1, -1])
    s.compact()
    s.resize([16 * 5, -1, -1, -1, -1])
    s.compact()


def test_more_pages_than_a_list_holds(q):
    """Rows that take 60000 pages from windows with holes: the list in LDS is filled more than once, inside a window too."""
    rng = np.random.default_rng(3)
    n, per = 140000, 30000
    s = Both(q, rng, n, 4, per, 16, caches=(), lens=[16 * per, 16 * per, 0, 0], others=20000)
    s.resize([7, -1, 16 * per, 16 * per])
    s.resize([16 * per, 0, 16 * 3 + 1, -1])
    s.resize([-1, 16 * per, 16 * per, 16 * per])


def test_most_rows(q):
    rng = np.random.default_rng(4)
    seqs, per = 4096, 9
    s = Both(q, rng, 30000, seqs, per, 16, caches=((1, 64),), wide=2)
    s.resize([int(x) for x in rng.integers(0, per * 16 + 1, seqs)])      # (the last rows lack theirs)
    s.resize([int(x) for x in rng.integers(-30, 100, seqs)])
    s.fork([int(x) for x in rng.integers(-1, seqs, seqs)])
    s.compact()


def test_steps_side_by_side(q):
    """The same calls on two pools, two streams at once, eager and captured."""
    rng = np.random.default_rng(5)
    both = [Both(q, rng, 9000, 48, 180, 16, caches=((2, 64),), lens=[int(x) for x in rng.integers(0, 2500, 48)]) for _ in range(2)]
    new = [[i32([int(x) for x in rng.integers(-100, 2800, 48)]) for _ in range(4)] for _ in range(2)]
    origin = [i32([int(x) for x in rng.integers(-1, 48, 48)]) for _ in range(2)]
    ws = [[torch.empty(f(s.pool, s.tables), dtype=torch.uint8, device="cuda") for f in (q.moe_kv_fork_workspace_bytes, q.moe_kv_compact_workspace_bytes)] for s in both]
    w, _, _, _ = matrix(q, rng, 4096, 512, 128, False)
    x = [rows16(rng, 40, 512, torch.bfloat16)[0].contiguous() for _ in range(2)]
    want = [torch.empty((40, 4096), device="cuda") for _ in range(2)]
    got = [torch.empty((40, 4096), device="cuda") for _ in range(2)]
    for i in range(2):
        q.moe_linear(w, x[i], want[i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for step in range(4):
        for i, s in enumerate(both):
            q.moe_kv_resize(s.pool, s.tables, new[i][step], stream=streams[i])
            q.moe_linear(w, x[i], got[i], stream=streams[i])
            if step == 2:
                q.moe_kv_fork(s.pool, s.tables, origin[i], ws[i][0], stream=streams[i])
        if step == 3:
            for i, s in enumerate(both):
                q.moe_kv_compact(s.pool, s.tables, ws[i][1], s.out, stream=streams[i])
    torch.cuda.synchronize()
    for i, s in enumerate(both):
        for step in range(4):
            s.o.resize(new[i][step].tolist())
            if step == 2:
                s.o.fork(origin[i].tolist())
        s.same(s.o.compact(), f"pool {i}")
        assert torch.equal(got[i], want[i])


def test_first_calls_inside_a_capture(q):
    """Sizes that no call had before: nothing is set up on the way that a capture does not allow."""
    rng = np.random.default_rng(6)
    w, _, _, _ = matrix(q, rng, 14336, 136, 64, True)
    x = rows16(rng, 61, 136, torch.float16)[0].contiguous()
    y, want = torch.empty((61, 14336), dtype=torch.float16, device="cuda"), torch.empty((61, 14336), dtype=torch.float16, device="cuda")
    s = Both(q, rng, 70000, 3000, 20, 16, caches=())
    new, missing = i32([16 * 20] * 3000), i32([0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.moe_linear(w, x, y)
        q.moe_kv_resize(s.pool, s.tables, new, missing)
    q.moe_linear(w, x, want)
    for step in range(3):
        g.replay()
        lack = s.o.resize(new.tolist())
        s.out.copy_(missing)
        s.same(lack, f"replay {step}")
        assert torch.equal(y, want)
        y.zero_()
        new.copy_(i32([(int(b) * 7 + step * 50) % 330 - 5 for b in range(3000)]))
