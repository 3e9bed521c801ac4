"""GPU parity of moe_rms_norm against the 64-bit oracle: every type, widths around the kernels' borders, heads, strides, in
place, 8-bit outputs code by code, rows that are zero, huge or not finite."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

from attn_fixture import f64, half_step, in_type, subnormal_half  # noqa: E402
from oracle import step_oracle as S  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU test needs a GPU"
    from bit_quantized_moe_02_amd import qmoe
    return qmoe


def vectors(x, dt, pad=0):
    """x [rows, (heads,) cols] on the GPU, rows `pad` elements further apart than they are long; the rest holds NaN."""
    wide = x[0].size
    buf = torch.full((x.shape[0], wide + pad), float("nan"), dtype=dt, device="cuda")
    view = buf[:, :wide].view(x.shape) if pad == 0 else buf[:, :wide].unflatten(1, x.shape[1:]) if x.ndim == 3 else buf[:, :wide]
    view.copy_(torch.from_numpy(np.ascontiguousarray(x)).to(dt))
    return view, buf


def blank(shape, dt, pad=0, fill=77):
    wide = int(np.prod(shape[1:]))
    buf = torch.full((shape[0], wide + pad), fill, dtype=dt, device="cuda")
    return (buf[:, :wide].unflatten(1, shape[1:]) if len(shape) == 3 else buf[:, :wide]), buf


def check_out(got, y, dt, what):
    """y in 64 bits; the kernel's is a product of three 32-bit numbers, one of them rounded (the root, from 64 bits):
    three roundings of 2^-24, and the output's own."""
    got = f64(got)
    assert np.array_equal(np.isnan(got), np.isnan(y)), what
    own = half_step(dt) if dt != torch.float32 else 0.0
    with np.errstate(all="ignore"):
        tol = (own * (1 + 2.0 ** -20) + 3.01 * 2.0 ** -24) * np.abs(y) + subnormal_half(dt) + 2.0 ** -148
        bad = ~(np.abs(got - y) <= tol) & np.isfinite(y)
    assert not bad.any(), f"{what}: {np.argwhere(bad)[:5].tolist()}"


def run(q, rng, rows, heads, cols, xt, rt, ot, wt="bf16", group=None, pads=(0, 0, 0, 0, 0), x=None, res=None, eps=1e-5, what=""):
    shape = (rows, cols) if heads == 1 else (rows, heads, cols)
    x = rng.standard_normal(shape) if x is None else x
    xd, _ = vectors(x, DT[xt], pads[0])
    h = f64(xd)
    rd = sd = sbuf = None
    if rt:
        rd, _ = vectors(3 * rng.standard_normal(shape) if res is None else res, DT[rt], pads[1])
        sd, sbuf = blank(shape, DT[rt], pads[2])
        h = S.add(h, f64(rd), lambda v: in_type(v, DT[rt]))
    w = wd = None
    if wt:
        wd = torch.from_numpy(1 + 0.1 * rng.standard_normal(cols)).to(DT[wt]).cuda()
        w = f64(wd)
    y = S.rms_norm(h, 1.0 if w is None else w, eps)
    od = obuf = cd = cbuf = sc = None
    if ot:
        od, obuf = blank(shape, DT[ot], pads[3])
    if group is not None:
        cd, cbuf = blank(shape, torch.int8, pads[4])
        sc = torch.full(q.moe_scales_shape(rows, cols, group, heads), -5.0, device="cuda")
    q.moe_rms_norm(xd, od, wd, eps, residual=rd, sum_out=sd, codes=cd, scales=sc, group=group or 0)
    torch.cuda.synchronize()
    if rt:
        assert np.array_equal(f64(sd), h, equal_nan=True), f"{what}: sum"
    if ot:
        check_out(od, y, DT[ot], what)
    if group is not None:
        codes, scales = S.codes8(y, group)
        got = f64(sc)
        want = scales.reshape(rows, -1).T
        assert np.array_equal(got[:, :rows], want, equal_nan=True), f"{what}: scales"
        assert (got[:, rows:] == -5).all(), f"{what}: scales behind the last row"
        assert np.array_equal(cd.cpu().numpy(), codes), f"{what}: codes"
    for buf, pad in ((sbuf, pads[2]), (obuf, pads[3]), (cbuf, pads[4])):
        if buf is not None and pad:
            assert (buf[:, -pad:] == 77).all(), f"{what}: written past a row's end"
    return h, y


@pytest.mark.parametrize("xt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rt", [None, "bf16", "fp16", "fp32"])
@pytest.mark.parametrize("cols", [72, 512, 4096, 8200])
def test_types(q, xt, rt, cols):
    rng = np.random.default_rng(cols + len(xt))
    for ot, wt, group in (("bf16", "bf16", 128), ("fp16", "fp32", 0), ("fp32", "fp16", None), ("bf16", None, None)):
        run(q, rng, 3, 1, cols, xt, rt, ot, wt, group, what=f"{ot} {wt} {group}")


@pytest.mark.parametrize("cols", [8, 16, 56, 64, 120, 128, 136, 248, 256, 264, 504, 520, 1024, 2048, 2056, 4104, 7168, 8192, 12296, 16376, 16384])
def test_widths(q, cols):
    rng = np.random.default_rng(cols)
    for rows in (1, 2, 7):
        for group in (0, 128):
            run(q, rng, rows, 1, cols, "bf16", "bf16", "bf16", "bf16", group, what=f"{rows} {group}")
            run(q, rng, rows, 1, cols, "fp32", "bf16", None, "bf16", group, what=f"codes alone, {rows} {group}")


@pytest.mark.parametrize("heads,cols", [(2, 8), (3, 64), (48, 128), (5, 136), (32, 256), (2, 512), (3, 1032), (4096, 8)])
def test_heads(q, heads, cols):
    """Vectors of their own, as queries and keys have, parts of a wider row."""
    rng = np.random.default_rng(heads * cols)
    run(q, rng, 5, heads, cols, "bf16", None, "bf16", "bf16", None, (64, 0, 0, 128, 0))
    run(q, rng, 3, heads, cols, "fp16", "fp16", "fp16", "fp32", 128, (8, 16, 24, 32, 40))
    run(q, rng, 2, heads, cols, "fp32", "fp32", None, None, 0, (8, 16, 24, 32, 40))


@pytest.mark.parametrize("cols", [128, 520, 4096, 16384])
def test_strides(q, cols):
    run(q, np.random.default_rng(cols), 6, 1, cols, "bf16", "fp32", "fp16", "bf16", 128, (8, 24, 40, 16, 8))


def test_many_rows(q):
    rng = np.random.default_rng(9)
    run(q, rng, 70001, 1, 64, "bf16", "bf16", "bf16", "bf16", 0)
    run(q, rng, 1000, 1, 2056, "fp32", "bf16", None, "bf16", 128)


@pytest.mark.parametrize("cols", [64, 4096])
def test_in_place(q, cols):
    rng = np.random.default_rng(cols)
    x, r = rng.standard_normal((4, cols)), rng.standard_normal((4, cols))
    w = torch.ones(cols, device="cuda")
    for into in ("residual", "x"):
        xd, rd = vectors(x, torch.bfloat16)[0], vectors(r, torch.bfloat16)[0]
        h = S.add(f64(xd), f64(rd), lambda v: in_type(v, torch.bfloat16))
        s, o = (rd, xd) if into == "residual" else (xd, rd)
        q.moe_rms_norm(xd, o, w, 1e-6, residual=rd, sum_out=s)
        assert np.array_equal(f64(s), h)
        check_out(o, S.rms_norm(h, 1.0, 1e-6), torch.bfloat16, into)
    # sum alone
    rd, s = vectors(r, torch.bfloat16)[0], torch.empty((4, cols), dtype=torch.bfloat16, device="cuda")
    q.moe_rms_norm(vectors(x, torch.bfloat16)[0], residual=rd, sum_out=s)
    assert np.array_equal(f64(s), h)


@pytest.mark.parametrize("cols", [64, 264, 2048, 7168])
def test_sizes_of_values(q, cols):
    """Squares past 32 bits, values that vanish in the scale, zeros, one large column."""
    rng = np.random.default_rng(cols)
    x = rng.standard_normal((8, cols))
    x[0] = 0
    x[1] *= 1e30
    x[2] *= 1e-30
    x[3] *= 3e38 / np.abs(x[3]).max()
    x[4, cols // 3] = 1e6
    x[5] = 1e-38 * np.sign(x[5])
    x[6, :-1] = 0
    x[7, cols // 2:] = 0
    for group in (0, 128):
        run(q, rng, 8, 1, cols, "fp32", None, "fp32", "bf16", group, x=x.copy(), what="eps")
        run(q, rng, 8, 1, cols, "fp32", None, "bf16", None, group, x=x.copy(), eps=0.0, what="no eps")
        run(q, rng, 8, 1, cols, "bf16", "fp32", None, "bf16", group, x=x[[0, 1, 2, 4, 5, 6, 7, 7]], what="sum")


@pytest.mark.parametrize("cols", [64, 512, 4096])
def test_not_finite(q, cols):
    """What is not finite stays in its vector (of the codes: in its group, where its root leaves the others zero)."""
    rng = np.random.default_rng(cols)
    x = rng.standard_normal((6, cols))
    x[1, 5] = np.inf
    x[2, cols - 1] = np.nan
    x[4, 0], x[4, 9] = -np.inf, np.inf
    for group in (0, 128):
        run(q, rng, 6, 1, cols, "bf16", None, "bf16", "bf16", group, x=x.copy())
        run(q, rng, 6, 1, cols, "fp32", "fp32", "fp32", None, group, x=x.copy())


def test_codes_next_to_borders(q):
    """Codes that 32 bits would round elsewhere: the weights put y / scale at a half and 2^-27 beside it."""
    rng = np.random.default_rng(5)
    cols = 512
    x = np.ones((1, cols))
    w = np.empty(cols)
    w[:] = (rng.integers(-126, 126, cols) + 0.5) / 127
    w[0] = 1.0
    w *= 1 + rng.choice([-1, 1], cols) * 2.0 ** rng.integers(-24, -19, cols)
    w[0] = 1.0
    xd, wd = torch.ones((1, cols), device="cuda"), torch.from_numpy(w).float().cuda()
    cd, sc = torch.empty((1, cols), dtype=torch.int8, device="cuda"), torch.empty((1, 4), device="cuda")
    q.moe_rms_norm(xd, None, wd, 0.0, codes=cd, scales=sc)
    codes, scales = S.codes8(S.rms_norm(x, f64(wd), 0.0), 0)
    assert float(sc[0, 0]) == scales[0, 0] and np.array_equal(cd.cpu().numpy(), codes)


def test_other_stream_and_graph(q):
    rng = np.random.default_rng(1)
    x, r = (torch.from_numpy(rng.standard_normal((3, 4096))).bfloat16().cuda() for _ in range(2))
    s, y = torch.empty_like(r), torch.empty_like(x)
    want_s, want_y = torch.empty_like(r), torch.empty_like(x)
    q.moe_rms_norm(x, want_y, None, residual=r, sum_out=want_s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q.moe_rms_norm(x, y, None, residual=r, sum_out=s, stream=side)
    side.synchronize()
    assert torch.equal(s, want_s) and torch.equal(y, want_y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.moe_rms_norm(x, y, None, residual=r, sum_out=s)
    for i in range(3):
        x.copy_(torch.from_numpy(rng.standard_normal((3, 4096))).bfloat16())
        q.moe_rms_norm(x, want_y, None, residual=r, sum_out=want_s)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(s, want_s) and torch.equal(y, want_y)


def test_binding_refusals(q):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    for kw in (dict(out=x[:3]), dict(out=torch.zeros((4, 64), dtype=torch.float64, device="cuda")), dict(out=x.cpu()),
               dict(out=torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")[:, ::2]), dict(sum_out=x.clone()),
               dict(residual=x, sum_out=x.half()), dict(out=x.clone(), weight=x[0, :32].contiguous()), dict(out=x.clone(), weight=x),
               dict(codes=x), dict(codes=x.to(torch.int8), scales=torch.zeros((2, 4), device="cuda")),
               dict(codes=x.to(torch.int8), scales=torch.zeros((1, 2), device="cuda")), dict(out=x.clone(), group=-1)):
        with pytest.raises(ValueError):
            q.moe_rms_norm(x, **kw)
    for kw in (dict(), dict(codes=x.to(torch.int8)), dict(out=x.clone(), eps=-1.0)):
        with pytest.raises(q.QmoeError):
            q.moe_rms_norm(x, **kw)
    with pytest.raises(ValueError):
        q.moe_rms_norm(torch.zeros(64, device="cuda"), None)
