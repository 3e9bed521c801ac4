"""GPU test of a serving program's run: pages, norm, projection in 8 bits, cache, attention, projection back, norm, experts,
step after step, eager (each call checked on what the calls before it left) and captured."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

import synth  # noqa: E402
from attn_fixture import attention_bounds, check_attention, f64, half_step, i32, in_type  # noqa: E402
from layer_fixture import device_layer, oracle_layer, rel_err  # noqa: E402
from oracle import attn_oracle as A  # noqa: E402
from oracle import step_oracle as S  # noqa: E402

BF = torch.bfloat16
SEQS, HQ, HK, D, PAGE = 4, 4, 2, 64, 16


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU test needs a GPU"
    from bit_quantized_moe_02_amd import qmoe
    return qmoe


class Program:
    """Everything a small server keeps; step() is one token of each sequence through one layer."""

    def __init__(self, q, seed):
        self.q, rng = q, np.random.default_rng(seed)
        wl = synth.WORKLOADS["tiny"]
        self.wl, self.layer, H = wl, device_layer(wl), wl.hidden
        E, k = wl.n_experts, wl.top_k
        cuda = lambda x, t: torch.from_numpy(np.asarray(x)).to(t).cuda()  # noqa: E731

        def matrix(n, kk, group, zeros):
            codes, scales, zp = q.moe_linear_quantize((rng.standard_normal((n, kk)) / kk ** 0.5).astype(np.float32), group, zeros)
            w = S.weights4(codes, scales, np.full(scales.shape, 8) if zp is None else zp, group)
            return q.LinearWeights(torch.from_numpy(q.moe_linear_pack(codes, scales, zp, group)).cuda(), n, kk, group, zeros), w

        self.qkv_w, self.qkv_v = matrix((HQ + 2 * HK) * D, H, 32, True)
        self.o_w, self.o_v = matrix(H, HQ * D, 128, False)
        self.norms = [cuda(1 + 0.1 * rng.standard_normal(H), BF) for _ in range(2)]
        n_pages, per = 24, 6
        self.cache = q.KvCache(torch.full((n_pages * 2 * PAGE * HK * D,), 0x7F, dtype=torch.uint8, device="cuda"), None, PAGE, HK, D)
        self.cache.scales.fill_(1.0)
        self.table, self.lens = torch.full((SEQS, per), -1, dtype=torch.int32, device="cuda"), i32([0] * SEQS)
        self.refs, self.new, self.origin = i32([0] * n_pages), i32([0] * SEQS), i32([-1] * SEQS)
        self.pool, self.tables = q.KvPool(self.refs, [self.cache]), q.KvTables(self.table, self.lens, PAGE)
        self.batch = q.KvBatch(self.table, self.lens, SEQS)
        self.freqs = q.moe_rope_freqs(D)
        self.rope = q.Rope(cuda(self.freqs, torch.float64), D)
        e = lambda t, *s: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        self.h, self.delta = cuda(rng.standard_normal((SEQS, H)), BF), cuda(rng.standard_normal((SEQS, H)), torch.float32)
        self.codes, self.scales = e(torch.int8, SEQS, H), e(torch.float32, *q.moe_scales_shape(SEQS, H, 128))
        self.qkv, self.attn = e(BF, SEQS, HQ + 2 * HK, D), e(BF, SEQS, HQ, D)
        self.o, self.x = e(BF, SEQS, H), e(BF, SEQS, H)
        self.idx, self.w = e(torch.int32, SEQS, k), e(torch.float32, SEQS, k)
        self.fork_ws = e(torch.uint8, q.moe_kv_fork_workspace_bytes(self.pool, self.tables))
        self.compact_ws = e(torch.uint8, q.moe_kv_compact_workspace_bytes(self.pool, self.tables))
        self.attn_ws = e(torch.uint8, q.moe_attn_decode_workspace_bytes(self.cache, self.batch, HQ))
        self.layer_ws = e(torch.uint8, q.moe_layer_decode_workspace_bytes(self.layer.w, SEQS, k))

    def step(self, look=lambda what: None):
        q = self.q
        q.moe_kv_compact(self.pool, self.tables, self.compact_ws)
        q.moe_kv_fork(self.pool, self.tables, self.origin, self.fork_ws)
        q.moe_kv_resize(self.pool, self.tables, self.new)
        look("pages")
        q.moe_rms_norm(self.delta, None, self.norms[0], 1e-6, residual=self.h, sum_out=self.h, codes=self.codes, scales=self.scales, group=128)
        look("norm in 8 bits")
        q.moe_linear(self.qkv_w, self.codes, self.qkv, self.scales, 128)
        look("projection")
        qs, ks, vs = self.qkv[:, :HQ], self.qkv[:, HQ:HQ + HK], self.qkv[:, HQ + HK:]
        q.moe_kv_append(self.cache, self.batch, ks, vs, self.rope, qs, qs, ks)
        q.moe_attn_decode(self.cache, self.batch, qs, self.attn, self.attn_ws, D ** -0.5)
        look("attention")
        q.moe_linear(self.o_w, self.attn, self.o)
        look("projection back")
        q.moe_rms_norm(self.o, self.x, self.norms[1], 1e-6, residual=self.h, sum_out=self.h)
        look("norm")
        q.moe_layer_decode(self.layer.w, self.layer.router, None, self.x, SEQS, self.wl.top_k, self.idx, self.w, self.delta, self.layer_ws)
        look("experts")

    def state(self):
        return [t.clone() for t in (self.h, self.delta, self.table, self.lens, self.refs, self.cache.codes, self.cache.scales)]


def plan(step, lens):
    """New lengths and forks of a step: sequences begin, grow, end, go on from others."""
    origin = [-1] * SEQS
    if step == 7:
        origin[3] = 0                                          # (row 3 is empty until here)
    if step in (20, 30):
        origin[1] = 3 if step == 20 else 2
    new = [n + 1 for n in lens]
    if step < 7:
        new[3] = 0
    for b, a in enumerate(origin):
        if a >= 0 and lens[b] == 0:
            new[b] = lens[a] + 1
    if step in (19, 29):
        new[1] = 0
    if step == 25:
        new[0] = 3                                             # cut back into a page that row 3 holds too
    if step == 26:
        origin[0] = 0
    return new, origin


def test_steps_checked_call_by_call(q):
    p = Program(q, 0)
    book = S.Pages(p.table.tolist(), [0] * SEQS, [0] * 24, PAGE)
    context = [np.zeros((0, 2, HK, D))] * SEQS                   # what each sequence's cache holds, as read back before the step
    bf = lambda v: in_type(v, BF)  # noqa: E731
    seen = {}

    def look(what):
        torch.cuda.synchronize()
        w = 2.0 ** -8 * 1.01
        if what == "pages":
            book.compact()
            book.fork(p.origin.tolist())
            book.resize(p.new.tolist())
            assert (p.table.tolist(), p.lens.tolist(), p.refs.tolist()) == (book.table, book.lens, book.refs)
            seen["h"] = S.add(f64(p.delta), seen["h0"], bf)
        elif what == "norm in 8 bits":
            assert np.array_equal(f64(p.h), seen["h"])
            c, s = S.codes8(S.rms_norm(seen["h"], f64(p.norms[0]), 1e-6), 128)
            assert np.array_equal(p.codes.cpu().numpy(), c) and np.array_equal(f64(p.scales)[:, :SEQS], s.T)
        elif what in ("projection", "projection back"):
            if what == "projection":
                x, v, got = f64(p.codes) * np.repeat(f64(p.scales)[:, :SEQS].T, 128, 1), p.qkv_v, f64(p.qkv)
            else:
                x, v, got = f64(p.attn), p.o_v, f64(p.o)
            y, mag = S.product(x.reshape(SEQS, -1), v)
            assert np.all(np.abs(got.reshape(SEQS, -1) - y) <= w * np.abs(y) + 2.0 ** -13 * mag), what
            seen["qkv"] = f64(p.qkv)
        elif what == "attention":
            for b, n in enumerate(p.lens.tolist()):
                if n == 0:
                    assert not f64(p.attn)[b].any()
                    continue
                one = q.KvBatch(p.table[b:b + 1], p.lens[b:b + 1], n)
                k, v = (torch.empty((n, HK, D), dtype=BF, device="cuda") for _ in range(2))
                q.moe_kv_read(p.cache, one, k, v)
                # the new token's row is the turned projection to half a step of an 8-bit code of its block's scale
                turned = A.rotate(seen["qkv"][b:b + 1, HQ:HQ + HK], [n - 1], p.freqs)
                assert np.abs(f64(k)[-1] - turned[0]).max() <= 2.0 ** -4 * np.abs(turned).max() + 2.0 ** -7
                # the tokens before it are what they were, or rounded again where its block's scale grew
                old = context[p.origin.tolist()[b] if p.origin.tolist()[b] >= 0 and len(context[b]) == 0 else b]
                have = np.stack([f64(k), f64(v)], 1)
                m = min(len(old), n - 1)
                assert np.abs(have[:m] - old[:m]).max(initial=0) <= 2.0 ** -4 * np.abs(have).max()
                whole = m // 16 * 16
                assert np.array_equal(have[:whole], old[:whole])
                ref, rl, mag, smag = A.attention(f64(p.qkv)[b:b + 1, :HQ], f64(k), f64(v), np.ones((1, n), bool), D ** -0.5)
                check_attention(p.attn[b:b + 1], torch.from_numpy(rl).float(), ref, rl, *attention_bounds(BF, D, f64(v), ref, mag, smag, n), "attention")
                seen.setdefault("context", {})[b] = have
        elif what == "norm":
            h = S.add(f64(p.o), seen["h"], bf)
            assert np.array_equal(f64(p.h), h)
            y = S.rms_norm(h, f64(p.norms[1]), 1e-6)
            assert np.all(np.abs(f64(p.x) - y) <= (half_step(BF) + 2.0 ** -21) * np.abs(y) + 2.0 ** -130)
        else:
            ref, idx, _ = oracle_layer(p.wl, f64(p.x))
            assert np.array_equal(p.idx.cpu().numpy(), idx) and rel_err(p.delta.cpu().numpy(), ref).max() <= 2e-3

    for step in range(36):
        new, origin = plan(step, p.lens.tolist())
        p.new.copy_(i32(new))
        p.origin.copy_(i32(origin))
        seen.clear()
        seen["h0"] = f64(p.h)
        p.step(look)
        for b, have in seen.get("context", {}).items():
            context[b] = have
        for b, n in enumerate(p.lens.tolist()):
            context[b] = context[b][:n]
    assert p.lens.tolist()[3] == 36 - 0 and max(p.refs.tolist()) > 1


def test_captured_steps_give_the_same_bits(q):
    torch.cuda.synchronize()
    eager, other = Program(q, 1), Program(q, 1)
    graph = torch.cuda.CUDAGraph()
    before = other.state()
    with torch.cuda.graph(graph):
        other.step()
    for a, b in zip(before, other.state()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    for step in range(36):
        new, origin = plan(step, eager.lens.tolist())
        for p in (eager, other):
            p.new.copy_(i32(new))
            p.origin.copy_(i32(origin))
        if step % 2:
            eager.step()
        else:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                eager.step()
            torch.cuda.current_stream().wait_stream(side)
        graph.replay()
        for a, b in zip(eager.state(), other.state()):
            assert torch.equal(a, b), step
