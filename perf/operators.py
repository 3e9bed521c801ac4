"""Attention beside the routed experts, over a paged cache held in 8 bits:
what is timed, in plain form and as the library's calls.

A layer step is attention and then the expert FFN.  The four operators here
are the attention half:

  append   new q and k rows turned by their positions, the k and v rows
           written to the cache (moe_kv_append), and the rows the call wrote
           or rescaled read back as the values they stand for (moe_kv_read)
  read     the last n rows of each sequence out of the cache (moe_kv_read),
           as a prompt that is processed in chunks needs them
  decode   attention of a few new tokens of each sequence over its whole
           context in the cache (moe_attn_decode)
  prefill  attention of whole prompts or chunks of them, packed one after
           the other (moe_attn_prefill)

The cache (include/qmoe.h, "Attention") holds blocks of 16 tokens of one head:
e4m3 codes of K and of V and one scale for each, a power of two.

With `own` false everything is computed with elementary torch operations in
32 bits (angles in 64), with it true by the library.
"""
import math
import random

import torch

own = False

BLOCK = 16          # tokens that share a scale
E4M3_MAX = 448.0


# --------------------------------------------------------------------------
# Cases.  Sizes: chunks of 2048 and 8192 tokens, one token a step, drafts of
# up to three tokens, 4096 = 32 x 128 columns; the rest is generic.

def listed():
    return [
        # one user's generation: one token goes into the cache; launches and latency count
        _case("append_one", "append", batch=1, new=1, ctx=4097),
        # a server's step: 64 users with 1..3 drafted tokens each, narrow heads, part of the head turned in
        # neighbouring pairs, far positions with stretched frequencies; the last user's slot is empty
        _case("append_batch", "append", dtype="fp16", batch=64, new=3, ragged=True, ctx=8191, heads=32, kv_heads=4,
              dim=64, page=16, rot=32, pairs="neighbours", stretch=8.0),
        # the last chunk of an 8192-token prompt goes into the cache
        _case("append_chunk", "append", batch=1, new=2048, ctx=8192),
        # the context so far of one chunked prompt is read back
        _case("read_chunk", "read", batch=1, new=2048, ctx=2048),
        # contexts of a batch of odd lengths, narrow heads
        _case("read_packed", "read", dtype="fp16", batch=7, new=8191, ragged=True, ctx=8191, dim=64, page=16),
        # one user, a short odd context: the smallest attention call
        _case("decode_one", "decode", batch=1, new=1, ctx=777),
        # one user, a long context
        _case("decode_long", "decode", batch=1, new=1, ctx=131071, page=128),
        # a server's step over contexts of mixed lengths, one slot empty
        _case("decode_batch", "decode", dtype="fp16", batch=64, new=1, ragged=True, ctx=8192),
        # draft verification: 1..3 tokens of each of 16 users, 8 query heads to a key head
        _case("decode_draft", "decode", batch=16, new=3, ragged=True, ctx=4099, heads=64),
        # a short prompt of odd length
        _case("prefill_short", "prefill", batch=1, new=309, ctx=309),
        # the last 2048-token chunk of an 8192-token prompt
        _case("prefill_chunk", "prefill", batch=1, new=2048, ctx=8192),
        # prompts of mixed lengths packed into one call, narrow heads
        _case("prefill_packed", "prefill", dtype="fp16", batch=8, new=2048, ragged=True, ctx=2048, heads=32, kv_heads=4,
              dim=64),
    ]


def _case(name, op, dtype="bf16", batch=1, new=1, ragged=False, ctx=1, heads=32, kv_heads=8, dim=128, page=64, rot=None,
          pairs="halves", stretch=1.0, causal=True):
    c = {"name": name, "op": op, "dtype": dtype, "batch": batch, "new": new, "ragged": ragged, "ctx": ctx,
         "heads": heads, "kv_heads": kv_heads, "dim": dim}
    if op != "prefill":
        c["page"] = page
    else:
        c["causal"] = causal
    if op == "append":
        c |= {"rot": dim if rot is None else rot, "pairs": pairs, "stretch": stretch}
    return c


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("append", "read", "decode", "decode", "prefill", "prefill"))
    dim = rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 4, 8))
    heads = kv_heads * rng.choice((1, 3, 4, 8))
    kw = dict(dtype=rng.choice(("bf16", "fp16")), heads=heads, kv_heads=kv_heads, dim=dim, ragged=rng.random() < 0.6)
    if op == "prefill":
        new = _log(rng, 1, 2048)
        ctx = new if rng.random() < 0.5 else min(8192, new + _log(rng, 1, 6144))
        c = _case("", op, batch=max(1, min(_log(rng, 1, 16), 4096 // new)), new=new, ctx=ctx, causal=rng.random() < 0.8, **kw)
        most = 2.4e11                                                  # flops of the largest listed chunk
        if work(c)["flops"] > most and c["batch"] > 1:
            c["batch"] = max(1, int(c["batch"] * most / work(c)["flops"]))
        if work(c)["flops"] > most:
            c["heads"], c["kv_heads"] = max(1, c["heads"] // c["kv_heads"]), 1
    elif op == "decode":
        new = rng.randint(1, 16) if rng.random() < 0.4 else 1
        ctx = max(new, _log(rng, 1, 131071))
        c = _case("", op, batch=max(1, min(_log(rng, 1, 128), 262144 // ctx)), new=new, ctx=ctx, page=rng.choice((16, 32, 64, 128)), **kw)
    elif op == "read":
        ctx = _log(rng, 1, 16384)
        c = _case("", op, batch=max(1, min(_log(rng, 1, 64), 32768 // ctx)), new=_log(rng, 1, ctx), ctx=ctx, page=rng.choice((16, 32, 64, 128)), **kw)
    else:
        new = rng.randint(1, 3) if rng.random() < 0.5 else _log(rng, 1, 2048)
        c = _case("", op, batch=max(1, min(_log(rng, 1, 128), 4096 // new)), new=new, ctx=max(new, _log(rng, 1, 16384)),
                  page=rng.choice((16, 32, 64, 128)), rot=rng.choice((dim, dim // 2, 16, 0)),
                  pairs=rng.choice(("halves", "neighbours")), stretch=rng.choice((1.0, 4.0)), **kw)
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, context lengths) of the sequences; a ragged decoding batch of three or more ends in an empty slot."""
    B, new, ctx = case["batch"], case["new"], case["ctx"]
    if not case["ragged"]:
        return [new] * B, [ctx] * B
    rng = random.Random("%s %d %d %d" % (case["op"], B, new, ctx))
    ctxs = [ctx] + [rng.randint(max(1, ctx // 16), ctx) for _ in range(B - 1)]
    if case["op"] == "prefill" and ctx == new:
        news = list(ctxs)
    elif case["op"] == "read" and ctx == new:
        news = list(ctxs)
    else:
        news = [new] + [rng.randint(max(1, new // 16), new) for _ in range(B - 1)]
        news = [min(n, c) for n, c in zip(news, ctxs)]
    if B >= 3 and new <= 16 and case["op"] in ("append", "decode"):
        ctxs[-1], news[-1] = 0, 1
    return news, ctxs


_DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _starts(ns):
    s = [0]
    for n in ns:
        s.append(s[-1] + n)
    return s


# --------------------------------------------------------------------------
# Inputs.

def _freqs(case):
    """Angle a position of each pair, in 64 bits: 10000^(-2i/rot), stretched by parts (slow pairs by the factor, fast ones not)."""
    rot = case["rot"]
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    turns = 8192 * f / (2 * math.pi)
    keep = ((turns - 1.0) / 31.0).clamp(0, 1)
    return f * (keep + (1 - keep) / case["stretch"])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DTYPE[case["dtype"]]
    D, Hq, Hk, B = case["dim"], case["heads"], case["kv_heads"], case["batch"]
    news, ctxs = _lengths(case)
    cu = _starts(news)
    T = cu[-1]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    rows = lambda n, h: torch.randn((n, h, D), generator=g, device="cuda").to(dt)  # noqa: E731
    s = {"case": case, "B": B, "T": T, "D": D, "Hq": Hq, "Hk": Hk, "dt": dt, "scale": D ** -0.5, "max_new": max(news),
         "max_ctx": max(max(ctxs), 1), "cu": i32(cu)}
    if case["op"] == "prefill":
        cuk = _starts(ctxs)
        s |= {"q": rows(T, Hq), "k": rows(cuk[-1], Hk), "v": rows(cuk[-1], Hk), "cuk": i32(cuk), "causal": case["causal"],
              "out": torch.empty((T, Hq, D), dtype=dt, device="cuda"), "lse": torch.empty((T, Hq), device="cuda")}
        if own:
            from bit_quantized_moe_02_amd import qmoe
            s["ws"] = torch.empty(qmoe.moe_attn_prefill_workspace_bytes(T, B, s["max_new"], cuk[-1], Hq, Hk, D), dtype=torch.uint8, device="cuda")
        return s
    page = case["page"]
    per = -(-s["max_ctx"] // page)
    n_pages = sum(-(-c // page) for c in ctxs) + 2
    free = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    used, at = [], 0
    for c in ctxs:
        n = -(-c // page)
        used.append(torch.cat([free[at:at + n], torch.full((per - n,), -1, dtype=torch.int32, device="cuda")]))
        at += n
    s["table"] = torch.stack(used)
    s["lens"] = i32(ctxs)
    s["codes"] = torch.empty((n_pages, Hk, page // BLOCK, 2, BLOCK * D), dtype=torch.uint8, device="cuda")
    for c in s["codes"].split(max(1, (1 << 28) // max(1, s["codes"][0].numel()))):
        c.copy_((torch.randn(c.shape, generator=g, device="cuda") * 112).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8))
    s["scales"] = 2.0 ** torch.randint(-8, -5, (n_pages, Hk, page // BLOCK, 2), generator=g, device="cuda").float()
    if case["op"] == "append":
        back = [min(c, n + BLOCK - 1) for n, c in zip(news, ctxs)]
        cub = _starts(back)
        # q, k and v come out of one projection, side by side
        qkv = rows(T, Hq + 2 * Hk)
        s |= {"q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hk], "v": qkv[:, Hq + Hk:], "freqs": _freqs(case).cuda(), "rot": case["rot"],
              "neighbours": case["pairs"] == "neighbours", "cub": i32(cub), "Tb": cub[-1], "max_back": max(max(back), 1),
              "q_out": torch.empty((T, Hq, D), dtype=dt, device="cuda"), "k_out": torch.empty((T, Hk, D), dtype=dt, device="cuda")}
        s["rot_scale"] = 1.0 if case["stretch"] == 1.0 else 0.1 * math.log(case["stretch"]) + 1.0
    elif case["op"] == "read":
        s |= {"cub": s["cu"], "Tb": T, "max_back": max(news)}
    else:
        s |= {"q": rows(T, Hq), "out": torch.empty((T, Hq, D), dtype=dt, device="cuda"), "lse": torch.empty((T, Hq), device="cuda")}
    if "Tb" in s:
        s["k_back"] = torch.empty((s["Tb"], Hk, D), dtype=dt, device="cuda")
        s["v_back"] = torch.empty((s["Tb"], Hk, D), dtype=dt, device="cuda")
    if own:
        from bit_quantized_moe_02_amd import qmoe
        s["cache"] = qmoe.KvCache(s["codes"], s["scales"], page, Hk, D)
        uniform = not case["ragged"]
        s["step"] = qmoe.KvBatch(s["table"], s["lens"], T, s["max_new"], None if uniform else s["cu"])
        if "Tb" in s:
            s["back"] = qmoe.KvBatch(s["table"], s["lens"], s["Tb"], s["max_back"], s["cub"])
        if case["op"] == "append":
            s["rope"] = qmoe.Rope(s["freqs"], s["rot"], s["neighbours"], s["rot_scale"])
        if case["op"] == "decode":
            s["ws"] = torch.empty(qmoe.moe_attn_decode_workspace_bytes(s["cache"], s["step"], Hq), dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------------------
# One pass.

def run(s):
    return (_run_own if own else _run_plain)(s, s["case"]["op"])


def _run_own(s, op):
    from bit_quantized_moe_02_amd import qmoe
    if op == "prefill":
        qmoe.moe_attn_prefill(s["q"], s["k"], s["v"], s["cu"], s["cuk"], s["max_new"], s["out"], s["ws"], s["scale"], s["causal"], s["lse"])
        return s["out"], s["lse"]
    if op == "decode":
        qmoe.moe_attn_decode(s["cache"], s["step"], s["q"], s["out"], s["ws"], s["scale"], s["lse"])
        return s["out"], s["lse"]
    if op == "append":
        qmoe.moe_kv_append(s["cache"], s["step"], s["k"], s["v"], s["rope"], s["q"], s["q_out"], s["k_out"])
    qmoe.moe_kv_read(s["cache"], s["back"], s["k_back"], s["v_back"])
    return (s["q_out"], s["k_out"], s["k_back"], s["v_back"]) if op == "append" else (s["k_back"], s["v_back"])


def _run_plain(s, op):
    if op == "prefill":
        return _plain_prefill(s)
    if op == "decode":
        return _plain_decode(s)
    if op == "read":
        return _plain_read(s)
    q, k = _plain_append(s)
    return (q, k) + _plain_read(s)


# ---- the cache's layout, as plain indexing

def _k_rows(codes, D):
    """[..., 16*D] codes of K blocks to [..., 16, D]: 64 columns a piece, (8-column group g, token n, column half a, j)."""
    lead = codes.shape[:-1]
    x = codes.view(*lead, D // 64, 4, BLOCK, 2, 8)                     # h g n a j
    n = len(lead)
    return x.permute(*range(n), n + 2, n, n + 3, n + 1, n + 4).reshape(*lead, BLOCK, D)


def _k_codes(rows, D):
    lead = rows.shape[:-2]
    n = len(lead)
    x = rows.reshape(*lead, BLOCK, D // 64, 2, 4, 8)                   # n h a g j
    return x.permute(*range(n), n + 1, n + 3, n, n + 2, n + 4).reshape(*lead, BLOCK * D)


def _v_rows(codes, D):
    """[..., 16*D] codes of V blocks to [..., 16, D]: (piece h, token group g, column c, 16-column tile w, token i)."""
    lead = codes.shape[:-1]
    x = codes.view(*lead, D // 64, 4, 16, 4, 4)                        # h g c w i
    n = len(lead)
    return x.permute(*range(n), n + 1, n + 4, n, n + 3, n + 2).reshape(*lead, BLOCK, D)


def _v_codes(rows, D):
    lead = rows.shape[:-2]
    n = len(lead)
    x = rows.reshape(*lead, 4, 4, D // 64, 4, 16)                      # g i h w c
    return x.permute(*range(n), n + 2, n, n + 4, n + 3, n + 1).reshape(*lead, BLOCK * D)


def _blocks(s, at):
    """Page, block in the page of token positions `at` [B, N]; positions that no page holds give page 0."""
    page = s["case"]["page"]
    at = at.clamp(min=0)
    slot = (at // page).clamp(max=s["table"].shape[1] - 1)
    return s["table"].gather(1, slot).long().clamp(min=0), at % page // BLOCK


def _spread(s, cu, most):
    """Sequence and index in it of each packed row."""
    t = torch.arange(cu.shape[0] - 1, device=cu.device).repeat_interleave((cu[1:] - cu[:-1]).long(), output_size=int(most))
    return t, torch.arange(int(most), device=cu.device) - cu[t]


# ---- append

def _plain_turn(s, x, pos):
    rot = s["rot"]
    if not rot:
        return x.float()
    turns = pos.double()[:, None] * (s["freqs"] / (2 * math.pi))
    angle = (turns - turns.floor()) * (2 * math.pi)
    cos, sin = (f(angle).float()[:, None] * s["rot_scale"] for f in (torch.cos, torch.sin))
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["neighbours"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * cos - b * sin, a * sin + b * cos
    return torch.cat([torch.stack([a, b], -1).flatten(-2) if s["neighbours"] else torch.cat([a, b], -1), x[..., rot:]], -1)


def _least_scale(amax):
    """Least power of two with amax <= 448 of it, not below 2^-64."""
    m, e = torch.frexp(amax)                                          # amax = m 2^e, m in [0.5, 1)
    e = e - 9 + (m > 0.875).int()                                     # 448 = 0.875 * 2^9
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, torch.full_like(e, -64)).clamp(min=-64))


def _plain_append(s):
    D, Hk, dt = s["D"], s["Hk"], s["dt"]
    cu, lens = s["cu"].long(), s["lens"].long()
    n = cu[1:] - cu[:-1]
    seq, i = _spread(s, cu, s["T"])
    pos = (lens - n)[seq] + i
    q, k = _plain_turn(s, s["q"], pos), _plain_turn(s, s["k"], pos)
    first = (lens - n).clamp(min=0)                                    # first position written
    nb = (s["max_new"] + 2 * BLOCK - 2) // BLOCK                       # blocks a sequence can touch
    blk = first[:, None] // BLOCK + torch.arange(nb, device=cu.device)
    at = blk[..., None] * BLOCK + torch.arange(BLOCK, device=cu.device)  # [B, nb, 16] positions
    new = (at >= first[:, None, None]) & (at < lens[:, None, None])
    row = (at - (lens - n)[:, None, None] + cu[:-1, None, None]).clamp(0, s["T"] - 1)
    touched = new.any(-1)
    page, b = _blocks(s, blk * BLOCK)
    codes, scales = s["codes"][page, :, b], s["scales"][page, :, b]    # [B, nb, Hk, 2, 16 D], [B, nb, Hk, 2]
    old = (at < first[:, None, None]) & touched[..., None]
    for part, x, to_rows, to_codes in ((0, k, _k_rows, _k_codes), (1, s["v"].float(), _v_rows, _v_codes)):
        put = x[row].transpose(2, 3)                                   # [B, nb, Hk, 16, D]
        amax = put.abs().amax(-1).masked_fill(~new[:, :, None], 0).amax(-1)
        was = torch.where(old.any(-1)[..., None], scales[..., part], torch.zeros_like(amax))
        now = torch.maximum(was, _least_scale(amax))
        held = to_rows(codes[..., part, :].contiguous(), D)
        kept = held.view(torch.float8_e4m3fn).float() * (was / now)[..., None, None]
        val = torch.where(new[:, :, None, :, None], put / now[..., None, None], kept)
        bits = torch.where((new | old)[:, :, None, :, None], val.to(torch.float8_e4m3fn).view(torch.uint8), held)
        t = touched.nonzero(as_tuple=True)
        s["codes"][page[t], :, b[t], part] = to_codes(bits, D)[t]
        s["scales"][page[t], :, b[t], part] = now[t]
    return q.to(dt), k.to(dt)


# ---- read

def _plain_values(s, page, b):
    """K and V of blocks in 32 bits: [..., Hk, 16, D] each."""
    codes, scales = s["codes"][page, :, b], s["scales"][page, :, b]
    return tuple(rows(codes[..., i, :].contiguous(), s["D"]).view(torch.float8_e4m3fn).float() * scales[..., i, None, None]
                 for i, rows in ((0, _k_rows), (1, _v_rows)))


def _plain_read(s):
    cu, lens = s["cub"].long(), s["lens"].long()
    seq, i = _spread(s, cu, s["Tb"])
    pos = lens[seq] - (cu[1:] - cu[:-1])[seq] + i
    nb = (s["max_back"] + 2 * BLOCK - 2) // BLOCK
    base = (lens - (cu[1:] - cu[:-1])).clamp(min=0) // BLOCK
    page, b = _blocks(s, (base[:, None] + torch.arange(nb, device=cu.device)) * BLOCK)
    K, V = (x.transpose(2, 3).flatten(1, 2) for x in _plain_values(s, page, b))      # [B, nb*16, Hk, D]
    off = pos - base[seq] * BLOCK
    return K[seq, off].to(s["dt"]), V[seq, off].to(s["dt"])


# ---- attention

def _plain_attend(q, k, v, keep, scale):
    """q [B, Hk, R, D], k and v [B, Hk, L, D], keep [B, 1, R, L]: outputs and log sums; rows that keep nothing give 0 and -inf."""
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(~keep, -math.inf)
    m = p.amax(-1, keepdim=True)
    p = p.sub_(m.masked_fill(m == -math.inf, 0)).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / total.masked_fill(total == 0, 1), (m + total.log()).squeeze(-1)


def _plain_packed(s, k, v, length, causal):
    """Attention of packed q rows, padded to [B, Hk, group * max_new, D], over padded keys [B, Hk, L, D] of `length` each."""
    B, Hk, D, N = s["B"], s["Hk"], s["D"], s["max_new"]
    G, L = s["Hq"] // Hk, k.shape[2]
    cu = s["cu"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(N, device=cu.device)
    q = s["q"].float()[(cu[:-1, None] + i).clamp(max=s["T"] - 1)]                      # [B, N, Hq, D]
    q = q.view(B, N, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * N, D)
    j = torch.arange(L, device=cu.device)
    last = (length - n)[:, None] + i if causal else (length - 1)[:, None].expand(B, N)
    keep = (j <= last[..., None]) & (j < length[:, None, None])                        # [B, N, L]
    keep = keep[:, None, None].expand(B, 1, G, N, L).reshape(B, 1, G * N, L)
    o, lse = _plain_attend(q, k, v.masked_fill(~(j < length[:, None])[:, None, :, None], 0), keep, s["scale"])
    seq, i = _spread(s, cu, s["T"])
    o = o.view(B, Hk, G, N, D).permute(0, 3, 1, 2, 4).reshape(B, N, s["Hq"], D)
    lse = lse.view(B, Hk, G, N).permute(0, 3, 1, 2).reshape(B, N, s["Hq"])
    return o[seq, i].to(s["dt"]), lse[seq, i]


def _plain_decode(s):
    nb = -(-s["max_ctx"] // BLOCK)
    at = (torch.arange(nb, device="cuda") * BLOCK).expand(s["B"], nb)
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in _plain_values(s, *_blocks(s, at)))
    return _plain_packed(s, k, v, s["lens"].long(), True)


def _plain_prefill(s):
    cu = s["cuk"].long()
    j = (cu[:-1, None] + torch.arange(s["max_ctx"], device=cu.device)).clamp(max=s["k"].shape[0] - 1)
    k, v = (x.float()[j].transpose(1, 2) for x in (s["k"], s["v"]))
    return _plain_packed(s, k, v, cu[1:] - cu[:-1], s["causal"])


# --------------------------------------------------------------------------
# What a pass cannot do without.

def work(case):
    news, ctxs = _lengths(case)
    D, Hq, Hk = case["dim"], case["heads"], case["kv_heads"]
    T = sum(news)
    if case["op"] == "append":
        read = sum(min(c, n + BLOCK - 1) for n, c in zip(news, ctxs))
        rows = T * 2 * D * 2 * (Hq + Hk) + T * D * 2 * Hk + T * 2 * Hk * D             # q, k in and out, v in, codes out
        return {"bytes": rows + read * Hk * D * 2 * 3, "flops": 3 * T * (Hq + Hk) * case["rot"] + 4 * T * Hk * D}
    if case["op"] == "read":
        return {"bytes": T * Hk * D * 2 * 3 + T * Hk // 2, "flops": 2 * T * Hk * D}
    causal = case["op"] == "decode" or case["causal"]
    pairs = sum(n * c - n * (n - 1) // 2 if causal else n * c for n, c in zip(news, ctxs) if c >= n)
    flops = 4 * pairs * Hq * D
    io = T * Hq * (4 * D + 4)
    if case["op"] == "decode":
        return {"bytes": io + sum(ctxs) * Hk * 2 * D + sum(-(-c // BLOCK) for c in ctxs) * Hk * 8, "flops": flops}
    return {"bytes": io + sum(ctxs) * Hk * 4 * D, "flops": flops}


# --------------------------------------------------------------------------
# The definitions in 64 bits, sequence by sequence.

def _e4m3(x):
    """Nearest value of the 8-bit format (4 exponent bits, 3 of mantissa, ties to even) to 64-bit x, |x| <= 448."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return torch.round(x / step) * step


def _decode8(bits):
    b = bits.long()
    sign, e, m = 1 - 2 * (b >> 7), (b >> 3) & 15, b & 7
    mant = torch.where(e == 0, m, m + 8).double()
    return sign * torch.ldexp(mant, e.clamp(min=1) - 10)


def _fetch(s, b, lo, hi):
    """Codes' values and scales of positions lo..hi-1 of sequence b: ([n, Hk, D], [n, Hk]) of K, then of V."""
    D, page = s["D"], s["case"]["page"]
    p = torch.arange(lo, hi, device="cuda")
    pg = s["table"][b].long()[p // page]
    blk, n = p % page // BLOCK, p % BLOCK
    d = torch.arange(D, device="cuda")
    at_k = 1024 * (d // 64) + 256 * (d % 32 // 8) + 8 * (d % 64 // 32) + d % 8 + 16 * n[:, None]
    at_v = 1024 * (d // 64) + 16 * (d % 16) + 4 * (d % 64 // 16) + (256 * (n // 4) + n % 4)[:, None]
    got = []
    for part, at in ((0, at_k), (1, at_v)):
        c = s["codes"][pg, :, blk, part]                                # [n, Hk, 16 D]
        got += [_decode8(c.gather(-1, at[:, None].expand(-1, s["Hk"], -1))), s["scales"][pg, :, blk, part].double()]
    return got


def exact(case, seed):
    news, ctxs = _lengths(case)
    w = work(case)
    if w["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    if case["op"] in ("decode", "prefill"):
        return _exact_attention(s, case, news, ctxs)
    qs, ks, kb, vb = [], [], [], []
    cu = _starts(news)
    for b, (n, c) in enumerate(zip(news, ctxs)):
        if case["op"] == "read":
            K, ks_, V, vs_ = _fetch(s, b, c - n, c)
            kb.append(K * ks_[..., None])
            vb.append(V * vs_[..., None])
            continue
        pos = torch.arange(c - n, c, device="cuda").double()
        rows = slice(cu[b], cu[b + 1])
        for src, to in ((s["q"], qs), (s["k"], ks)):
            x = src[rows].double()
            y = x.clone()
            for i in range(case["rot"] // 2):
                u, v = (2 * i, 2 * i + 1) if s["neighbours"] else (i, i + case["rot"] // 2)
                a = (pos * s["freqs"][i])[:, None]
                y[..., u] = (x[..., u] * a.cos() - x[..., v] * a.sin()) * s["rot_scale"]
                y[..., v] = (x[..., u] * a.sin() + x[..., v] * a.cos()) * s["rot_scale"]
            to.append(y)
        if c == 0:
            continue
        lo = (c - n) // BLOCK * BLOCK
        before = _fetch(s, b, lo, c - n) if c - n > lo else None
        back = min(c, n + BLOCK - 1)
        for part, x, to in ((0, ks[-1], kb), (1, s["v"][rows].double(), vb)):
            vals = torch.empty((c - lo, s["Hk"], s["D"]), dtype=torch.float64, device="cuda")
            for at in range(lo, c, BLOCK):
                end, start = min(at + BLOCK, c), max(at, c - n)
                fresh = x[start - (c - n):end - (c - n)]
                amax = fresh.abs().amax((0, 2))
                m, e = torch.frexp(amax / E4M3_MAX)
                scale = torch.ldexp(torch.ones_like(amax), torch.where(m == 0.5, e - 1, e).clamp(min=-64))
                scale = torch.where(amax == 0, 2.0 ** -64, scale)
                if start > at:
                    codes, was = before[2 * part], before[2 * part + 1]
                    scale = torch.maximum(scale, was[0])
                    vals[:start - at] = _e4m3(codes * (was[0] / scale)[:, None]) * scale[:, None]
                vals[start - lo:end - lo] = _e4m3(fresh / scale[:, None]) * scale[:, None]
            if c - back < lo:
                K, a, V, v = _fetch(s, b, c - back, lo)
                vals = torch.cat([(V if part else K) * (v if part else a)[..., None], vals])
            to.append(vals[-back:])
    if case["op"] == "read":
        return torch.cat(kb), torch.cat(vb)
    return torch.cat(qs), torch.cat(ks), torch.cat(kb), torch.cat(vb)


def _exact_attention(s, case, news, ctxs):
    G, Hk = s["Hq"] // s["Hk"], s["Hk"]
    cu, cuk = _starts(news), _starts(ctxs)
    outs, lses = [], []
    for b, (n, c) in enumerate(zip(news, ctxs)):
        q = s["q"][cu[b]:cu[b + 1]].double()
        o = torch.zeros_like(q)
        lse = torch.full((n, s["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
        if c:
            if case["op"] == "decode":
                K, a, V, v = _fetch(s, b, 0, c)
                K, V = K * a[..., None], V * v[..., None]
            else:
                K, V = (s[x][cuk[b]:cuk[b + 1]].double() for x in ("k", "v"))
            seen = torch.arange(c, device="cuda") <= (torch.arange(n, device="cuda") + c - n)[:, None]
            if case["op"] == "prefill" and not case["causal"]:
                seen[:] = True
            for h in range(Hk):
                for i in range(h * G, h * G + G):
                    z = torch.where(seen, q[:, i] @ K[:, h].T * s["scale"], -math.inf)
                    lse[:, i] = torch.logsumexp(z, -1)
                    o[:, i] = torch.where(seen, (z - lse[:, i, None]).exp(), 0.0) @ V[:, h]
        outs.append(o)
        lses.append(lse)
    return torch.cat(outs), torch.cat(lses)
