"""The operators around an 8-bit paged cache: rotary positions, the quantising write with its read back,
decode attention over the 8-bit cache, and decode attention with a sliding window and sinks.

``run`` computes them in their plain form (elementary torch operations) while ``own`` is false, and through
the entry points of ``long_context_layer_b200`` while it is true.

Definitions
-----------
Cache: pages of 16 tokens; a block is one (page, KV head) of K or of V.  A block holds 16 x D 8-bit values and
one scale s = 2^e, e the smallest integer >= -100 with max|x| <= QMAX * s (QMAX 448 for e4m3, 127 for int8);
a value stands for payload * s.  Writing tokens into a block that holds older tokens keeps the larger of the
block's scale and the new tokens', and rounds the older values to the new scale when it grew.
Attention: o = sum_t softmax_t(q.k_t / sqrt(D)) v_t over the visible tokens, 0 without any; query head h reads
KV head h // G.
"""
import math

import torch

own = False

PAGE = 16
LOG2_MIN = -100
QMAX = {"e4m3": 448.0, "int8": 127.0}
PAYLOAD = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of one sequence: the smallest call of the rotary operator
        dict(name="rope step", op="rope", rows=1, hq=28, hkv=4, d=128, rd=128, dtype="bf16", layout="half",
             scaling="none", factor=1.0, first=8191),
        # a long prompt, half of each head rotated, adjacent pairs, stretched to eight times its context
        dict(name="rope prompt", op="rope", rows=32768, hq=32, hkv=8, d=128, rd=64, dtype="bf16",
             layout="interleaved", scaling="bands", factor=8.0, first=0),
        # the token each of 16 sequences appends in one layer of a decode step, and its page read back
        dict(name="cache append", op="cache", batch=16, hkv=8, d=128, dtype="bf16", fmt="e4m3", have=16384, new=1,
             ragged=False),
        # the prompts of 4 sequences written at once and read back
        dict(name="cache prompt", op="cache", batch=4, hkv=8, d=128, dtype="bf16", fmt="e4m3", have=0, new=16384,
             ragged=False),
        # prompt chunks of uneven lengths that start inside a page
        dict(name="cache chunks", op="cache", batch=7, hkv=1, d=64, dtype="f32", fmt="int8", have=1003, new=2501,
             ragged=True),
        # full layer, one sequence: latency
        dict(name="full 8k", op="full", batch=1, hq=28, hkv=4, d=128, dtype="bf16", fmt="e4m3", ctx=8192,
             ragged=False),
        # full layer, long contexts: bandwidth
        dict(name="full 64k", op="full", batch=4, hq=32, hkv=8, d=128, dtype="bf16", fmt="int8", ctx=65536,
             ragged=False),
        # delta-layer: attention, page scores and the page selection
        dict(name="select 16k", op="select", batch=16, hq=40, hkv=8, d=128, dtype="bf16", fmt="e4m3", ctx=16385,
             ragged=False, budget=128, sink=16, recency=512),
        # sparse layer: the selected pages only
        dict(name="sparse 16k", op="sparse", batch=16, hq=40, hkv=8, d=128, dtype="bf16", fmt="int8", ctx=16385,
             ragged=False, budget=128, sink=16, recency=512),
        # window layer of one sequence
        dict(name="window 1k", op="window", batch=1, hq=28, hkv=4, d=128, dtype="bf16", fmt="none", ctx=8192,
             ragged=False, window=1024, sink=16),
        # window layer of a batch
        dict(name="window 4k", op="window", batch=16, hq=40, hkv=8, d=128, dtype="bf16", fmt="none", ctx=32768,
             ragged=True, window=4096, sink=16),
        # window over the 8-bit cache, odd window, uneven lengths (an empty and a one-token sequence among them)
        dict(name="window 8-bit", op="window", batch=9, hq=8, hkv=1, d=64, dtype="f32", fmt="e4m3", ctx=20011,
             ragged=True, window=1001, sink=5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    hq, hkv, d = rng.choice([(28, 4, 128), (32, 8, 128), (40, 8, 128), (8, 1, 64), (6, 2, 64), (3, 3, 128),
                             (16, 2, 128)])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    op = rng.choice(["rope", "cache", "full", "select", "sparse", "window", "window"])
    if op == "rope":
        scaling = rng.choice(["none", "linear", "bands"])
        return dict(op=op, rows=_log(rng, 1, 16384), hq=hq, hkv=hkv, d=d, rd=2 * rng.randint(1, d // 2), dtype=dtype,
                    layout=rng.choice(["half", "interleaved"]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]),
                    first=_log(rng, 1, 1000000) - 1)
    if op == "cache":
        batch = rng.randint(1, 16)
        return dict(op=op, batch=batch, hkv=hkv, d=d, dtype=dtype, fmt=rng.choice(["e4m3", "int8"]),
                    have=_log(rng, 1, 4096) - 1, new=_log(rng, 1, 32768 // batch), ragged=rng.random() < 0.5)
    batch = rng.randint(1, 16)
    ctx = _log(rng, 1, min(65536, 4 * 65536 // batch))
    fmt = rng.choice(["e4m3", "int8"])
    case = dict(op=op, batch=batch, hq=hq, hkv=hkv, d=d, dtype=dtype, fmt=fmt, ctx=ctx, ragged=rng.random() < 0.5)
    if op == "window":
        case["fmt"] = rng.choice(["none", "none", "e4m3", "int8"])
        case["ctx"] = _log(rng, 1, 32768)
        case.update(window=_log(rng, 1, 8192), sink=rng.choice([0, 1, 4, 16, 37, 128]))
    elif op != "full":
        case.update(budget=_log(rng, 1, 256), sink=rng.choice([0, 1, 16, 40]), recency=rng.choice([0, 64, 250, 512]))
    return case


# ---------------------------------------------------------------------------------------------- inputs
def _lengths(case):
    """Tokens of each sequence: all `ctx`, or uneven with an empty and a one-token sequence where there are four."""
    b, n = case["batch"], case["ctx"]
    if not case["ragged"]:
        return [n] * b
    got = torch.randint(1, n + 1, (b,), generator=torch.Generator().manual_seed(n + b)).tolist()
    got[0] = n
    if b >= 4:
        got[1], got[2] = 0, 1
    return got


def _frequencies(case):
    """Turns per token of each rotated pair, in 64 bits, and the magnitude of the rotation."""
    rd, factor = case["rd"], case["factor"]
    f = 10000.0 ** (-torch.arange(0, rd, 2, dtype=torch.float64) / rd) / (2 * math.pi)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "bands":  # pairs of few turns over the original context are stretched, of many kept
        keep = ((f * 4096.0 - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return f / factor * (1 - keep) + f * keep, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _block_scale(amax, fmt):
    """2^e, e the smallest integer >= -100 with amax <= QMAX * 2^e."""
    m, x = torch.frexp(amax)  # amax = m * 2^x, 0.5 <= m < 1
    top, shift = (0.875, 9) if fmt == "e4m3" else (0.9921875, 7)  # QMAX = top * 2^shift
    e = torch.where(amax > 0, x - shift + (m > top).int(), torch.full_like(x, LOG2_MIN)).clamp_min(LOG2_MIN)
    return ((e.int() + 127) << 23).view(torch.float32)


def _round8(y, fmt):
    """Payload bytes of scaled values."""
    q = y.to(torch.float8_e4m3fn) if fmt == "e4m3" else y.round().to(torch.int8)
    return q.view(torch.uint8)


def _values(payload, scale, fmt):
    """Blocks [..., 16, D] of bytes and their scales [...] as the numbers they stand for, in 32 bits."""
    return payload.view(PAYLOAD[fmt]).float() * scale[..., None, None]


def _normal(shape, gen, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda") * std


def _pool(pages, case, gen):
    """[pages, Hkv, 16, D] values as a cache holds them: normal, some channels and some pages larger."""
    hkv, d = case["hkv"], case["d"]
    x = _normal((pages, hkv, PAGE, d), gen)
    x *= torch.exp(0.3 * _normal((pages, hkv, 1, 1), gen))
    return x


def _store(x, case):
    """The values as the case's cache stores them: (payload, scale), or (values, None)."""
    if case["fmt"] == "none":
        return x.to(DTYPE[case["dtype"]]), None
    s = _block_scale(x.abs().amax(dim=(2, 3)), case["fmt"])
    return _round8(x / s[..., None, None], case["fmt"]), s


def _page_table(lens, gen):
    """CSR page table over a pool with a few spare pages: (indptr, indices, kv_len, pages, longest)."""
    n_pages = [-(-n // PAGE) for n in lens]
    pages = sum(n_pages) + 3
    perm = torch.randperm(pages, generator=gen)[:sum(n_pages)]
    indptr = torch.tensor([0] + torch.tensor(n_pages).cumsum(0).tolist(), dtype=torch.int32)
    return indptr.cuda(), torch.cat([perm, perm.new_zeros(1)]).int().cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), \
        pages, max(1, max(n_pages))


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case=case)
    dt = DTYPE[case["dtype"]]
    if case["op"] == "rope":
        turns, magnitude = _frequencies(case)
        rows = case["rows"]
        pos = torch.arange(rows, dtype=torch.int32) + case["first"] + int(torch.randint(0, 64, (1,), generator=host))
        st.update(turns=turns.cuda(), magnitude=magnitude, positions=pos.cuda(),
                  q=_normal((rows, case["hq"], case["d"]), gen).to(dt),
                  k=_normal((rows, case["hkv"], case["d"]), gen).to(dt))
    elif case["op"] == "cache":
        b, hkv, d = case["batch"], case["hkv"], case["d"]
        new, have = [case["new"]] * b, [case["have"]] * b
        if case["ragged"]:
            sizes = torch.Generator().manual_seed(case["new"] + b)
            new = [case["new"]] + torch.randint(0, case["new"] + 1, (b - 1,), generator=sizes).tolist()
            have = torch.randint(0, case["have"] + 1, (b,), generator=sizes).tolist()
        lens = [x + y for x, y in zip(have, new)]
        indptr, indices, kv_len, pages, longest = _page_table(lens, host)
        k, ks = _store(_pool(pages, case, gen), case)
        v, vs = _store(_pool(pages, case, gen), case)
        starts = [(x - x % PAGE) if m else x for x, m in zip(have, new)]  # read back from the first page written
        reads = [x + m - s for x, m, s in zip(have, new, starts)]
        cum = lambda v: torch.tensor([0] + torch.tensor(v).cumsum(0).tolist(), dtype=torch.int32).cuda()  # noqa: E731
        t, tr = sum(new), sum(reads)
        st.update(indptr=indptr, indices=indices, kv_len=kv_len, pages=pages, longest=longest, k=k, ks=ks, v=v, vs=vs,
                  tokens=cum(new), most=max(new), reads=cum(reads), most_read=max(reads),
                  starts=torch.tensor(starts, dtype=torch.int32).cuda(),
                  k_new=(_normal((t, hkv, d), gen, 1.5)).to(dt), v_new=(_normal((t, hkv, d), gen, 1.5)).to(dt),
                  k_out=torch.zeros((tr, hkv, d), dtype=dt, device="cuda"),
                  v_out=torch.zeros((tr, hkv, d), dtype=dt, device="cuda"))
    else:
        lens = _lengths(case)
        indptr, indices, kv_len, pages, longest = _page_table(lens, host)
        b, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]
        q = _normal((b, hq, d), gen).to(dt)
        x = _pool(pages, case, gen)
        st.update(indptr=indptr, indices=indices, kv_len=kv_len, pages=pages, longest=longest, q=q,
                  o=torch.zeros((b, hq, d), dtype=dt, device="cuda"))
        if case["op"] in ("select", "sparse"):
            _plan_selection(st, case, lens, x, host)
        st["k"], st["ks"] = _store(x, case)
        del x
        st["v"], st["vs"] = _store(_pool(pages, case, gen), case)
    if own:
        _handles(st, case)
    return st


def _kept(n, case):
    """(pages, sink pages, first recency page) of a context of n tokens."""
    pages = -(-n // PAGE)
    sink = min(pages, -(-case["sink"] // PAGE))
    first = max(n - case["recency"], 0) // PAGE if case["recency"] and n else pages
    return pages, sink, max(first, sink)


def _plan_selection(st, case, lens, x, host):
    """As many pages as the budget takes hold keys near the queries (passages that the step asks for), and a
    sparse layer attends to those, the sink and the recent pages."""
    b, hkv, d = case["batch"], case["hkv"], case["d"]
    toward = st["q"].float().view(b, hkv, -1, d).mean(2)
    toward = toward / toward.norm(dim=-1, keepdim=True)
    stride = case["budget"] + -(-case["sink"] // PAGE) + (-(-case["recency"] // PAGE) + 1 if case["recency"] else 0)
    stride = max(stride, 1)
    cnt, sel = [], torch.full((b, stride), -1, dtype=torch.int32)
    offset, table = st["indptr"].tolist(), st["indices"].cpu()
    for i, n in enumerate(lens):
        pages, sink, first = _kept(n, case)
        middle = torch.arange(sink, first)
        picked = middle[torch.randperm(len(middle), generator=host)[: case["budget"]]]
        phys = table[offset[i] + picked].long().cuda()
        x[phys] = 0.5 * x[phys] + 4.0 * toward[i][None, :, None, :]
        keep = torch.cat([torch.arange(0, sink), picked, torch.arange(first, pages)]).sort().values
        cnt.append(len(keep))
        sel[i, : len(keep)] = keep.int()
    if case["op"] == "sparse":
        st.update(sel_cnt=torch.tensor(cnt, dtype=torch.int32).cuda(), sel_pages=sel.cuda(), stride=stride)
    else:
        st.update(sel_cnt=torch.zeros(b, dtype=torch.int32).cuda(), sel_pages=torch.full_like(sel, -1).cuda(),
                  stride=stride, scores=torch.zeros((b, st["longest"]), device="cuda"))


def _handles(st, case):
    """What a program that uses the framework keeps next to its buffers: descriptors and a workspace."""
    import long_context_layer_b200 as L
    dt = L.DELTA_BF16 if case["dtype"] == "bf16" else L.DELTA_F32
    st["L"] = L
    if case["op"] == "rope":
        st["desc"] = L.DeltaDesc(case["hq"], case["hkv"], case["d"], PAGE, dt, 0.0, 0)
        st["rope"] = L.DeltaRope(st["turns"].data_ptr(), case["rd"],
                                 L.DELTA_ROPE_HALF if case["layout"] == "half" else L.DELTA_ROPE_INTERLEAVED,
                                 st["magnitude"], st["positions"].data_ptr(), case["rows"], 0)
        return
    st["desc"] = L.DeltaDesc(case.get("hq", case["hkv"]), case["hkv"], case["d"], PAGE, dt, 0.0, st["pages"])
    st["pt"] = L.DeltaPageTable(st["indptr"].data_ptr(), st["indices"].data_ptr(), st["kv_len"].data_ptr(), case["batch"],
                                st["longest"])
    if case["fmt"] != "none":
        st["cache"] = L.DeltaQ8Cache(st["k"].data_ptr(), st["v"].data_ptr(), st["ks"].data_ptr(), st["vs"].data_ptr(),
                                     L.DELTA_E4M3 if case["fmt"] == "e4m3" else L.DELTA_INT8)
    if case["op"] == "cache":
        return
    size = L.workspace_size if case["fmt"] == "none" else L.workspace_size_q8
    st["bytes"] = size(st["desc"], case["batch"], st["longest"])
    st["ws"] = torch.empty(st["bytes"], dtype=torch.uint8, device="cuda")
    L.workspace_init(st["ws"], st["bytes"], torch.cuda.current_stream().cuda_stream)
    if case["op"] == "select":
        st["sp"] = L.DeltaSelectParams(case["budget"], case["sink"], case["recency"], L.DELTA_HEAD_SUM)


# ---------------------------------------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        return _run_own(st, case, op)
    if op == "rope":
        return _plain_rope(st, case)
    if op == "cache":
        return _plain_cache(st, case)
    if op == "window":
        return _plain_window(st, case)
    if op == "sparse":
        return _plain_sparse(st, case)
    return _plain_full(st, case)


def _run_own(st, case, op):
    L, s = st["L"], torch.cuda.current_stream().cuda_stream
    if op == "rope":
        q, k = torch.empty_like(st["q"]), torch.empty_like(st["k"])
        L.rope(st["desc"], st["rope"], case["rows"], st["q"], q, st["k"], k, stream=s)
        return [q, k]
    d, pt = st["desc"], st["pt"]
    if op == "cache":
        if case["new"] == 1 and not case["ragged"]:
            L.kv_append_q8(d, pt, st["k_new"], st["v_new"], st["cache"], s)
        else:
            L.kv_write_q8(d, pt, st["tokens"], st["most"], st["k_new"], st["v_new"], st["cache"], stream=s)
        L.kv_read_q8(d, pt, st["reads"], st["most_read"], st["starts"], st["cache"], st["k_out"], st["v_out"], s)
        return [st["k_out"], st["v_out"], st["ks"], st["vs"]]
    if op == "window":
        if case["fmt"] == "none":
            L.window_attn(d, pt, case["window"], case["sink"], st["q"], st["k"], st["v"], st["o"], st["ws"], st["bytes"], s)
        else:
            L.window_attn_q8(d, pt, case["window"], case["sink"], st["q"], st["cache"], st["o"], st["ws"], st["bytes"], s)
        return [st["o"]]
    if op == "full":
        L.full_attn_q8(d, pt, st["q"], st["cache"], st["o"], st["ws"], st["bytes"], s)
        return [st["o"]]
    if op == "select":
        L.select_attn_q8(d, pt, st["sp"], st["q"], st["cache"], st["o"], st["sel_cnt"], st["sel_pages"], st["stride"],
                         st["scores"], st["ws"], st["bytes"], s)
        return [st["o"], st["sel_cnt"], st["sel_pages"], st["scores"]]
    L.sparse_attn_q8(d, pt, st["sel_cnt"], st["sel_pages"], st["stride"], st["q"], st["cache"], st["o"], st["ws"],
                     st["bytes"], s)
    return [st["o"]]


# ---------------------------------------------------------------------------------------------- plain forms
def _plain_rope(st, case):
    rd = case["rd"]
    angle = st["positions"].double()[:, None] * st["turns"][None, :] * (2 * math.pi)
    cos = (angle.cos() * st["magnitude"]).float()[:, None, :]
    sin = (angle.sin() * st["magnitude"]).float()[:, None, :]

    def turn(x):
        y = x.float()
        if case["layout"] == "half":
            a, b = y[..., : rd // 2], y[..., rd // 2: rd]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = y[..., 0:rd:2], y[..., 1:rd:2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([r, y[..., rd:]], -1).to(x.dtype)

    return [turn(st["q"]), turn(st["k"])]


def _plain_cache(st, case):
    fmt, dt = case["fmt"], DTYPE[case["dtype"]]
    lens, cum = st["kv_len"].long(), st["tokens"].long()
    start = lens - (cum[1:] - cum[:-1])
    count = torch.where(lens > start, (lens + PAGE - 1) // PAGE - start // PAGE, torch.zeros_like(lens))
    seq = torch.repeat_interleave(torch.arange(len(lens), device=lens.device), count)
    nth = torch.arange(len(seq), device=lens.device) - (count.cumsum(0) - count)[seq]
    page = start[seq] // PAGE + nth                                     # logical page of each block row
    phys = st["indices"].long()[st["indptr"].long()[seq] + page]
    pos = page[:, None] * PAGE + torch.arange(PAGE, device=lens.device)
    fresh = (pos >= start[seq][:, None]) & (pos < lens[seq][:, None])
    held = pos < start[seq][:, None]
    row = (cum[:-1][seq][:, None] + pos - start[seq][:, None]).clamp(0, max(len(st["k_new"]) - 1, 0))

    def write(pool, scale, x):
        y = torch.where(fresh[:, :, None, None], x.float()[row], 0.0).transpose(1, 2)   # [blocks, Hkv, 16, D]
        need = _block_scale(y.abs().amax(dim=(2, 3)), fmt)
        before = scale[phys]
        s = torch.where(held.any(1)[:, None], torch.maximum(before, need), need)
        older = _round8(pool[phys].view(PAYLOAD[fmt]).float() * (before / s)[..., None, None], fmt)
        newer = _round8(y / s[..., None, None], fmt)
        f, h = fresh[:, None, :, None], held[:, None, :, None]
        pool[phys] = torch.where(f, newer, torch.where(h, older, pool[phys]))
        scale[phys] = s

    write(st["k"], st["ks"], st["k_new"])
    write(st["v"], st["vs"], st["v_new"])
    reads = st["reads"].long()
    seq = torch.repeat_interleave(torch.arange(len(lens), device=lens.device), reads[1:] - reads[:-1])
    pos = st["starts"].long()[seq] + torch.arange(len(seq), device=lens.device) - reads[:-1][seq]
    phys = st["indices"].long()[st["indptr"].long()[seq] + pos // PAGE]

    def read(pool, scale):
        return (pool[phys, :, pos % PAGE].view(PAYLOAD[fmt]).float() * scale[phys][..., None]).to(dt)

    return [read(st["k"], st["ks"]), read(st["v"], st["vs"]), st["ks"], st["vs"]]


def _gather(pool, scale, pages, fmt):
    """Pages [B, N] of the pool as [B, Hkv, N * 16, D] in 32 bits."""
    x = pool[pages].float() if scale is None else _values(pool[pages], scale[pages], fmt)
    return x.transpose(1, 2).flatten(2, 3)


def _attend(q, k, v, seen, dt):
    """q [B, Hq, D]; k, v [B, Hkv, T, D]; seen [B, T] -> (o, probabilities [B, Hkv, G, T])."""
    b, hq, d = q.shape
    x = q.float().view(b, k.shape[1], -1, d) @ k.transpose(2, 3) / math.sqrt(d)
    x = x.masked_fill(~seen[:, None, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top.isinf(), torch.zeros_like(top), top))
    p = p / p.sum(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).tiny)
    return (p @ v).reshape(b, hq, d).to(dt), p


def _table(st):
    """The page table as [B, longest] (entries past a sequence's pages repeat its own)."""
    cols = torch.arange(st["longest"], device="cuda")
    at = torch.minimum(st["indptr"].long()[:-1, None] + cols, (st["indptr"].long()[1:, None] - 1).clamp_min(0))
    return st["indices"].long()[at]


def _plain_full(st, case):
    dt, lens = DTYPE[case["dtype"]], st["kv_len"].long()
    table = _table(st)
    k = _gather(st["k"], st["ks"], table, case["fmt"])
    v = _gather(st["v"], st["vs"], table, case["fmt"])
    t = torch.arange(k.shape[2], device=k.device)
    o, p = _attend(st["q"], k, v, t < lens[:, None], dt)
    if case["op"] == "full":
        return [o]
    score = p.sum((1, 2)).view(len(lens), -1, PAGE).sum(-1)                       # [B, pages]
    pages = (lens + PAGE - 1) // PAGE
    j = torch.arange(score.shape[1], device=k.device)[None]
    valid = j < pages[:, None]
    recent = (j >= (lens - case["recency"]).clamp_min(0)[:, None] // PAGE) & valid & (case["recency"] > 0)
    always = ((j < -(-case["sink"] // PAGE)) & valid) | recent
    rank = torch.where(always | ~valid, -math.inf, score).argsort(dim=1, descending=True, stable=True).argsort(dim=1)
    keep = always | (valid & ~always & (rank < case["budget"]))
    cnt = keep.sum(1)
    order = torch.where(keep, j, score.shape[1]).sort(1).values[:, : st["stride"]]
    order = torch.nn.functional.pad(order, (0, st["stride"] - order.shape[1]), value=score.shape[1])
    sel = torch.where(torch.arange(st["stride"], device=k.device) < cnt[:, None], order, -1)
    return [o, cnt.int(), sel.int(), torch.where(valid, score, 0.0)]


def _plain_sparse(st, case):
    lens = st["kv_len"].long()
    sel = st["sel_pages"].long()
    there = torch.arange(st["stride"], device=sel.device) < st["sel_cnt"][:, None]
    sel = torch.where(there, sel, 0)
    last = (st["indptr"].long()[1:, None] - 1).clamp_min(0)
    pages = st["indices"].long()[torch.minimum(st["indptr"].long()[:-1, None] + sel, last)]
    pos = sel[:, :, None] * PAGE + torch.arange(PAGE, device=sel.device)
    seen = (there[:, :, None] & (pos < lens[:, None, None])).flatten(1)
    return [_attend(st["q"], _gather(st["k"], st["ks"], pages, case["fmt"]),
                    _gather(st["v"], st["vs"], pages, case["fmt"]), seen, DTYPE[case["dtype"]])[0]]


def _plain_window(st, case):
    lens, w, sink = st["kv_len"].long(), case["window"], case["sink"]
    tail = (lens - w).clamp_min(sink)[:, None] + torch.arange(w, device="cuda")   # after the sinks, at most w tokens
    pos = torch.cat([torch.arange(sink, device="cuda").expand(len(lens), sink), tail], 1)
    seen = pos < lens[:, None]
    pos = torch.where(seen, pos, 0)
    last = (st["indptr"].long()[1:, None] - 1).clamp_min(0)
    pages = st["indices"].long()[torch.minimum(st["indptr"].long()[:-1, None] + pos // PAGE, last)]

    def rows(pool, scale):
        x = pool[pages, :, pos % PAGE]                                            # [B, T, Hkv, D]
        x = x.float() if scale is None else x.view(PAYLOAD[case["fmt"]]).float() * scale[pages][..., None]
        return x.transpose(1, 2)

    return [_attend(st["q"], rows(st["k"], st["ks"]), rows(st["v"], st["vs"]), seen, DTYPE[case["dtype"]])[0]]


# ---------------------------------------------------------------------------------------------- work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rope":
        n = case["rows"] * (case["hq"] + case["hkv"])
        return {"bytes": 2 * n * case["d"] * e + 4 * case["rows"], "flops": 3 * n * case["rd"]}
    if case["op"] == "cache":
        part = 0.5 if case["ragged"] else 1.0     # uneven lengths are half of the longest on average
        t = case["batch"] * max(1.0, case["new"] * part)
        back = t + case["batch"] * (case["have"] % PAGE if not case["ragged"] else 7.5)
        row = 2 * case["hkv"] * case["d"]
        return {"bytes": t * row * (e + 1) + back * row * (e + 1), "flops": 4 * t * row}
    b, n = case["batch"], case["ctx"]
    tokens = b * n if not case["ragged"] else n + max(0, b - 1 - 2 * (b >= 4)) * n / 2
    if case["op"] == "window":
        tokens = min(tokens, b * (case["window"] + case["sink"]))
    if case["op"] == "sparse":
        tokens = min(tokens, b * (case["budget"] * PAGE + case["sink"] + case["recency"]))
    store = e if case["fmt"] == "none" else 1 + 4.0 / (PAGE * case["d"])
    size = 2 * tokens * case["hkv"] * case["d"] * store + 2 * b * case["hq"] * case["d"] * e
    if case["op"] == "select":
        size += 4 * tokens / PAGE
    return {"bytes": size, "flops": 4 * tokens * case["hq"] * case["d"]}


# ---------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(st, case)
    if case["op"] == "cache":
        return _exact_cache(st, case)
    return _exact_attention(st, case)


def _exact_rope(st, case):
    """Each pair as a complex number times e^(i angle)."""
    rd = case["rd"]
    z = torch.polar(torch.full_like(st["turns"], st["magnitude"]).expand(case["rows"], -1).contiguous(),
                    2 * math.pi * torch.frac(st["positions"].double()[:, None] * st["turns"]))
    got = []
    for x in (st["q"], st["k"]):
        y = x.double().clone()
        head = y[..., :rd]
        pair = head.unflatten(-1, (2, rd // 2)).movedim(-2, -1) if case["layout"] == "half" else head.unflatten(-1, (rd // 2, 2))
        r = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z[:, None, :])
        y[..., :rd] = (r.movedim(-1, -2) if case["layout"] == "half" else r).flatten(-2)
        got.append(y)
    return got


def _two(e):
    """2^e for whole e, to the last bit."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest8(y, fmt):
    """The nearest 8-bit value to y in 64 bits, ties to even."""
    if fmt == "int8":
        return torch.round(y)
    size = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -30))).clamp_min(-6.0)
    size = torch.where(_two(size + 1) <= y.abs(), size + 1, size)
    size = torch.where((_two(size) > y.abs()) & (size > -6), size - 1, size)
    step = _two(size - 3)
    return torch.round(y / step) * step


def _exact_cache(st, case):
    fmt = case["fmt"]
    indptr, indices, lens = st["indptr"].tolist(), st["indices"].long(), st["kv_len"].tolist()
    cum, reads, starts = st["tokens"].tolist(), st["reads"].tolist(), st["starts"].tolist()
    out = []
    scales = []
    for pool, scale, x in ((st["k"], st["ks"], st["k_new"]), (st["v"], st["vs"], st["v_new"])):
        got, scale64 = [], scale.double().clone()
        for i, n in enumerate(lens):
            m = cum[i + 1] - cum[i]
            first = starts[i]
            if reads[i + 1] == reads[i]:
                continue
            phys = indices[indptr[i] + first // PAGE: indptr[i] + -(-n // PAGE)]
            old = n - m - first                                       # older tokens of the first page
            held = pool[phys[:1]].view(PAYLOAD[fmt]).double()[0, :, :old] * scale.double()[phys[0]][:, None, None]
            fresh = x[cum[i]: cum[i + 1]].double().transpose(0, 1)    # [Hkv, m, D]
            pad = len(phys) * PAGE - old - m
            gap = lambda k: fresh.new_zeros((fresh.shape[0], k, fresh.shape[2]))  # noqa: E731
            blocks = torch.cat([gap(old), fresh, gap(pad)], 1).unflatten(1, (len(phys), PAGE))
            big = blocks.abs().amax((2, 3))                           # [Hkv, pages]
            e = torch.ceil(torch.log2(big.clamp_min(1e-300) / QMAX[fmt])).clamp_min(LOG2_MIN)
            e = torch.where(big > QMAX[fmt] * _two(e), e + 1, e)
            e = torch.where((big <= QMAX[fmt] * _two(e - 1)) & (e > LOG2_MIN), e - 1, e)
            s = _two(e)
            if old:
                s[:, 0] = torch.maximum(s[:, 0], scale.double()[phys[0]])
            y = _nearest8(blocks / s[..., None, None], fmt) * s[..., None, None]
            y = y.flatten(1, 2)
            if old:
                y[:, :old] = _nearest8(held / s[:, :1, None], fmt) * s[:, :1, None]
            got.append(y[:, : old + m].transpose(0, 1))
            scale64[phys] = s.transpose(0, 1)
        out.append(torch.cat(got) if got else x.double()[:0])
        scales.append(scale64)
    return out + scales


def _exact_attention(st, case):
    """Sequence by sequence, head by head: the tokens that are seen, softmax, mean."""
    indptr, indices, lens = st["indptr"].tolist(), st["indices"].long(), st["kv_len"].tolist()
    d, group = case["d"], case["hq"] // case["hkv"]
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    select = case["op"] == "select"
    if select:
        scores = torch.zeros((len(lens), st["longest"]), dtype=torch.float64, device="cuda")
        sel = torch.full((len(lens), st["stride"]), -1, dtype=torch.int32, device="cuda")
        cnt = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
    for i, n in enumerate(lens):
        if n == 0:
            continue
        if case["op"] == "sparse":
            pages = st["sel_pages"][i, : int(st["sel_cnt"][i])].long()
            at = (pages[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten()
            at = at[at < n]
        else:
            at = torch.arange(n, device="cuda")
        if case["op"] == "window":
            at = at[(at < case["sink"]) | (at >= n - case["window"])]
        if not len(at):
            continue
        phys = indices[indptr[i] + at // PAGE]
        for g in range(case["hkv"]):
            def head(pool, scale):
                x = pool[phys, g, at % PAGE]
                return x.double() if scale is None else x.view(PAYLOAD[case["fmt"]]).double() * scale[phys, g].double()[:, None]
            k, v = head(st["k"], st["ks"]), head(st["v"], st["vs"])
            p = torch.softmax(st["q"][i, g * group: (g + 1) * group].double() @ k.T * d ** -0.5, dim=-1)
            o[i, g * group: (g + 1) * group] = p @ v
            if select:
                scores[i].index_add_(0, at // PAGE, p.sum(0))
        if select:
            pages, sink, first = _kept(n, case)
            by = sorted(range(sink, first), key=lambda j, s=scores[i].tolist(): (-s[j], j))[: case["budget"]]
            keep = sorted(list(range(sink)) + by + list(range(first, pages)))
            cnt[i] = len(keep)
            sel[i, : len(keep)] = torch.tensor(keep, dtype=torch.int32)
    return [o, cnt, sel, scores] if select else [o]
