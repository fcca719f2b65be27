"""Cases that measure the norm + rotation of new tokens and the 4-bit paged cache:
dsa_qk_norm_rope, dsa_paged_q4_append, dsa_paged_q4_read and dsa_paged_q4_attn.

A layer of a serving process normalises the new tokens' query heads and KV rows and turns them by
position, writes the KV rows into pages in 4 bits, reads rows back where a packed copy is wanted,
and attends over the pages: the whole context, or a sliding window and the first few tokens.

A row of the cache is 384 bytes: 448 elements in 4 bits with a scale per 16, and the 64 rotated
ones in bf16. With A the row's largest of the 448 magnitudes and E = floor(log2 A) - 10 (-123 at
least), a group's scale is s = amax / 7 / 2^E in e4m3 and an element n = x / (s 2^E) rounded to a
whole number of -7 .. 7, ties to even; it stands for n s 2^E. Twelve 32-byte places hold
  bytes 32 j + 16 h + ..: half h (32 dims) of chunk c (64 dims)
  j = 0: the 14 scales of the half, two a chunk, then a byte E + 137, then zero
  j = 1 .. 7: chunk j - 1; a word has eight dims: dim 2 k is nibble k, dim 2 k + 1 nibble k + 4,
              as n + 8
  j = 8 .. 11: the 64 bf16 in order
Lengths are part of the case (``_lengths``); values come from the seed.
"""
import math
import random

import torch

own = False

DIM = 512    # one KV row, key and value of every head
ROPE = 64    # rotated elements at the end of a row, 32 pairs
NOPE = DIM - ROPE
GROUP = 16   # elements that share a scale
ROW = 384    # bytes of a row in 4 bits
WORKSPACE = 40 << 20   # bytes the attention wants to join partial results
EPS = 1e-6


def _case(name, op, seqs, new, ctx, heads=64, page=64, window=0, sinks=0, rope=True, ragged=False,
          pad=0, shape=0):
    """``new``/``ctx``: the largest number of new tokens and the largest length of a sequence."""
    return dict(name=name, op=op, seqs=seqs, new=new, ctx=ctx, heads=heads, page=page,
                window=window, sinks=sinks, rope=rope, ragged=ragged, pad=pad, shape=shape)


def listed():
    return [
        # one user's new token: latency
        _case("norm_one", "norm", 1, 1, 131072),
        # a decode step of 64 users
        _case("norm_64_users", "norm", 64, 1, 8192, ragged=True, shape=1),
        # a 4096-row prompt chunk
        _case("norm_chunk", "norm", 1, 4096, 131072),
        # a decode step of 256 users: one row each, written and read back
        _case("append_256_users", "append", 256, 1, 2048, ragged=True, shape=6),
        # many prompts at once in small pages, written and read back
        _case("append_prompts", "append", 16, 8191, 16384, page=16, ragged=True, pad=3, shape=7),
        # the 128 rows before a chunk, as the window + selected attention wants them
        _case("read_window", "read", 1, 128, 131072),
        # the contexts of 16 users
        _case("read_16_users", "read", 16, 16384, 16384, page=128, ragged=True, shape=8),
        # one user, one new token, a 128K context: latency of a long decode step
        _case("decode_128k", "attn", 1, 1, 131072),
        # a server's decode step: 64 users of different lengths up to 8K
        _case("decode_batch_8k", "attn", 64, 1, 8192, ragged=True, shape=1),
        # decode of 96 long chats in a layer with a window and a few first tokens that stay
        _case("decode_sinks", "attn", 96, 1, 16384, window=1024, sinks=4, ragged=True, shape=9),
        # ragged prompts on a 16-head shard with a window, padded to a captured batch size
        _case("prompts_sinks", "attn", 7, 1701, 2999, heads=16, page=32, window=512, sinks=16,
              ragged=True, pad=5, shape=5),
        # the last 2048-row chunk of a 16K prompt
        _case("chunk_16k", "attn", 1, 2048, 16384),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    page = rng.choice([16, 32, 64, 128, 256])
    ragged, pad, shape = rng.random() < 0.7, rng.choice([0, 0, 1, 9]), rng.randrange(1 << 20)
    heads = rng.choice([1, 5, 8, 16, 24, 32, 48, 64, 64, 64, 96, 128])
    op = rng.choice(["norm", "append", "read", "attn", "attn", "attn"])
    common = dict(op=op, heads=heads, page=page, rope=rng.random() < 0.75, ragged=ragged, pad=pad,
                  shape=shape)
    if op != "attn":
        seqs, new, ctx = _log(rng, 1, 256), _log(rng, 1, 8191), _log(rng, 1, 131072)
        while seqs * new * (heads if op == "norm" else 1) > 1 << 17:
            seqs, new = (seqs + 1) // 2, (new + 1) // 2
        ctx = max(ctx, new)
        while seqs * ctx > 1 << 18:
            seqs = (seqs + 1) // 2 if seqs > 1 else 1
            ctx = max(new, ctx // 2)
            new = min(new, max(1, (1 << 18) // seqs))
        return dict(common, seqs=seqs, new=min(new, ctx), ctx=ctx, window=0, sinks=0)
    window = rng.choice([0, 0, 128, _log(rng, 1, 4096)])
    sinks = rng.choice([0, 1, 4, _log(rng, 1, 128)]) if window else 0
    new = 1 if rng.random() < 0.5 else _log(rng, 2, 4096)
    seqs, ctx = _log(rng, 1, 128), max(new, _log(rng, 1, 131072))
    while True:
        span = min(ctx, new + window + sinks) if window else ctx
        if seqs * new * heads * span <= 1 << 30 and seqs * ctx <= 1 << 20:
            break
        if seqs > 1:
            seqs = (seqs + 1) // 2
        elif new > 1:
            new = (new + 1) // 2
        else:
            ctx = (ctx + 1) // 2
    return dict(common, seqs=seqs, new=new, ctx=ctx, window=window, sinks=sinks)


def _lengths(case):
    """(new tokens, total length) of every sequence: whole numbers fixed by the case."""
    rng = random.Random(case["shape"])
    out = []
    for _ in range(case["seqs"]):
        if case["ragged"]:
            new = rng.randint(1, case["new"])
            out.append((new, rng.randint(max(new, case["ctx"] // 8), case["ctx"])))
        else:
            out.append((case["new"], case["ctx"]))
    return out


def _low(case, new, ctx):
    """First position that any of the new tokens sees within its window."""
    return max(0, ctx - new - case["window"] + 1) if case["window"] else 0


def _times_two(x, e):
    """x * 2^e, exactly, for whole numbers e of -252 .. 252 (in two steps of half the size)."""
    a = e // 2
    for k in (a, e - a):
        x = x * ((k + 127) << 23).to(torch.int32).view(torch.float32)
    return x


def _pack(x):
    """Rows [n, 512] bf16 -> [n, 384] uint8."""
    n, dev = x.shape[0], x.device
    v = x[:, :NOPE].float()
    group = v.view(n, NOPE // GROUP, GROUP).abs().amax(-1)
    top = group.amax(-1, keepdim=True)
    e = ((top.view(torch.int32) >> 23) - 127).clamp(min=-113)     # of the row
    # (tensors: a division by a number may be a product with its reciprocal)
    s = (_times_two(group, 10 - e) / torch.full_like(group, 7)).to(torch.float8_e4m3fn)
    unit = s.float().repeat_interleave(GROUP, 1)
    code = torch.where(unit > 0, (_times_two(v, 10 - e) / unit).round(), 0.0)
    code = code.clamp(-7, 7).to(torch.int32) + 8
    row = torch.zeros(n, ROW, dtype=torch.uint8, device=dev)
    # scales: [n, chunk, half, 2] -> [n, half, (chunk, 2)]
    sides = s.view(torch.uint8).view(n, 7, 2, 2).transpose(1, 2).reshape(n, 2, 14)
    head = row[:, :32].view(n, 2, 16)
    head[:, :, :14] = sides
    head[:, :, 14] = (e + 127).to(torch.uint8)
    # nibbles: a word's dims 2 k and 2 k + 1 are nibbles k and k + 4, two nibbles a byte
    pair = code.view(n, NOPE // 8, 4, 2)
    low = pair[:, :, 0::2] | pair[:, :, 1::2] << 4     # [n, word, byte, even | odd dims]
    row[:, 32:256] = low.transpose(2, 3).reshape(n, NOPE // 2).to(torch.uint8)
    row[:, 256:] = x[:, NOPE:].contiguous().view(torch.uint8)
    return row


def _unpack(row):
    """Rows [..., 384] uint8 -> [..., 512] fp32."""
    shape = row.shape[:-1]
    row = row.reshape(-1, ROW)
    n = row.shape[0]
    head = row[:, :32].view(n, 2, 16)
    s = head[:, :, :14].contiguous().view(torch.float8_e4m3fn).float()
    s = s.view(n, 2, 7, 2).transpose(1, 2).reshape(n, NOPE // GROUP)
    e = head[:, 0, 14].to(torch.int32) - 137
    s = _times_two(s, e[:, None])
    b = row[:, 32:256].view(n, NOPE // 8, 2, 2)        # [n, word, even | odd dims, byte]
    code = torch.stack([b & 15, b >> 4], -1).view(n, NOPE // 8, 2, 4).transpose(2, 3)
    v = (code.reshape(n, NOPE // GROUP, GROUP).float() - 8) * s[:, :, None]
    rope = row[:, 256:].contiguous().view(torch.bfloat16).float()
    return torch.cat([v.view(n, NOPE), rope], -1).view(*shape, DIM)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    lens, page, op = _lengths(case), case["page"], case["op"]
    ctx = max(c for _, c in lens)
    cols = -(-ctx // page)
    counts = [-(-c // page) for _, c in lens]
    news = [n for n, _ in lens]
    starts = torch.tensor([0] + news, device=dev).cumsum(0).to(torch.int32)
    rows = sum(news) + case["pad"]
    angle = (torch.arange(ctx, device=dev, dtype=torch.float64)[:, None]
             * 10000.0 ** (-torch.arange(ROPE // 2, device=dev, dtype=torch.float64)
                           / (ROPE // 2)))
    state = dict(op=op, new_start=starts,
                 seq_len=torch.tensor([c for _, c in lens], device=dev, dtype=torch.int32),
                 cos_sin=torch.stack([angle.cos(), angle.sin()], -1).to(torch.float32)
                 if case["rope"] else None, rows=sum(news), max_new=max(news))

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    if op == "norm":
        # what a projection gives: rows of different sizes
        size = (randn(rows, 1, 1, dtype=torch.float32) * 0.5).exp() * 2
        q = (randn(rows, case["heads"], DIM) * size).bfloat16()
        kv = (randn(rows, DIM) * size[:, 0]).bfloat16()
        return state | dict(
            q=q, kv=kv, q_weight=None, kv_weight=1 + 0.1 * randn(DIM, dtype=torch.float32),
            q_out=torch.zeros_like(q), kv_out=torch.zeros_like(kv))
    n_pages = sum(counts) + 3                     # a few free pages
    order = torch.randperm(n_pages, generator=g, device=dev, dtype=torch.int64)
    pages = torch.empty(n_pages, page, ROW, dtype=torch.uint8, device=dev)
    for part in pages.view(-1, ROW).split(1 << 16):
        part.copy_(_pack(randn(part.shape[0], DIM)))
    ends = torch.tensor(counts, device=dev).cumsum(0)
    col = torch.arange(cols, device=dev)
    held = col[None, :] < torch.tensor(counts, device=dev)[:, None]
    flat = (ends - torch.tensor(counts, device=dev))[:, None] + col[None, :]
    state |= dict(pages=pages, page_table=torch.where(
        held, order[flat.clamp(max=n_pages - 1)], -1).to(torch.int32))
    if op == "append":
        state["kv"] = randn(rows, DIM)
    if op != "attn":
        return state | dict(out=torch.zeros(rows, DIM, device=dev, dtype=torch.bfloat16))
    # rows past a sequence's end were never written: whatever the memory held
    last = order[ends - 1]
    stale = torch.arange(page, device=dev)[None, :] >= torch.tensor(
        [(c - 1) % page + 1 for _, c in lens], device=dev)[:, None]
    pages[last] = pages[last].masked_fill(stale[..., None], 255)
    return state | dict(q=randn(rows, case["heads"], DIM),
                        out=torch.zeros(rows, case["heads"], DIM, device=dev, dtype=torch.bfloat16),
                        window=case["window"], sinks=case["sinks"], scale=1.0 / math.sqrt(DIM),
                        max_span=max(c - _low(case, n, c) for n, c in lens),
                        workspace=torch.empty(WORKSPACE, device=dev, dtype=torch.uint8))


def _positions(s):
    """Of every new token: its sequence, its index among the sequence's new tokens, its position."""
    r = torch.arange(s["rows"], device=s["seq_len"].device)
    start = s["new_start"].long()
    seq = torch.searchsorted(start[1:], r, right=True)
    i = r - start[seq]
    return seq, i, s["seq_len"].long()[seq] - (start[seq + 1] - start[seq]) + i


def _rotate(x, cs, sign):
    """Turn the last 32 pairs of x [..., 512] by the angles of cs [..., 32, 2]."""
    pair = x[..., NOPE:].unflatten(-1, (ROPE // 2, 2))
    c, sn = cs[..., 0], sign * cs[..., 1]
    turned = torch.stack([pair[..., 0] * c - pair[..., 1] * sn,
                          pair[..., 0] * sn + pair[..., 1] * c], -1).flatten(-2)
    return torch.cat([x[..., :NOPE], turned], -1)


def _plain_norm(s):
    n = s["rows"]
    pos = _positions(s)[2]

    def norm(x, weight, cs):
        x = x.float()
        y = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
        y = y if weight is None else y * weight
        return y if cs is None else _rotate(y, cs, 1.0)

    cs = None if s["cos_sin"] is None else s["cos_sin"][pos]
    s["q_out"][:n] = norm(s["q"][:n], s["q_weight"], None if cs is None else cs[:, None])
    s["kv_out"][:n] = norm(s["kv"][:n], s["kv_weight"], cs)
    return s["q_out"], s["kv_out"]


def _plain_rows(s):
    """The append (where there are rows to append), and the rows of the new tokens read back."""
    seq, _, pos = _positions(s)
    page = s["pages"].shape[1]
    at, row = s["page_table"][seq, pos // page].long(), pos % page
    if s["op"] == "append":
        x = s["kv"][:s["rows"]]
        if s["cos_sin"] is not None:
            x = _rotate(x.float(), s["cos_sin"][pos], 1.0).to(x.dtype)
        s["pages"][at, row] = _pack(x)
    s["out"][:s["rows"]] = _unpack(s["pages"][at, row]).to(s["out"].dtype)
    return s["out"]


def _plain_attn(s):
    seq, i, pos = _positions(s)
    n, heads, window, sinks = s["rows"], s["q"].shape[1], s["window"], s["sinks"]
    seqs, page, dev = s["page_table"].shape[0], s["pages"].shape[1], s["q"].device
    q = s["q"][:n].float()
    if s["cos_sin"] is not None:
        q = _rotate(q, s["cos_sin"][pos][:, None], 1.0)
    # queries padded to [sequence, new token, head], keys to the first tokens and the span of
    # positions from the lowest that a window holds
    qp = q.new_zeros(seqs, s["max_new"], heads, DIM)
    qp[seq, i] = q
    start, length = s["new_start"].long(), s["seq_len"].long()
    first = length - (start[1:] - start[:-1])
    low = (first - window + 1).clamp(min=0) if window else torch.zeros_like(first)
    kpos = low[:, None] + torch.arange(s["max_span"], device=dev)
    real = kpos < length[:, None]
    if sinks:
        head = torch.arange(sinks, device=dev).expand(seqs, -1)
        kpos = torch.cat([head, kpos], 1)
        real = torch.cat([head < low[:, None], real], 1)
    at = torch.where(real, kpos, 0)
    kv = s["pages"][s["page_table"].gather(1, at // page).long(), at % page]
    kv = _unpack(kv.masked_fill(~real[..., None], 0))
    x = (qp.flatten(1, 2) @ kv.transpose(1, 2)).mul_(s["scale"]).unflatten(1, (s["max_new"], heads))
    qpos = first[:, None] + torch.arange(s["max_new"], device=dev)
    seen = real[:, None] & (kpos[:, None] <= qpos[..., None])
    if window:
        seen &= (kpos[:, None] > qpos[..., None] - window) | (kpos[:, None] < sinks)
    x.masked_fill_(~seen[:, :, None], -torch.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top.isfinite(), top, 0.0)).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.flatten(1, 2) @ kv).unflatten(1, (s["max_new"], heads)).div_(total)[seq, i]
    if s["cos_sin"] is not None:
        o = _rotate(o, s["cos_sin"][pos][:, None], -1.0)
    s["out"][:n] = o.to(s["out"].dtype)
    return s["out"]


def run(state):
    s = state
    if not own:
        return {"norm": _plain_norm, "attn": _plain_attn}.get(s["op"], _plain_rows)(s)
    import deepseek_v4_sparse_ratio_gb300 as dsa
    if s["op"] == "norm":
        dsa.dsa_qk_norm_rope(s["q"], s["kv"], s["new_start"], s["seq_len"], s["q_out"], s["kv_out"],
                             s["cos_sin"], s["q_weight"], s["kv_weight"], EPS)
        return s["q_out"], s["kv_out"]
    batch = s["new_start"], s["seq_len"], s["page_table"], s["pages"]
    if s["op"] == "append":
        dsa.dsa_paged_q4_append(s["kv"], *batch, s["cos_sin"])
    if s["op"] != "attn":
        dsa.dsa_paged_q4_read(*batch, s["out"])
        return s["out"]
    dsa.dsa_paged_q4_attn(s["q"], *batch, s["window"], s["sinks"], s["scale"], s["workspace"],
                          s["out"], s["cos_sin"])
    return s["out"]


def work(case):
    """Each input once, each output once: queries, rows in and out, a sequence's seen rows of the
    pages, the angles of the new positions, lengths and page-table entries."""
    lens, window, sinks, heads = _lengths(case), case["window"], case["sinks"], case["heads"]
    page, new = case["page"], sum(n for n, _ in lens)
    meta = 4 * (2 * len(lens) + 1) + (new * ROPE * 4 if case["rope"] else 0)
    if case["op"] == "norm":
        turn = 3 * ROPE if case["rope"] else 0
        return {"bytes": new * (heads + 1) * DIM * 4 + DIM * 4 + meta,
                "flops": new * (heads + 1) * (4 * DIM + turn)}
    if case["op"] != "attn":
        touched = sum((c - 1) // page - (c - n) // page + 1 for n, c in lens)
        one = ROW + DIM * 2          # a row of the pages and a packed one
        if case["op"] == "read":
            return {"bytes": new * one + 4 * (2 * len(lens) + 1) + 4 * touched, "flops": new * DIM}
        return {"bytes": new * (one + DIM * 2) + meta + 4 * touched, "flops": new * DIM * 6}
    keys = pages = pairs = 0                       # pairs: (new token, key it sees)
    for n, c in lens:
        low = _low(case, n, c)
        keys += c - low + min(sinks, low)
        pages += (c - 1) // page - low // page + 1 + (1 if sinks and low >= page else 0)
        first = c - n                              # token i sees min(window, first + i + 1) rows
        whole = n if not window else max(0, min(n, window - first))
        pairs += whole * first + whole * (whole + 1) // 2 + (n - whole) * window
        for i in range(whole, n) if sinks else ():  # and the first ones before its window
            pairs += min(sinks, first + i + 1 - window)
    return {"bytes": keys * ROW + new * heads * DIM * 4 + meta + 4 * pages,
            "flops": 4 * DIM * heads * pairs}


def _power(e):
    """2^e in float64 for whole numbers e, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_row(x):
    """What a row [n, 512] float64 stands for in the cache: from the definition, in float64."""
    g = x[:, :NOPE].reshape(-1, NOPE // GROUP, GROUP)
    amax = g.abs().amax(-1)
    e = (torch.frexp(amax.amax(-1)).exponent - 1).clamp(min=-113)
    s = amax / torch.full_like(amax, 7) * _power(10 - e)[:, None]
    # e4m3: steps of 2^-3 of the power of two below, 2^-9 at least
    step = _power((torch.frexp(s).exponent - 1).clamp(min=-6) - 3)
    s = torch.round(s / step) * step
    unit = (s * _power(e - 10)[:, None])[..., None]
    n = torch.round(g / torch.where(unit > 0, unit, 1.0)).clamp(-7, 7)
    return torch.cat([(n * unit).reshape(-1, NOPE), x[:, NOPE:]], -1)


def _exact_value(row):
    """What rows [n, 384] uint8 stand for, element by element, in float64."""
    n = row.shape[0]
    dim = torch.arange(NOPE, device=row.device)
    chunk, half, word, k = dim // 64, dim // 32 % 2, dim // 8 % 4, dim % 8
    nib = k // 2 + 4 * (k % 2)
    byte = row[:, 32 * (chunk + 1) + 16 * half + 4 * word + nib // 2].long()
    code = torch.where(nib % 2 > 0, byte >> 4, byte & 15).double() - 8
    b = row[:, 16 * half + 2 * chunk + dim // 16 % 2].long()
    exp, man = b >> 3 & 15, (b & 7).double()
    scale = torch.where(exp > 0, (1 + man / 8) * _power(exp - 7), man / 512)
    scale = torch.where(b == 127, torch.nan, scale)
    unit = _power(row[:, 14].long() - 137)[:, None]
    rope = row[:, 256:].reshape(n, ROPE, 2).long()
    rope = ((rope[..., 1] << 8 | rope[..., 0]) << 16).to(torch.int32).view(torch.float32).double()
    return torch.cat([code * scale * unit, rope], -1)


def exact(case, seed):
    """The definition in float64, sequence by sequence and a few tokens at a time."""
    s = prepare(case, seed)
    lens, page, window, sinks = _lengths(case), case["page"], case["window"], case["sinks"]
    cs = s["cos_sin"].double() if case["rope"] else None

    def turned(x, table):                          # complex product on the last 32 pairs
        z = torch.view_as_complex(x[..., NOPE:].reshape(*x.shape[:-1], ROPE // 2, 2))
        x = x.clone()
        x[..., NOPE:] = torch.view_as_real(z * table).flatten(-2)
        return x

    if case["op"] == "norm":
        outs, r0 = (s["q_out"].double(), s["kv_out"].double()), 0
        for n, c in lens:
            for x, w, out in zip((s["q"], s["kv"]), (s["q_weight"], s["kv_weight"]), outs):
                for i in range(0, n, 512):
                    part = slice(r0 + i, r0 + min(n, i + 512))
                    y = x[part].double()
                    y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / DIM + EPS)
                    if w is not None:
                        y = y * w.double()
                    if cs is not None:
                        z = torch.view_as_complex(cs[c - n + i:c - n + i + y.shape[0]])
                        y = turned(y, z[:, None] if y.dim() == 3 else z)
                    out[part] = y
            r0 += n
        return outs
    out, r0 = s["out"].double(), 0
    for b, (n, c) in enumerate(lens):
        where = torch.arange(c, device=out.device)
        at, row = s["page_table"][b].long()[where // page], where % page
        first = c - n
        if case["op"] == "append":
            x = s["kv"][r0:r0 + n].double()
            out[r0:r0 + n] = _exact_row(
                x if cs is None else turned(x, torch.view_as_complex(cs[first:c])))
        elif case["op"] == "read":
            out[r0:r0 + n] = _exact_value(s["pages"][at[first:], row[first:]])
        else:
            low = _low(case, n, c)
            u = torch.cat([where[:min(sinks, low)], where[low:]])
            kv = _exact_value(s["pages"][at[u], row[u]])
            step = max(1, (1 << 28) // (case["heads"] * len(u)))
            for i in range(0, n, step):
                t = where[first + i:first + min(n, i + step)]
                q = s["q"][r0 + i:r0 + i + len(t)].double()
                if cs is not None:
                    z = torch.view_as_complex(cs[t])[:, None]
                    q = turned(q, z)
                x = torch.einsum("thd,kd->thk", q, kv) * s["scale"]
                hidden = u[None] > t[:, None]
                if window:
                    hidden |= (u[None] <= t[:, None] - window) & (u[None] >= sinks)
                p = torch.softmax(x.masked_fill(hidden[:, None], -torch.inf), -1)
                o = torch.einsum("thk,kd->thd", p, kv)
                out[r0 + i:r0 + i + len(t)] = turned(o, z.conj()) if cs is not None else o
        r0 += n
    return out
