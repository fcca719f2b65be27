"""Cases that measure the paged-cache operators: dsa_paged_append and dsa_paged_attn.

A serving process holds the 512-wide KV rows of many sequences in pages and runs a ragged
batch through one layer: the new tokens' rows are rotated by their positions and written into
the pages, then every new token attends over its sequence's rows (all of them, or its window).
Lengths are part of the case (``_lengths``); values come from the seed.
"""
import math
import random

import torch

own = False

DIM = 512    # one KV row, key and value of every head
ROPE = 64    # rotated elements at the end of a row, 32 pairs
WORKSPACE = 40 << 20   # bytes the attention wants to join partial results


def _case(name, op, seqs, new, ctx, heads=64, page=64, window=0, rope=True, ragged=False, pad=0,
          shape=0):
    """``new``/``ctx``: the largest number of new tokens and the largest length of a sequence."""
    return dict(name=name, op=op, seqs=seqs, new=new, ctx=ctx, heads=heads, page=page,
                window=window, rope=rope, ragged=ragged, pad=pad, shape=shape)


def listed():
    return [
        # one user, one new token, a 128K context: latency of a long decode step
        _case("decode_128k", "attn", 1, 1, 131072),
        # a server's decode step: 64 users of different lengths up to 8K
        _case("decode_batch_8k", "attn", 64, 1, 8192, ragged=True, shape=1),
        # a few short chats on a 16-head shard, small pages: launch-bound
        _case("decode_short", "attn", 4, 1, 509, heads=16, page=16, ragged=True, shape=2),
        # decode of a layer with 128 query heads
        _case("decode_128_heads", "attn", 32, 1, 4096, heads=128, page=64, rope=False,
              ragged=True, shape=3),
        # exact bands of up to four tokens (draft verification), page of 128 rows
        _case("bands_16k", "attn", 16, 4, 16384, page=128, ragged=True, shape=4),
        # the last 2048-row chunk of a 16K prompt
        _case("chunk_16k", "attn", 1, 2048, 16384),
        # a mixed batch of short prompts on a 16-head shard, padded to a captured batch size
        _case("prompts_ragged", "attn", 7, 701, 1499, heads=16, page=32, ragged=True, pad=5,
              shape=5),
        # local attention: a 4096-row chunk at 128K that sees its 128-row window alone
        _case("window_128k", "attn", 1, 4096, 131072, window=128),
        # one row appended
        _case("append_one", "append", 1, 1, 131072),
        # a decode step of 256 users
        _case("append_256_users", "append", 256, 1, 2048, ragged=True, shape=6),
        # a 4096-row prompt chunk
        _case("append_chunk", "append", 1, 4096, 131072),
        # many prompts at once in small pages
        _case("append_prompts", "append", 16, 8191, 16384, page=16, ragged=True, pad=3, shape=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    page = rng.choice([16, 32, 64, 128, 256])
    ragged, pad, shape = rng.random() < 0.7, rng.choice([0, 0, 1, 9]), rng.randrange(1 << 20)
    rope = rng.random() < 0.75
    if rng.random() < 0.3:
        seqs, new, ctx = _log(rng, 1, 256), _log(rng, 1, 8191), _log(rng, 1, 131072)
        while seqs * new > 65536:
            seqs, new = (seqs + 1) // 2, (new + 1) // 2
        ctx = max(ctx, new)
        while seqs * ctx > 1 << 18:
            seqs = (seqs + 1) // 2 if seqs > 1 else 1
            ctx = max(new, ctx // 2)
            new = min(new, max(1, (1 << 18) // seqs))
        return dict(op="append", seqs=seqs, new=min(new, ctx), ctx=ctx, heads=64, page=page,
                    window=0, rope=True, ragged=ragged, pad=pad, shape=shape)
    heads = rng.choice([1, 5, 8, 16, 24, 32, 48, 64, 64, 64, 96, 128])
    window = rng.choice([0, 0, 0, 128, _log(rng, 1, 4096)])
    new = 1 if rng.random() < 0.5 else _log(rng, 2, 4096)
    seqs, ctx = _log(rng, 1, 128), max(new, _log(rng, 1, 131072))
    while True:
        span = min(ctx, new + window) if window else ctx
        if seqs * new * heads * span <= 1 << 30 and seqs * ctx <= 1 << 20:
            break
        if seqs > 1:
            seqs = (seqs + 1) // 2
        elif new > 1:
            new = (new + 1) // 2
        else:
            ctx = (ctx + 1) // 2
    return dict(op="attn", seqs=seqs, new=new, ctx=ctx, heads=heads, page=page, window=window,
                rope=rope, ragged=ragged, pad=pad, shape=shape)


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


def _span(new, ctx, window):
    """First and one-past-last position that any of the new tokens sees."""
    return (max(0, ctx - new - window + 1) if window else 0), ctx


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    lens, page, window = _lengths(case), case["page"], case["window"]
    seqs, ctx = len(lens), max(c for _, c in lens)
    cols = -(-ctx // page)
    counts = [-(-c // page) for _, c in lens]
    n_pages = sum(counts) + 3                     # a few free pages
    order = torch.randperm(n_pages, generator=g, device=dev, dtype=torch.int64)
    pages = torch.randn(n_pages, page, DIM, generator=g, device=dev, dtype=torch.bfloat16)
    ends = torch.tensor(counts, device=dev).cumsum(0)
    col = torch.arange(cols, device=dev)
    held = col[None, :] < torch.tensor(counts, device=dev)[:, None]
    flat = (ends - torch.tensor(counts, device=dev))[:, None] + col[None, :]
    page_table = torch.where(held, order[flat.clamp(max=n_pages - 1)], -1).to(torch.int32)
    news = [n for n, _ in lens]
    starts = torch.tensor([0] + news, device=dev).cumsum(0).to(torch.int32)
    rows = sum(news) + case["pad"]
    angle = (torch.arange(ctx, device=dev, dtype=torch.float64)[:, None]
             * 10000.0 ** (-torch.arange(ROPE // 2, device=dev, dtype=torch.float64)
                           / (ROPE // 2)))
    spans = [_span(n, c, window) for n, c in lens]
    state = dict(op=case["op"], pages=pages, page_table=page_table, new_start=starts,
                 seq_len=torch.tensor([c for _, c in lens], device=dev, dtype=torch.int32),
                 cos_sin=torch.stack([angle.cos(), angle.sin()], -1).to(torch.float32)
                 if case["rope"] else None,
                 rows=sum(news), max_new=max(news), max_span=max(b - a for a, b in spans))
    if case["op"] == "append":
        state["kv"] = torch.randn(rows, DIM, generator=g, device=dev, dtype=torch.bfloat16)
        return state
    # rows past a sequence's end were never written: whatever the memory held
    last = order[ends - 1]
    stale = torch.arange(page, device=dev)[None, :] >= torch.tensor(
        [(c - 1) % page + 1 for _, c in lens], device=dev)[:, None]
    pages[last] = pages[last].masked_fill(stale[..., None], float("nan"))
    state |= dict(q=torch.randn(rows, case["heads"], DIM, generator=g, device=dev,
                                dtype=torch.bfloat16),
                  out=torch.zeros(rows, case["heads"], DIM, device=dev, dtype=torch.bfloat16),
                  window=window, scale=1.0 / math.sqrt(DIM),
                  workspace=torch.empty(WORKSPACE, device=dev, dtype=torch.uint8))
    return state


def _positions(s):
    """Of every new token: its sequence, its index among the sequence's new tokens, its position."""
    r = torch.arange(s["rows"], device=s["pages"].device)
    start = s["new_start"].long()
    seq = torch.searchsorted(start[1:], r, right=True)
    i = r - start[seq]
    return seq, i, s["seq_len"].long()[seq] - (start[seq + 1] - start[seq]) + i


def _rotate(x, cs, sign):
    """Turn the last 32 pairs of x [..., 512] by the angles of cs [..., 32, 2]."""
    pair = x[..., DIM - ROPE:].unflatten(-1, (ROPE // 2, 2))
    c, sn = cs[..., 0], sign * cs[..., 1]
    turned = torch.stack([pair[..., 0] * c - pair[..., 1] * sn,
                          pair[..., 0] * sn + pair[..., 1] * c], -1).flatten(-2)
    return torch.cat([x[..., :DIM - ROPE], turned], -1)


def _plain_append(s):
    seq, _, pos = _positions(s)
    row = _rotate(s["kv"][:s["rows"]].float(), s["cos_sin"][pos], 1.0)
    page = s["pages"].shape[1]
    at = s["page_table"][seq, pos // page].long()
    s["pages"][at, pos % page] = row.to(s["pages"].dtype)
    return s["pages"]


def _plain_attn(s):
    seq, i, pos = _positions(s)
    n, heads = s["rows"], s["q"].shape[1]
    seqs, page = s["page_table"].shape[0], s["pages"].shape[1]
    q = s["q"][:n].float()
    if s["cos_sin"] is not None:
        q = _rotate(q, s["cos_sin"][pos][:, None], 1.0)
    # queries padded to [sequence, new token, head], keys to [sequence, span of seen positions]
    qp = q.new_zeros(seqs, s["max_new"], heads, DIM)
    qp[seq, i] = q
    start, length = s["new_start"].long(), s["seq_len"].long()
    first = length - (start[1:] - start[:-1])
    low = (first - s["window"] + 1).clamp(min=0) if s["window"] else torch.zeros_like(first)
    kpos = low[:, None] + torch.arange(s["max_span"], device=q.device)
    real = kpos < length[:, None]
    at = torch.where(real, kpos, 0)
    kv = s["pages"][s["page_table"].gather(1, at // page).long(), at % page].float()
    kv = kv.masked_fill(~real[..., None], 0.0)
    x = (qp.flatten(1, 2) @ kv.transpose(1, 2)).mul_(s["scale"]).unflatten(1, (s["max_new"], heads))
    qpos = first[:, None] + torch.arange(s["max_new"], device=q.device)
    seen = real[:, None] & (kpos[:, None] <= qpos[..., None])
    if s["window"]:
        seen &= kpos[:, None] > qpos[..., None] - s["window"]
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
        return _plain_append(s) if s["op"] == "append" else _plain_attn(s)
    import deepseek_v4_sparse_ratio_gb300 as dsa
    if s["op"] == "append":
        dsa.dsa_paged_append(s["kv"], s["new_start"], s["seq_len"], s["page_table"], s["pages"],
                             s["cos_sin"])
        return s["pages"]
    dsa.dsa_paged_attn(s["q"], s["new_start"], s["seq_len"], s["page_table"], s["pages"],
                       s["window"], s["scale"], s["workspace"], s["out"], s["cos_sin"])
    return s["out"]


def work(case):
    """Each input once, each output once: a sequence's seen rows, queries and outputs (or rows in
    and out), the angles of the new positions, lengths and page-table entries."""
    lens, window, heads = _lengths(case), case["window"], case["heads"]
    new = sum(n for n, _ in lens)
    table = new * ROPE * 4 if case["rope"] else 0
    meta = 4 * (2 * len(lens) + 1)
    if case["op"] == "append":
        touched = sum((c - 1) // case["page"] - (c - n) // case["page"] + 1 for n, c in lens)
        return {"bytes": new * DIM * 4 + table + meta + 4 * touched, "flops": new * ROPE * 3}
    spans = [_span(n, c, window) for n, c in lens]
    keys = sum(b - a for a, b in spans)
    pairs = 0                                      # (new token, key it sees)
    for n, c in lens:
        first = c - n                              # token i sees min(window, first + i + 1) rows
        whole = n if not window else max(0, min(n, window - first))
        pairs += whole * first + whole * (whole + 1) // 2 + (n - whole) * window
    return {"bytes": keys * DIM * 2 + new * heads * DIM * 4 + table + meta
            + 4 * sum((b - 1) // case["page"] - a // case["page"] + 1 for a, b in spans),
            "flops": 4 * DIM * heads * pairs}


def exact(case, seed):
    """The definition in float64, sequence by sequence and a few tokens at a time."""
    s = prepare(case, seed)
    lens, page, window = _lengths(case), case["page"], case["window"]
    cs = s["cos_sin"].double() if case["rope"] else None
    out = (s["pages"] if case["op"] == "append" else s["out"]).double()

    def turned(x, table):                          # complex product on the last 32 pairs
        z = torch.view_as_complex(x[..., DIM - ROPE:].reshape(*x.shape[:-1], ROPE // 2, 2))
        x = x.clone()
        x[..., DIM - ROPE:] = torch.view_as_real(z * table).flatten(-2)
        return x

    r0 = 0
    for b, (n, c) in enumerate(lens):
        where = torch.arange(c, device=out.device)
        place = s["page_table"][b].long()[where // page], where % page
        first = c - n
        if case["op"] == "append":
            rows = turned(s["kv"][r0:r0 + n].double(), torch.view_as_complex(cs[first:c]))
            out[place[0][first:], place[1][first:]] = rows
            r0 += n
            continue
        low, _ = _span(n, c, window)
        kv = s["pages"][place[0][low:], place[1][low:]].double()
        step = max(1, (1 << 28) // (case["heads"] * (c - low)))
        for i in range(0, n, step):
            t = where[first + i:first + min(n, i + step)]
            q = s["q"][r0 + i:r0 + i + len(t)].double()
            if cs is not None:
                z = torch.view_as_complex(cs[t])[:, None]
                q = turned(q, z)
            x = torch.einsum("thd,kd->thk", q, kv) * s["scale"]
            u = where[low:]
            hidden = u[None] > t[:, None]
            if window:
                hidden |= u[None] <= t[:, None] - window
            p = torch.softmax(x.masked_fill(hidden[:, None], -torch.inf), -1)
            o = torch.einsum("thk,kd->thd", p, kv)
            out[r0 + i:r0 + i + len(t)] = turned(o, z.conj()) if cs is not None else o
        r0 += n
    return out
