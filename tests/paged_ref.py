"""Plain float64 forms of the paged operators, token by token, and the error bounds that the
kernels' roundings allow. Shares no code with the package.

Bounds (half-step roundings; U = 2^-8 for bf16, relative to the value):

append: an element is (x c - y s) in fp32 (three roundings of terms no larger than |x| + |y|,
  |c|, |s| <= 1), then one bf16 rounding:  U |ref| + 4 * 2^-24 (|x| + |y|).

attention: out = sum w_u v_u with w = softmax(l). Let A = sum w_u |v_u| (per element).
  - the probabilities are rounded to bf16 and the sum takes the rounded ones: every weight is
    off by a factor within (1 + U) / (1 - U):  2.02 U A;
  - the last 64 elements of the rotated query are rounded to bf16: a logit moves by at most
    U Lr, Lr = scale * max_u sum |q_i k_i| over them;
  - the fp32 sums: 512 products in a logit (512 * 2^-23 L, L the same sum over all 512), the
    exponent's argument (2^-22 * (|l| + 16) * 1.45, the running maximum may lag by 8 in log2) and
    exp2 (2^-21), and n additions over the keys (n * 2^-23);
  - a logit error e moves every weight by a factor within exp(+-2 e);
  - turning the output back: fp32, 2^-22 A; one bf16 rounding of the output: U |ref|.
"""
import numpy as np
import torch

DIM, ROPE = 512, 64
U = 2.0 ** -8


def angles(n_pos, base=10000.0):
    """[n_pos, 32, 2] fp32 (cos, sin) on the CPU, from float64 angles."""
    a = torch.arange(n_pos, dtype=torch.float64)[:, None] * base ** (
        -torch.arange(ROPE // 2, dtype=torch.float64) / (ROPE // 2))
    return torch.stack([a.cos(), a.sin()], -1).float()


def turn(x, cs, sign=1.0):
    """x [..., 512] float64 with its last 32 pairs turned by cs [32, 2]."""
    x = x.clone()
    c, s = cs[:, 0].double(), sign * cs[:, 1].double()
    a, b = x[..., DIM - ROPE::2].clone(), x[..., DIM - ROPE + 1::2].clone()
    x[..., DIM - ROPE::2] = a * c - b * s
    x[..., DIM - ROPE + 1::2] = a * s + b * c
    return x


def valid(batch, s, n_new):
    r0, r1, ln = int(batch["new_start"][s]), int(batch["new_start"][s + 1]), int(batch["seq_len"][s])
    limit = batch["page_table"].shape[1] * batch["pages"].shape[1]
    if batch["cos_sin"] is not None:
        limit = min(limit, batch["cos_sin"].shape[0])
    return 0 <= r0 <= r1 <= n_new and r1 - r0 <= ln <= limit


def place(batch, s, p):
    """(page, row) of position p of sequence s, or None when the entry is no page."""
    n_pages, page = batch["pages"].shape[:2]
    e = int(batch["page_table"][s, p // page])
    return (e, p % page) if 0 <= e < n_pages else None


def append(batch, kv):
    """(pages, allowed error): float64 pages after the append."""
    pages = batch["pages"].double().clone()
    tol = torch.zeros_like(pages)
    for s in range(len(batch["seq_len"])):
        if not valid(batch, s, kv.shape[0]):
            continue
        r0, r1 = int(batch["new_start"][s]), int(batch["new_start"][s + 1])
        for r in range(r0, r1):
            p = int(batch["seq_len"][s]) - r1 + r
            at = place(batch, s, p)
            if at is None:
                continue
            x = kv[r].double()
            if batch["cos_sin"] is not None:
                pair = x[DIM - ROPE:].abs().view(-1, 2).sum(-1)
                x = turn(x, batch["cos_sin"][p])
                t = torch.zeros(DIM, dtype=torch.float64)
                t[DIM - ROPE:] = (U * x[DIM - ROPE:].abs()
                                  + 4 * 2.0 ** -24 * pair.repeat_interleave(2))
                tol[at] = t
            pages[at] = x
    return pages, tol


def attention(batch, q, window, scale):
    """(out, allowed error, rows that are written) in float64; rows of no valid sequence NaN."""
    n_new, heads = q.shape[:2]
    out = torch.full((n_new, heads, DIM), float("nan"), dtype=torch.float64)
    tol = torch.zeros_like(out)
    written = np.zeros(n_new, dtype=bool)
    pages, cs = batch["pages"].double(), batch["cos_sin"]
    for s in range(len(batch["seq_len"])):
        if not valid(batch, s, n_new):
            continue
        r0, r1 = int(batch["new_start"][s]), int(batch["new_start"][s + 1])
        ln = int(batch["seq_len"][s])
        for r in range(r0, r1):
            t = ln - r1 + r
            written[r] = True
            at = [place(batch, s, u) for u in range(max(0, t - window + 1) if window else 0, t + 1)]
            at = [a for a in at if a is not None]
            if not at:
                out[r] = 0.0
                continue
            a = torch.tensor(at)
            kv = pages[a[:, 0], a[:, 1]]
            qr = q[r].double()
            if cs is not None:
                qr = turn(qr, cs[t])
            logits = scale * qr @ kv.T
            w = torch.softmax(logits, -1)
            o = w @ kv
            big = w @ kv.abs()
            if cs is not None:
                o = turn(o, cs[t], -1.0)
                b = big[:, DIM - ROPE:].view(heads, -1, 2).sum(-1).repeat_interleave(2, -1)
                big = torch.cat([big[:, :DIM - ROPE], b], -1)
            size = scale * (qr.abs() @ kv.abs().T).amax(-1)
            e = 512 * 2.0 ** -23 * size + 2.0 ** -22 * 1.45 * (logits.abs().amax(-1) + 16)
            if cs is not None:
                e = e + U * scale * (qr[:, DIM - ROPE:].abs()
                                     @ kv[:, DIM - ROPE:].abs().T).amax(-1)
            spread = torch.expm1(2 * e) + 2.02 * U + 2.0 ** -20 + len(at) * 2.0 ** -23
            out[r] = o
            tol[r] = U * o.abs() + big * spread[:, None]
    return out, tol, written


def make(lens, page=16, extra_pages=3, rope=True, seed=0, max_pages=None, n_new=None):
    """A CPU batch of sequences [(new, total)], every page filled, in shuffled pages."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-c // page) for _, c in lens]
    n_pages = sum(counts) + extra_pages
    order = torch.randperm(n_pages, generator=g)
    cols = max_pages or max(1, max(counts))
    table = torch.full((len(lens), cols), -1, dtype=torch.int32)
    at = 0
    for s, c in enumerate(counts):
        table[s, :c] = order[at:at + c].int()
        at += c
    starts = torch.tensor([0] + [n for n, _ in lens]).cumsum(0).int()
    return dict(pages=torch.randn(n_pages, page, DIM, generator=g).bfloat16(), page_table=table,
                new_start=starts, seq_len=torch.tensor([c for _, c in lens]).int(),
                cos_sin=angles(cols * page) if rope else None)
