"""Plain float64 forms of the 4-bit paged operators and of the norm with rotation, and the error
bounds that the kernels' roundings allow. Shares no code with the package.

Bounds (half-step roundings; U = 2^-8 for bf16, relative to the value):

cache: codes, scales and exponents are whole numbers fixed by the inputs, so rows of the pages are
  equal byte for byte, the 64 rotated dims up to their fp32 rotation and one bf16 rounding (as in
  paged_ref.append); what is read back without angles is exact, with angles one such rotation more.

attention: as derived in paged_ref (the rows are bf16 exactly); with q turned by the caller the
  rounding of the rotated query is the caller's.

norm: y = x r w, r = 1 / sqrt(mean x^2 + eps) in fp32: 511 additions of rounded squares (512 * 2^-23
  of the sum at most, half of that in the root), root, division and two products (2^-22 together):
  e = 2^-15 relative to y. Turned: the products and their sum add 3 * 2^-24 (|a| + |b|) to e (|a| +
  |b|); then one bf16 rounding, U |y|.
"""
import numpy as np
import torch

from paged_ref import DIM, ROPE, U, angles, place, turn, valid  # noqa: F401

NOPE, GROUP, ROW = DIM - ROPE, 16, 384
E4M3 = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7)
                 for e in range(16) for m in range(8)][:127])   # by code; 127 is NaN


def nearest_e4m3(v):
    """Code of the e4m3 value next to v >= 0, ties to even codes."""
    i = int(np.searchsorted(E4M3, v))
    if i == 0:
        return 0
    below, above = v - E4M3[i - 1], E4M3[i] - v
    return i - 1 if below < above or (below == above and (i - 1) % 2 == 0) else i


def encode(x):
    """The 384 bytes of a row [512] float64 (its last 64 are bf16 values)."""
    out = np.zeros(ROW, dtype=np.uint8)
    x = x.numpy()
    groups = x[:NOPE].reshape(-1, GROUP)
    with np.errstate(invalid="ignore"):
        ok = (np.abs(groups) < 2.0 ** 124).all(-1)      # (a NaN is not)
    top = np.abs(groups[ok]).max(initial=0.0)
    e = max(int(np.floor(np.log2(top))) if top > 0 else -113, -113)
    for d in range(NOPE):
        g = d // GROUP
        code = 8
        if ok[g]:
            s = nearest_e4m3(np.abs(groups[g]).max() / 7 * 2.0 ** (10 - e))
            if s:
                n = np.rint(x[d] / (E4M3[s] * 2.0 ** (e - 10)))
                code = int(np.clip(n, -7, 7)) + 8
        else:
            s = 0x7F
        chunk, half = d // 64, d // 32 % 2
        out[16 * half + 2 * chunk + d // 16 % 2] = s
        nib = d % 8 // 2 + 4 * (d % 2)
        out[32 * (chunk + 1) + 16 * half + 4 * (d // 8 % 4) + nib // 2] |= code << 4 * (nib % 2)
    out[14] = out[30] = e + 127
    out[256:] = torch.from_numpy(x[NOPE:]).bfloat16().view(torch.uint8).numpy()
    return torch.from_numpy(out)


def decode(row):
    """What 384 bytes stand for: [512] float64."""
    row = row.numpy()
    out = np.zeros(DIM)
    for d in range(NOPE):
        chunk, half = d // 64, d // 32 % 2
        s = int(row[16 * half + 2 * chunk + d // 16 % 2])
        nib = d % 8 // 2 + 4 * (d % 2)
        byte = int(row[32 * (chunk + 1) + 16 * half + 4 * (d // 8 % 4) + nib // 2])
        n = (byte >> 4 * (nib % 2) & 15) - 8
        scale = np.nan if s & 127 == 127 else E4M3[s & 127] * (-1.0 if s > 127 else 1.0)
        out[d] = n * scale * 2.0 ** (int(row[14]) - 137)
    out[NOPE:] = torch.from_numpy(row[256:].copy()).view(torch.bfloat16).double().numpy()
    return torch.from_numpy(out)


def pack(rows):
    """[..., 512] bf16 -> [..., 384] uint8, many rows at once (finite values)."""
    x = rows.reshape(-1, DIM).double()
    n = x.shape[0]
    g = x[:, :NOPE].view(n, -1, GROUP)
    amax = g.abs().amax(-1)
    top = amax.amax(-1)
    e = torch.where(top > 0, torch.frexp(top).exponent - 1, -113).clamp(min=-113)
    two = lambda k: torch.ldexp(torch.ones_like(k, dtype=torch.float64), k)  # noqa: E731
    want = amax / 7 * two(10 - e)[:, None]
    table = torch.from_numpy(E4M3)
    i = torch.searchsorted(table, want).clamp(1, 126)
    below, above = want - table[i - 1], table[i] - want
    s = torch.where((below < above) | ((below == above) & ((i - 1) % 2 == 0)), i - 1, i)
    s = torch.where(want == 0, 0, s)
    unit = (table[s] * two(e - 10)[:, None])[..., None]
    code = torch.where(unit > 0, (g / unit.clamp(min=2.0 ** -140)).round(), 0.0).clamp(-7, 7) + 8
    code = code.view(n, NOPE).to(torch.int64)
    out = torch.zeros(n, ROW, dtype=torch.int64)
    d = torch.arange(NOPE)
    chunk, half, nib = d // 64, d // 32 % 2, d % 8 // 2 + 4 * (d % 2)
    for k in range(8):                       # (one nibble of every byte at a time)
        at = nib == k
        where = (32 * (chunk + 1) + 16 * half + 4 * (d // 8 % 4) + nib // 2)[at]
        out[:, where] |= code[:, at] << 4 * (k % 2)
    first = d % GROUP == 0
    out[:, (16 * half + 2 * chunk + d // 16 % 2)[first]] = s
    out[:, 14] = out[:, 30] = e + 127
    out = out.to(torch.uint8)
    out[:, 256:] = rows.reshape(-1, DIM)[:, NOPE:].contiguous().view(torch.uint8)
    return out.view(*rows.shape[:-1], ROW)


def unpack(pages):
    """[..., 384] uint8 -> [..., 512] float64, many rows at once."""
    row = pages.reshape(-1, ROW)
    d = torch.arange(NOPE)
    chunk, half, nib = d // 64, d // 32 % 2, d % 8 // 2 + 4 * (d % 2)
    byte = row[:, 32 * (chunk + 1) + 16 * half + 4 * (d // 8 % 4) + nib // 2].int()
    code = ((byte >> 4 * (nib % 2)) & 15).double() - 8
    s = row[:, 16 * half + 2 * chunk + d // 16 % 2].long()
    table = torch.from_numpy(np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]]))
    e = row[:, 14].int() - 137
    unit = torch.ldexp(torch.ones_like(e, dtype=torch.float64), e)[:, None]
    rope = row[:, 256:].contiguous().view(torch.bfloat16).double()
    return torch.cat([code * table[s] * unit, rope], -1).view(*pages.shape[:-1], DIM)


def append(batch, kv):
    """(pages, allowed error of the rotated dims): uint8 pages after the append."""
    pages = batch["pages"].clone()
    tol = torch.zeros(*pages.shape[:2], ROPE, dtype=torch.float64)
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
                pair = x[NOPE:].abs().view(-1, 2).sum(-1).repeat_interleave(2)
                x = turn(x, batch["cos_sin"][p])
                tol[at] = 2 * U * x[NOPE:].abs() + 4 * 2.0 ** -24 * pair
            pages[at] = encode(x)
    return pages, tol


def visible(t, window, sinks):
    low = max(0, t - window + 1) if window else 0
    return list(range(min(sinks if window else 0, low))) + list(range(low, t + 1))


def attention(batch, q, window, sinks, scale, q_turned=False):
    """(out, allowed error, rows that are written) in float64; rows of no valid sequence NaN."""
    n_new, heads = q.shape[:2]
    out = torch.full((n_new, heads, DIM), float("nan"), dtype=torch.float64)
    tol = torch.zeros_like(out)
    written = np.zeros(n_new, dtype=bool)
    pages, cs = unpack(batch["pages"]), batch["cos_sin"]
    for s in range(len(batch["seq_len"])):
        if not valid(batch, s, n_new):
            continue
        r0, r1 = int(batch["new_start"][s]), int(batch["new_start"][s + 1])
        for r in range(r0, r1):
            t = int(batch["seq_len"][s]) - r1 + r
            written[r] = True
            at = [place(batch, s, u) for u in visible(t, window, sinks)]
            at = [a for a in at if a is not None]
            if not at:
                out[r] = 0.0
                continue
            a = torch.tensor(at)
            kv = pages[a[:, 0], a[:, 1]]
            qr = q[r].double()
            rounds = cs is not None and not q_turned
            if rounds:
                qr = turn(qr, cs[t])
            logits = scale * qr @ kv.T
            w = torch.softmax(logits, -1)
            o = w @ kv
            big = w @ kv.abs()
            if cs is not None:
                o = turn(o, cs[t], -1.0)
                b = big[:, NOPE:].view(heads, -1, 2).sum(-1).repeat_interleave(2, -1)
                big = torch.cat([big[:, :NOPE], b], -1)
            size = scale * (qr.abs() @ kv.abs().T).amax(-1)
            e = 512 * 2.0 ** -23 * size + 2.0 ** -22 * 1.45 * (logits.abs().amax(-1) + 16)
            if rounds:
                e = e + U * scale * (qr[:, NOPE:].abs() @ kv[:, NOPE:].abs().T).amax(-1)
            spread = torch.expm1(2 * e) + 2.02 * U + 2.0 ** -20 + len(at) * 2.0 ** -23
            out[r] = o
            tol[r] = U * o.abs() + big * spread[:, None]
    return out, tol, written


def norm(x, weight, eps, cs):
    """(y, allowed error) of rows [..., 512], cs [32, 2] or None."""
    x = x.double()
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        y = y * weight.double()
    size = y.abs()
    if cs is not None:
        pair = size[..., NOPE:].unflatten(-1, (-1, 2)).sum(-1).repeat_interleave(2, -1)
        size = torch.cat([size[..., :NOPE], pair], -1)
        y = turn(y, cs)
    return y, U * y.abs() + size * (2.0 ** -15 + 2.0 ** -22)


def make(lens, page=16, extra_pages=3, rope=True, seed=0, max_pages=None):
    """A CPU batch of sequences [(new, total)], every page filled, in shuffled pages."""
    import paged_ref
    batch = paged_ref.make(lens, page, extra_pages, rope, seed, max_pages)
    batch["pages"] = pack(batch["pages"])
    return batch
