"""Plain 64-bit forms of the paged-cache operators for the parity tests (torch, CPU)."""
import math

import torch

BLOCK = 16
E_MIN, E_MAX = -110, 120


def plan_ref(seq, new, table, free, used, total, cap):
    """A step's plan, one token after another."""
    table = table.clone()
    cu, pos, slots, lens = [0], [], [], []
    for b, (s, n) in enumerate(zip(seq.tolist(), new.tolist())):
        for i in range(n):
            p = s + i
            if p % BLOCK == 0:
                table[b, p // BLOCK] = free[used]
                used += 1
            pos.append(p)
            slots.append(int(table[b, p // BLOCK]) * BLOCK + p % BLOCK)
        cu.append(len(pos))
        lens.append(s + n)
    fill = [-1] * (total - len(pos))
    t = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return t(lens), t(cu), t(pos + fill), t(slots + fill), t([used]), table


def frequencies(rotary_dim, base=10000.0):
    return torch.tensor([base ** (-2 * i / rotary_dim) for i in range(rotary_dim // 2)], dtype=torch.float64)


def rotate_ref(x, pos, freq, mag=1.0, interleaved=False, inverse=False):
    """x [..., rows, heads?, D] in 64 bits; pos broadcasts against x's leading dims. Returns (y, |x1| + |x2| of each element)."""
    r = 2 * freq.numel()
    a = pos.double()[..., None] * freq * (-1.0 if inverse else 1.0)
    c, s = torch.cos(a) * mag, torch.sin(a) * mag
    y, size = x.clone(), torch.zeros_like(x)
    if interleaved:
        i1, i2 = slice(0, r, 2), slice(1, r, 2)
    else:
        i1, i2 = slice(0, r // 2), slice(r // 2, r)
    x1, x2 = x[..., i1], x[..., i2]
    y[..., i1], y[..., i2] = x1 * c - x2 * s, x2 * c + x1 * s
    size[..., i1] = size[..., i2] = (x1.abs() + x2.abs()) * abs(mag)
    return y, size


# A turned element's error, relative to (|x1| + |x2|) * magnitude: the angle's
# remainder is rounded to fp32 (2^-25 half turns, 2^-23.3 rad), sine and cosine
# to 2^-23 at most, magnitude * cosine and the two products and their sum add
# three roundings of 2^-24: below 2^-21 together.
TURN_REL = 2.0 ** -21


def values(codes, scales):
    """What a cache's codes (uint8) and exponent bytes stand for, 64 bits [NB, H, 16, D]."""
    v = codes.view(torch.float8_e4m3fn).double()
    return v * torch.exp2(scales.double() - 127)[:, :, None, None]


def exponent(amax):
    """The smallest e of [E_MIN, E_MAX] with amax <= 448 * 2^e (a float)."""
    if amax == 0.0:
        return E_MIN
    e = math.frexp(amax / 448.0)[1]
    if amax <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    return min(max(e, E_MIN), E_MAX)


def dense(vals, table, lens, width):
    """[B, H, width, D] of page values [NB, H, 16, D]; zero behind the lengths."""
    B, H, D = table.shape[0], vals.shape[1], vals.shape[3]
    out = torch.zeros(B, H, width, D, dtype=vals.dtype)
    for b in range(B):
        n = min(int(lens[b]), width)
        if n > 0:
            ids = table[b, : (n + BLOCK - 1) // BLOCK].long()
            out[b, :, :n] = vals[ids].transpose(0, 1).reshape(H, -1, D)[:, :n]
    return out


def attend_ref(q, k, v, scale, limit):
    """q [Hk, R, D], k, v [Hk, S, D] in 64 bits; row r sees keys [0, limit[r]).

    Returns (O, LSE, sum p |v|, max score size, max weight part): the sizes that
    the tolerances are made of. Rows that see nothing give O = 0, LSE = -inf.
    """
    S = k.shape[1]
    sees = torch.arange(S)[None, :] < limit[:, None]
    x = scale * q @ k.transpose(1, 2)
    x = x.masked_fill(~sees[None], -math.inf)
    lse = torch.logsumexp(x, -1) if S else torch.full(x.shape[:2], -math.inf, dtype=torch.float64)
    p = torch.exp(x - torch.where(torch.isinf(lse), 0.0, lse)[..., None])
    p = p.masked_fill(~sees[None], 0.0)
    size = (scale * q.abs() @ k.abs().transpose(1, 2)).masked_fill(~sees[None], 0.0)
    return p @ v, lse, p @ v.abs(), (size.amax(-1) if S else torch.zeros(x.shape[:2], dtype=torch.float64)), p


def random_cache(g, num_blocks, heads, dim, table, lens, spread=3.0):
    """Codes and scales whose live tokens are random and everything else is NaN (code 0x7f, scale byte 255).

    The scales of a sequence's blocks differ by powers of two around 2^-spread .. 2^spread.
    """
    codes = torch.full((num_blocks, heads, BLOCK, dim), 0x7F, dtype=torch.uint8)
    scales = torch.full((num_blocks, heads), 255, dtype=torch.uint8)
    for b in range(table.shape[0]):
        n = int(lens[b])
        for j in range((n + BLOCK - 1) // BLOCK):
            blk, live = int(table[b, j]), min(BLOCK, n - j * BLOCK)
            x = torch.randn(heads, live, dim, generator=g) * torch.exp2(
                (torch.rand(heads, 1, 1, generator=g) * 2 - 1) * spread)
            for h in range(heads):
                e = exponent(float(x[h].abs().max()))
                codes[blk, h, :live] = (x[h].double() * 2.0 ** -e).float().to(torch.float8_e4m3fn).view(torch.uint8)
                scales[blk, h] = e + 127
    return codes, scales


def tables(g, lens, width, spare=3):
    """Shuffled distinct pages for each sequence's tokens, -1 behind them; returns (table, num_blocks)."""
    need = [(int(n) + BLOCK - 1) // BLOCK for n in lens]
    num = sum(need) + spare
    order = torch.randperm(num, generator=g).to(torch.int32)
    table = torch.full((len(need), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, num
