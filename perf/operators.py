"""Cases of the paged-cache operators, for measuring them.

The operators are those of one serving step over a paged key/value cache, and
of training next to the dense prefill:

* ``plan``    block tables, positions and slots of a step from request lengths;
* ``rotary``  rotary positions on queries and keys, and its gradient;
* ``append``  queries and keys rotated, keys and values written into the pages
              (bf16, or E4M3 codes with a power-of-two scale for each block of
              16 tokens and head), read back as the values the pages stand for;
* ``decode``  one query token per sequence over the 8-bit pages;
* ``prefill`` chunks of queries over the 8-bit pages, causal bottom-right.

With ``own`` false, :func:`run` computes them with elementary torch operations
in 32 bits; with ``own`` true it makes the library's calls.
"""
import math

import torch

own = False

BLOCK = 16          # tokens of a cache block
E_MIN, E_MAX = -110, 120  # exponents of the block scales
DEV = "cuda"


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 64 sequences of up to 32K tokens: the smallest, latency alone counts
        dict(name="plan_decode_b64", op="plan", batch=64, max_new=1, context=32768),
        # admission of a ragged batch of prompts, some requests idle
        dict(name="plan_prompts_b300", op="plan", batch=300, max_new=1500, context=4096),
        # the query and key rows of one decode step
        dict(name="rotary_step_t64", op="rotary", packed=True, batch=1, seqlen=64, q_heads=32, kv_heads=8, head_dim=128,
             rotary_dim=128, interleaved=False, inverse=False, f32=False, scaling="none", start=32000),
        # training forward at the dense prefill's shape
        dict(name="rotary_4x32x2048", op="rotary", packed=False, batch=4, seqlen=2048, q_heads=32, kv_heads=8, head_dim=128,
             rotary_dim=128, interleaved=False, inverse=False, f32=False, scaling="none", start=0),
        # gradient of a partial, interleaved rotation at an odd length, fp32 as the backward returns it
        dict(name="rotary_grad_2x12x1999", op="rotary", packed=False, batch=2, seqlen=1999, q_heads=12, kv_heads=4, head_dim=64,
             rotary_dim=32, interleaved=True, inverse=True, f32=True, scaling="by_parts", start=0),
        # one decode step's tokens into the 8-bit pages, short contexts
        dict(name="append_step_b32", op="append", batch=32, max_new=1, context=40, q_heads=32, kv_heads=8, head_dim=128,
             rotary_dim=128, interleaved=False, fp8=True, scaling="none"),
        # prompt chunks into the 8-bit pages, blocks that are partly filled already
        dict(name="append_chunks_b9", op="append", batch=9, max_new=1400, context=700, q_heads=32, kv_heads=8, head_dim=128,
             rotary_dim=64, interleaved=False, fp8=True, scaling="by_parts"),
        # a single request answering: latency
        dict(name="decode_b1_4097", op="decode", batch=1, lo=4097, hi=4097, q_heads=32, kv_heads=8, head_dim=128),
        # a full decode batch, 1K to 32K tokens
        dict(name="decode_b64_1k_32k", op="decode", batch=64, lo=1024, hi=32768, q_heads=32, kv_heads=8, head_dim=128),
        # odd sizes: group of three, head_dim 64, sequences of no and of one token among them
        dict(name="decode_b17_d64_g3", op="decode", batch=17, lo=0, hi=9000, q_heads=12, kv_heads=4, head_dim=64),
        # a ragged batch of chunks over earlier context
        dict(name="prefill_b5_chunk300", op="prefill", batch=5, chunk=300, context=3000, q_heads=16, kv_heads=4, head_dim=128),
        # a long prompt's late chunk
        dict(name="prefill_b1_2048_32k", op="prefill", batch=1, chunk=2048, context=30000, q_heads=32, kv_heads=8, head_dim=128),
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("plan", "rotary", "append", "decode", "prefill"))
    if op == "plan":
        batch = _log_int(rng, 1, 700)
        most = rng.choice((1, _log_int(rng, 2, 3000)))
        return dict(op=op, batch=batch, max_new=min(most, 450000 // batch), context=_log_int(rng, 1, 32768))
    kv, group = rng.choice((1, 2, 3, 4, 8)), rng.choice((1, 2, 3, 4, 5, 8))
    heads = dict(q_heads=kv * group, kv_heads=kv, head_dim=rng.choice((64, 128)))
    if op == "rotary":
        packed = rng.random() < 0.5
        batch = 1 if packed else rng.randint(1, 4)
        return dict(op=op, packed=packed, batch=batch, seqlen=_log_int(rng, 1, 8192 // batch), **heads,
                    rotary_dim=rng.choice((16, 32, 48, 64, heads["head_dim"])), interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.4, f32=rng.random() < 0.3,
                    scaling=rng.choice(("none", "linear", "base", "by_parts")), start=rng.choice((0, _log_int(rng, 1, 1000000))))
    if op == "append":
        batch = _log_int(rng, 1, 64)
        return dict(op=op, batch=batch, max_new=rng.choice((1, _log_int(rng, 2, max(2, 8192 // batch)))),
                    context=_log_int(rng, 1, max(2, 8192 // batch)), **heads, rotary_dim=rng.choice((32, 64, heads["head_dim"])),
                    interleaved=rng.random() < 0.5, fp8=rng.random() < 0.7, scaling=rng.choice(("none", "linear", "base", "by_parts")))
    if op == "decode":
        batch = _log_int(rng, 1, 64)
        hi = min(_log_int(rng, 1, 32768), (1 << 20) // batch)
        return dict(op=op, batch=batch, lo=rng.randint(0, hi), hi=hi, **heads)
    return dict(op=op, batch=rng.randint(1, 6), chunk=_log_int(rng, 1, 512), context=_log_int(rng, 1, 6000), **heads)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _frequencies(case):
    """Angles per position of each pair, in 64 bits, and the factor on the rotated elements."""
    r, base, factor, length = case["rotary_dim"], 10000.0, 4.0, 4096
    i = torch.arange(0, r, 2, dtype=torch.float64, device=DEV) / r
    scaling = case["scaling"]
    if scaling == "base" and r > 2:
        base = base * factor ** (r / (r - 2))
    f = base ** -i
    if scaling == "linear":
        f = f / factor
    if scaling == "by_parts":
        keep = ((length * f / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
        return f * keep + f / factor * (1 - keep), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _fixed(g, count, *ranges):
    """Ragged lengths whose sums are the case's own, dealt out to the requests by `g`."""
    h = torch.Generator(device=DEV)
    h.manual_seed(97)
    deal = torch.randperm(count, generator=g, device=DEV)
    return [_ragged(h, count, lo, hi)[deal] for lo, hi in ranges]


def _ragged(g, count, lo, hi):
    return torch.randint(lo, hi + 1, (count,), generator=g, device=DEV, dtype=torch.int32)


def _exponents(amax):
    """The smallest e of [E_MIN, E_MAX] with amax <= 448 * 2^e."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _pow2(e):
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _pool(g, blocks, heads, dim, lens, table, fp8, spread):
    """Pages holding `lens` tokens of each sequence; everything behind them and every spare block holds NaN."""
    live = torch.zeros(blocks, BLOCK, dtype=torch.bool, device=DEV)
    at = torch.arange(table.shape[1] * BLOCK, device=DEV)
    has = at[None, :] < lens[:, None]
    blk = table.long()[:, :, None].expand(-1, -1, BLOCK).reshape(table.shape[0], -1)
    live[blk[has], (at % BLOCK).expand_as(has)[has]] = True
    x = torch.randn(blocks, heads, BLOCK, dim, generator=g, device=DEV, dtype=torch.float32)
    if spread:  # keys have a few loud channels
        x.mul_(torch.exp(0.5 * torch.randn(1, heads, 1, dim, generator=g, device=DEV)))
    if not fp8:
        return x.masked_fill_(~live[:, None, :, None], math.nan).to(torch.bfloat16), None
    e = _exponents((x.abs() * live[:, None, :, None]).amax(dim=(2, 3)))
    codes = x.mul_(_pow2(-e)[:, :, None, None]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    codes.masked_fill_(~live[:, None, :, None], 0x7F)
    scales = torch.where(live.any(1)[:, None], e + 127, torch.full_like(e, 255)).to(torch.uint8)
    return codes, scales


def _tables(g, total, width, spare=5):
    """A block table of distinct, shuffled pages for each sequence, and the pages that are left."""
    pages = torch.randperm(total * width + spare, generator=g, device=DEV).to(torch.int32)
    return pages[: total * width].reshape(total, width).contiguous(), pages[total * width:].contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case=dict(case))
    op = case["op"]
    bf16 = lambda *shape: torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    if op == "plan":
        b, c, n = case["batch"], case["context"], case["max_new"]
        s["seq_lens"] = _ragged(g, b, 0, c)
        some, idle = _fixed(g, b, (0, n), (0, 7))
        s["new_lens"] = torch.ones_like(some) if n == 1 else some * (idle > 0)
        width = -(-(c + n) // BLOCK)
        s["table"], s["free"] = _tables(g, b, width, b * (-(-n // BLOCK) + 1) + 16)
        held = torch.arange(width, device=DEV)[None, :] < ((s["seq_lens"] + BLOCK - 1) // BLOCK)[:, None]
        s["table"].masked_fill_(~held, -1)
        s["blocks"] = s["table"].numel() + s["free"].numel()
        s["used"] = torch.full((1,), 3, dtype=torch.int32, device=DEV)
        s["total"] = int(s["new_lens"].sum()) + 5  # rows behind the last request
        empty = lambda k: torch.empty(k, dtype=torch.int32, device=DEV)  # noqa: E731
        s["lens_out"], s["cu"], s["pos"], s["slots"], s["used_out"] = empty(b), empty(b + 1), empty(s["total"]), empty(s["total"]), empty(1)
        return s
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if op == "rotary":
        b, t = case["batch"], case["seqlen"]
        s["freq"], s["mag"] = _frequencies(case)
        lead = lambda h: (t, h, d) if case["packed"] else (b, h, t, d)  # noqa: E731
        s["q"], s["k"] = torch.randn(lead(hq), generator=g, device=DEV), torch.randn(lead(hk), generator=g, device=DEV)
        if not case["f32"]:
            s["q"], s["k"] = s["q"].to(torch.bfloat16), s["k"].to(torch.bfloat16)
        start = case["start"] + _ragged(g, t if case["packed"] else b, 0, 1000)
        s["pos"] = start.to(torch.int32) if case["packed"] else (start[:, None] + torch.arange(t, device=DEV)[None, :]).to(torch.int32).contiguous()
        return s
    b = case["batch"]
    if op == "append":
        n, c = case["max_new"], case["context"]
        old, new = _fixed(g, b, (0, c), (1, n))
        s["lens"], s["longest"] = old + new, int((old + new).max())
        s["table"], spare = _tables(g, b, -(-s["longest"] // BLOCK))
        blocks = s["table"].numel() + spare.numel()
        s["k_cache"], s["k_scales"] = _pool(g, blocks, hk, d, old, s["table"], case["fp8"], True)
        s["v_cache"], s["v_scales"] = _pool(g, blocks, hk, d, old, s["table"], case["fp8"], False)
        seq = torch.repeat_interleave(torch.arange(b, device=DEV), new.long())
        t = seq.numel()
        first = torch.cumsum(new, 0) - new
        pos = old[seq] + torch.arange(t, device=DEV) - first[seq]
        s["pos"] = pos.to(torch.int32)
        s["slots"] = (s["table"][seq, pos // BLOCK] * BLOCK + pos % BLOCK).to(torch.int32)
        qkv = bf16(t, hq + 2 * hk, d)  # one projection's rows
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["freq"], s["mag"] = _frequencies(case)
        return s
    if op == "decode":
        lens = _ragged(g, b, case["lo"], case["hi"])
        if case["lo"] == 0 and b > 2:
            lens[1], lens[2] = 0, 1
        s["q"], s["longest"] = bf16(b, hq, d), max(1, case["hi"])
    else:
        new, = _fixed(g, b, (max(1, case["chunk"] // 2), case["chunk"]))
        lens = new + _ragged(g, b, case["context"] // 2, case["context"])
        s["cu"] = torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), torch.cumsum(new, 0).to(torch.int32)])
        s["most"], s["longest"] = case["chunk"], case["chunk"] + case["context"]
        s["q"] = bf16(int(s["cu"][-1]), hq, d)
    s["lens"] = lens
    # pages for the tokens that there are, in one shuffled pool; entries behind a sequence's own are -1
    width = -(-s["longest"] // BLOCK)
    held = torch.arange(width, device=DEV)[None, :] < ((lens + BLOCK - 1) // BLOCK)[:, None]
    blocks = int(held.sum()) + 5
    s["table"] = torch.full((b, width), blocks - 1, dtype=torch.int32, device=DEV)
    s["table"][held] = torch.randperm(blocks - 1, generator=g, device=DEV)[: int(held.sum())].to(torch.int32)
    s["k_cache"], s["k_scales"] = _pool(g, blocks, hk, d, lens, s["table"], True, True)
    s["v_cache"], s["v_scales"] = _pool(g, blocks, hk, d, lens, s["table"], True, False)
    s["table"].masked_fill_(~held, -1)
    s["scale"] = d ** -0.5
    return s


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------

def _plan_plain(s):
    seq, new, table, free = s["seq_lens"], s["new_lens"], s["table"], s["free"]
    b = seq.numel()
    had, has = (seq + BLOCK - 1) // BLOCK, (seq + new + BLOCK - 1) // BLOCK
    need = has - had
    base = s["used"] + torch.cumsum(need, 0) - need
    col = torch.arange(table.shape[1], device=seq.device)[None, :]
    fresh = (col >= had[:, None]) & (col < has[:, None])
    pick = (base[:, None] + col - had[:, None]).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[pick.long()], table))
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=seq.device), torch.cumsum(new, 0)])
    t = torch.arange(s["total"], device=seq.device)
    at = (torch.searchsorted(cu, t, right=True) - 1).clamp(0, b - 1)
    live = t < cu[-1]
    pos = seq[at] + t - cu[at]
    slot = table[at, (pos // BLOCK).clamp(0, table.shape[1] - 1)].long() * BLOCK + pos % BLOCK
    pos, slot = torch.where(live, pos, -1).to(torch.int32), torch.where(live, slot, -1).to(torch.int32)
    return dict(lens=(seq + new).to(torch.int32), cu=cu.to(torch.int32), positions=pos, slots=slot,
                used=(s["used"] + need.sum()).to(torch.int32), table=table)


def _rotate_plain(x, pos, freq, mag, interleaved, inverse):
    """x [..., rows, D] in fp32, pos [rows] of every leading index it broadcasts to."""
    r = 2 * freq.numel()
    a = pos.double().unsqueeze(-1) * freq
    cos, sin = (torch.cos(a) * mag).float(), (torch.sin(a) * (-mag if inverse else mag)).float()
    if interleaved:
        x1, x2 = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1).flatten(-2)
    else:
        x1, x2 = x[..., : r // 2], x[..., r // 2:r]
        y = torch.cat((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1)
    return torch.cat((y, x[..., r:]), -1)


def _values(codes, scales):
    if scales is None:
        return codes.float()
    return codes.view(torch.float8_e4m3fn).float() * _pow2(scales.int() - 127)[:, :, None, None]


def _write_plain(cache, scales, x, slots):
    """Rows x [T, H, D] (fp32) into the pages; a page's scale covers what it kept in front of them and what is new."""
    blk, off = (slots // BLOCK).long(), (slots % BLOCK).long()
    if scales is None:
        cache[blk, :, off] = x.to(torch.bfloat16)
        return
    nb = cache.shape[0]
    new = torch.zeros(nb, BLOCK, dtype=torch.bool, device=x.device)
    new[blk, off] = True
    at = torch.arange(BLOCK, device=x.device)
    first = torch.where(new, at, BLOCK).amin(1)
    touched = first < BLOCK
    kept = (at[None, :] < first[:, None]) & touched[:, None]
    value = torch.where(kept[:, None, :, None], _values(cache, scales), 0.0)
    value[blk, :, off] = x
    e = _exponents(value.abs().amax(dim=(2, 3)))
    code = (value * _pow2(-e)[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    cache.copy_(torch.where((kept | new)[:, None, :, None], code, cache))
    scales.copy_(torch.where(touched[:, None], (e + 127).to(torch.uint8), scales))


def _dense_plain(cache, scales, table, lens, width):
    """Each sequence's tokens [B, H, width, D] in fp32, zero behind its length."""
    v = _values(cache, scales)[table.long().clamp(min=0)]
    b, nb, h, _, d = v.shape
    v = v.permute(0, 2, 1, 3, 4).reshape(b, h, nb * BLOCK, d)[:, :, :width]
    return v.masked_fill_((torch.arange(width, device=v.device)[None, :] >= lens[:, None])[:, None, :, None], 0.0)


def _attend_plain(q, k, v, sees, scale):
    """q [B, Hk, R, D], k and v [B, Hk, S, D], sees [B, 1, R, S]: outputs and log-sum-exps."""
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(~sees, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / torch.where(total > 0, total, 1.0)
    return o, (m + torch.log(total)).squeeze(-1)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "plan":
        return _plan_plain(s)
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if op == "rotary":
        pos = s["pos"][:, None] if case["packed"] else s["pos"][:, None, :]
        turn = lambda x: _rotate_plain(x.float(), pos, s["freq"], s["mag"], case["interleaved"], case["inverse"]).to(x.dtype)  # noqa: E731
        return dict(q=turn(s["q"]), k=turn(s["k"]))
    if op == "append":
        turn = lambda x: _rotate_plain(x.float(), s["pos"][:, None], s["freq"], s["mag"], case["interleaved"], False)  # noqa: E731
        _write_plain(s["k_cache"], s["k_scales"], turn(s["k"]), s["slots"])
        _write_plain(s["v_cache"], s["v_scales"], s["v"].float(), s["slots"])
        dense = lambda c, e: _dense_plain(c, e, s["table"], s["lens"], s["longest"]).to(torch.bfloat16)  # noqa: E731
        return dict(q=turn(s["q"]).to(torch.bfloat16), k=dense(s["k_cache"], s["k_scales"]), v=dense(s["v_cache"], s["v_scales"]))
    width = s["table"].shape[1] * BLOCK
    k = _dense_plain(s["k_cache"], s["k_scales"], s["table"], s["lens"], width)
    v = _dense_plain(s["v_cache"], s["v_scales"], s["table"], s["lens"], width)
    b, group, key = case["batch"], hq // hk, torch.arange(width, device=DEV)
    if op == "decode":
        sees = (key[None, :] < s["lens"][:, None])[:, None, None, :]
        o, lse = _attend_plain(s["q"].float().reshape(b, hk, group, d), k, v, sees, s["scale"])
        return dict(o=o.reshape(b, hq, d).to(torch.bfloat16), lse=lse.reshape(b, hq))
    cu, most = s["cu"].long(), s["most"]
    new = cu[1:] - cu[:-1]
    row = torch.arange(most, device=DEV)
    real = row[None, :] < new[:, None]
    at = (cu[:-1, None] + row[None, :]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][at].float().reshape(b, most, hk, group, d).permute(0, 2, 3, 1, 4).reshape(b, hk, group * most, d)
    sees = key[None, None, :] <= row[None, :, None] + (s["lens"] - new)[:, None, None]
    o, lse = _attend_plain(q, k, v, sees.repeat(1, group, 1)[:, None], s["scale"])
    o = o.reshape(b, hk, group, most, d).permute(0, 3, 1, 2, 4).reshape(b, most, hq, d)[real]
    lse = lse.reshape(b, hq, most).permute(0, 2, 1)[real].transpose(0, 1)
    return dict(o=o.to(torch.bfloat16), lse=lse.contiguous())


# ----------------------------------------------------------------------------
# the library's calls
# ----------------------------------------------------------------------------

def _run_own(s):
    from attention_tiled_exact_b200 import binding as attn
    case = s["case"]
    op = case["op"]
    if op == "plan":
        attn.plan_paged_step(s["seq_lens"], s["new_lens"], s["table"], s["free"], s["used"], s["total"], s["blocks"],
                             seq_lens_out=s["lens_out"], cu_seqlens_q=s["cu"], positions=s["pos"], slot_map=s["slots"],
                             num_used_out=s["used_out"])
        return dict(lens=s["lens_out"], cu=s["cu"], positions=s["pos"], slots=s["slots"], used=s["used_out"], table=s["table"])
    if op == "rotary":
        q, k = attn.rotary(s["q"], s["k"], s["freq"], s["pos"], interleaved=case["interleaved"], inverse=case["inverse"],
                           magnitude=s["mag"])
        return dict(q=q, k=k)
    if op == "append":
        q = attn.append_paged(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], q=s["q"],
                              inv_freq=s["freq"], positions=s["pos"], interleaved=case["interleaved"], magnitude=s["mag"])
        k, v = attn.gather_paged(s["k_cache"], s["v_cache"], s["table"], s["lens"], s["longest"], s["k_scales"], s["v_scales"])
        return dict(q=q, k=k, v=v)
    if op == "decode":
        o, lse = attn.decode_paged_block_scaled(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"],
                                                s["lens"], scale=s["scale"], max_seq_len=s["longest"])
        return dict(o=o, lse=lse)
    o, lse = attn.prefill_paged_block_scaled(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"], s["lens"],
                                             scale=s["scale"], causal=True, cu_seqlens_q=s["cu"], max_seqlen_q=s["most"],
                                             max_seqlen_k=s["longest"])
    return dict(o=o, lse=lse)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    op, b = case["op"], case["batch"]
    if op == "plan":
        tokens = b if case["max_new"] == 1 else b * case["max_new"] * 7 / 16  # an eighth of the requests add none
        return dict(bytes=16 * b + 8 * tokens + 8 * tokens / BLOCK, flops=0)
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if op == "rotary":
        rows = b * case["seqlen"] * (hq + hk)
        return dict(bytes=rows * d * 2 * (4 if case["f32"] else 2), flops=rows * case["rotary_dim"] * 3)
    if op == "append":
        tokens = b * (1 if case["max_new"] == 1 else (1 + case["max_new"]) / 2)
        kept = b * case["context"] / 2
        size = 1 if case["fp8"] else 2
        # rows in, rotated queries out, pages out; pages in again and their values out
        return dict(bytes=tokens * d * (4 * hq + 4 * hk + 2 * hk * size) + (tokens + kept) * hk * d * (2 * size + 4),
                    flops=tokens * (hq + hk) * case["rotary_dim"] * 3)
    if op == "decode":
        keys = b * (case["lo"] + case["hi"]) / 2
        return dict(bytes=keys * hk * (2 * d + 2 / BLOCK) + b * hq * (4 * d + 4), flops=4 * keys * hq * d)
    new = 0.75 * case["chunk"]
    keys = 0.75 * case["context"] + new
    return dict(bytes=b * (keys * hk * 2 * d + new * hq * (4 * d + 4)), flops=4 * b * hq * d * new * (keys - new / 2))


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def _turned(x, angle, mag, interleaved):
    """Rotation of x [..., D] (64 bits) as a product of complex numbers, angle [..., r / 2]."""
    r = 2 * angle.shape[-1]
    head = x[..., :r]
    z = torch.view_as_complex(head.unflatten(-1, (-1, 2)).contiguous()) if interleaved else torch.complex(*(h.contiguous() for h in head.chunk(2, -1)))
    z = z * torch.polar(torch.full_like(angle, mag), angle)
    y = torch.view_as_real(z).flatten(-2) if interleaved else torch.cat((z.real, z.imag), -1)
    return torch.cat((y, x[..., r:]), -1)


def _e4m3(x):
    """x rounded to the E4M3 grid (3 fraction bits, steps of 2^-9 below 2^-6), ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _stored(x, dims):
    """What a page's scale and codes make of its tokens x (64 bits)."""
    top = x.abs().amax(dims, keepdim=True)
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -300) / 448))
    e = torch.where(448 * torch.exp2(e - 1) >= top, e - 1, e).clamp(E_MIN, E_MAX)
    return _e4m3(x * torch.exp2(-e)) * torch.exp2(e)


def _page_values(cache, scales, ids):
    """Tokens [H, n * 16, D] of the listed pages, 64 bits."""
    if scales is None:
        v = cache[ids].double()
    else:
        v = cache[ids].view(torch.float8_e4m3fn).double() * torch.exp2(scales[ids].double() - 127)[:, :, None, None]
    return v.transpose(0, 1).flatten(1, 2)


def _softmax64(q, k, v, scale, limit):
    """q [H, R, D], k and v [H, S, D], row r sees keys below limit[r]."""
    x = scale * torch.matmul(q, k.transpose(1, 2))
    x = x.masked_fill(torch.arange(k.shape[1], device=q.device)[None, None, :] >= limit[None, :, None], -math.inf)
    lse = torch.logsumexp(x, -1)
    return torch.matmul(torch.exp(x - lse[..., None]), v), lse


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    op, d = case["op"], case["head_dim"]
    hq, hk = case["q_heads"], case["kv_heads"]
    if op == "rotary":
        angle = (s["pos"].double()[..., None] * s["freq"] * (-1.0 if case["inverse"] else 1.0)).unsqueeze(1)
        return {n: _turned(s[n].double(), angle.expand(*s[n].shape[:-1], -1), s["mag"], case["interleaved"]) for n in ("q", "k")}
    if op == "append":
        angle = (s["pos"].double()[:, None] * s["freq"])[:, None]
        turned = {n: _turned(s[n].double(), angle.expand(-1, s[n].shape[1], -1), s["mag"], case["interleaved"]) for n in ("q", "k")}
        rows = {"k": turned["k"], "v": s["v"].double()}
        out = {n: torch.zeros(case["batch"], hk, s["longest"], d, dtype=torch.float64, device=DEV) for n in rows}
        lens, pos = s["lens"].tolist(), s["pos"].tolist()
        t = 0
        for b, n in enumerate(lens):
            first = pos[t]
            count = n - first
            pages = -(-n // BLOCK)
            for name in rows:
                x = _page_values(s[name + "_cache"], s[name + "_scales"], s["table"][b, :pages].long())
                x[:, n:] = 0.0
                x[:, first:n] = rows[name][t:t + count].transpose(0, 1)
                if s[name + "_scales"] is not None:
                    at = first // BLOCK * BLOCK
                    x[:, at:] = _stored(x[:, at:].unflatten(1, (-1, BLOCK)), (2, 3)).flatten(1, 2)
                out[name][b, :, :n] = x[:, :n]
            t += count
        return dict(q=turned["q"], **out)
    group, lens = hq // hk, s["lens"].tolist()
    if op == "decode":
        o = torch.zeros(case["batch"], hq, d, dtype=torch.float64, device=DEV)
        lse = torch.full((case["batch"], hq), -math.inf, dtype=torch.float64, device=DEV)
        for b, n in enumerate(lens):
            if n:
                ids = s["table"][b, : -(-n // BLOCK)].long()
                k, v = (_page_values(s[c + "_cache"], s[c + "_scales"], ids)[:, :n] for c in "kv")
                y, z = _softmax64(s["q"][b].double().reshape(hk, group, d), k, v, s["scale"], torch.full((group,), n, device=DEV))
                o[b], lse[b] = y.reshape(hq, d), z.reshape(hq)
        return dict(o=o, lse=lse)
    cu = s["cu"].tolist()
    o = torch.zeros(cu[-1], hq, d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(hq, cu[-1], dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        ids = s["table"][b, : -(-n // BLOCK)].long()
        k, v = (_page_values(s[c + "_cache"], s[c + "_scales"], ids)[:, :n] for c in "kv")
        rows = cu[b + 1] - cu[b]
        limit = torch.arange(n - rows + 1, n + 1, device=DEV)
        for h in range(hq):
            y, z = _softmax64(s["q"][cu[b]:cu[b + 1], h].double()[None], k[h // group][None], v[h // group][None], s["scale"], limit)
            o[cu[b]:cu[b + 1], h], lse[h, cu[b]:cu[b + 1]] = y[0], z[0]
    return dict(o=o, lse=lse)
