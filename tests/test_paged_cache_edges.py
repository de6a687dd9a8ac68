"""What the operators of a serving step over a paged cache do at their edges: requests over
their limits, scales far apart, far positions, paths that only some sizes take, faults."""
import ctypes
import math
from decimal import Decimal, getcontext
from fractions import Fraction

import pytest
import torch

from tests import paged_cache_ref as ref
from tests.test_paged_cache import _attention_tol, _decode_case, _decode_run, _decode_want, _gen, _i32, _within

gpu = pytest.mark.gpu
STRUCTS = ("PlanParams", "RotaryParams", "AppendParams", "GatherParams", "DecodeParams", "PrefillParams")


def test_packed_parameters_fill_the_structs(lib):
    """The bytes that the calls pass are as long as the C struct, which may be copied as a whole."""
    for cls in (getattr(lib, name) for name in STRUCTS):
        args = [i + 0.5 if t is ctypes.c_float else i + 1 for i, (_, t) in enumerate(cls._fields_)]
        packed = lib._packer(cls)(*args)
        assert len(packed) == ctypes.sizeof(cls) and packed == bytes(cls(*args)), cls.__name__


# ---------------------------------------------------------------------------- plan: requests over their limits


def _plan_by_rows(seq, new, table, free, used, total, cap):
    """A step's plan row by row: request b's rows begin behind all that the requests in front of it ask for."""
    table, lens, cu, start, end = table.clone(), [], [], 0, 0
    pos, slots = [-1] * total, [-1] * total
    for b, (s, asked) in enumerate(zip(seq.tolist(), new.tolist())):
        s = min(max(s, 0), cap)
        cu.append(start)
        had = s
        for i in range(max(asked, 0)):
            row = start + i
            if had + i >= cap or row >= total:
                break
            if s % 16 == 0:
                table[b, s // 16] = free[used]
                used += 1
            pos[row], slots[row] = s, int(table[b, s // 16]) * 16 + s % 16
            s, end = s + 1, row + 1
        lens.append(s)
        start += max(asked, 0)
    cu = [min(c, end) for c in cu] + [end]
    return [_i32(x) for x in (lens, cu, pos, slots, [used])] + [table]


@gpu
@pytest.mark.parametrize("batch,most,every,clip", [(3, 9, 2, 0), (64, 1, 5, 0), (64, 1, 64, 0), (300, 40, 7, 0), (2300, 1, 3, 0),
                                                   (2300, 5, 900, 0), (300, 40, 7, 500), (64, 3, 1, 0), (2300, 4, 5, 2000)])
@pytest.mark.parametrize("in_place", [True, False])
def test_plan_keeps_the_rows_behind_a_request_over_its_limit(lib, batch, most, every, clip, in_place):
    g = _gen(batch + most)
    width = 4
    cap = width * 16
    seq = torch.randint(0, cap - most, (batch,), generator=g)
    new = torch.randint(1 if most == 1 else 0, most + 1, (batch,), generator=g)
    over = torch.arange(batch) % every == every // 2
    seq[over] = cap - torch.randint(0, 2, (int(over.sum()),), generator=g)  # full, or one token short of it
    new[over] += torch.randint(1, 4, (int(over.sum()),), generator=g)
    if batch > 3:
        seq[0], new[batch - 2], seq[batch - 3] = -5, -3, cap + 9
    pages = torch.randperm(3 * batch * width, generator=g).to(torch.int32)
    table, free = pages[: batch * width].reshape(batch, width).clone(), pages[batch * width:].contiguous()
    total = int(new.clamp(min=0).sum()) + 4 - clip
    want = _plan_by_rows(seq, new, table, free, 2, total, cap)
    d = [t.cuda() for t in (_i32(seq), _i32(new), table, free, _i32([2]))]
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    state = dict(seq_lens_out=d[0], num_used_out=d[4]) if in_place else {}
    out = lib.plan_paged_step(*d, total, 3 * batch * width, error_flags=flags, **state)
    for name, a, b in zip(("lens", "cu", "positions", "slots", "used", "table"), list(out) + [d[2]], want):
        assert torch.equal(a.cpu(), b), name
    assert int(flags.item()) == lib.ATTN_FAULT_BAD_LENGTH


@gpu
def test_a_full_sequence_leaves_the_others_alone(lib):
    """One decode step with a sequence whose table row is full: the others' tokens go to their own pages."""
    Hq, Hk, D, width = 4, 2, 64, 2
    seq, new = _i32([7, 32, 31, 16]), _i32([1, 1, 1, 1])
    table = _i32([[0, -1], [1, 2], [3, 4], [5, -1]])
    kc, vc = (torch.zeros(9, Hk, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rows = torch.randn(4, Hq + 2 * Hk, D, generator=_gen(1)).to(torch.bfloat16).cuda()
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    freq = ref.frequencies(D).cuda()
    t = table.cuda()
    lens, cu, pos, slots, used = lib.plan_paged_step(seq.cuda(), new.cuda(), t, _i32([6, 7]).cuda(), _i32([0]).cuda(), 4, 9,
                                                     error_flags=flags)
    assert int(flags.item()) == lib.ATTN_FAULT_BAD_LENGTH
    assert pos.tolist() == [7, -1, 31, 16] and slots.tolist() == [7, -1, 79, 96] and lens.tolist() == [8, 32, 32, 17]
    assert cu.tolist() == [0, 1, 2, 3, 4] and used.tolist() == [1]
    q = lib.append_paged(rows[:, Hq:Hq + Hk], rows[:, Hq + Hk:], slots, kc, vc, q=rows[:, :Hq], inv_freq=freq, positions=pos)
    alone = lib.rotary(rows[:, :Hq + Hk], None, freq, _i32([7, 0, 31, 16]).cuda())[0]
    for b, (blk, off) in {0: (0, 7), 2: (4, 15), 3: (6, 0)}.items():
        assert torch.equal(q[b], alone[b, :Hq]) and torch.equal(kc[blk, :, off], alone[b, Hq:])
        assert torch.equal(vc[blk, :, off], rows[b, Hq + Hk:])
        kc[blk, :, off] = vc[blk, :, off] = 0
    assert not kc.any() and not vc.any()


# ---------------------------------------------------------------------------- prefill over the 8-bit pages: paths that only some sizes take


@gpu
def test_prefill_block_scaled_of_no_keys_in_a_large_batch(lib):
    """More row tiles than the few-rows kernel's grid has, and a bound of no keys: rows of 0, longer sequences flagged."""
    B, D = 65600, 64
    q = torch.randn(B, 1, D, generator=_gen(3)).to(torch.bfloat16).cuda()
    pool, scales = torch.zeros(2, 1, 16, D, dtype=torch.uint8, device="cuda"), torch.full((2, 1), 127, dtype=torch.uint8, device="cuda")
    table, lens = torch.zeros(B, 1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    for over in (0, 1):
        lens[B - 3] = over
        o, lse = lib.prefill_paged_block_scaled(q, pool, pool, scales, scales, table, lens, cu_seqlens_q=cu, max_seqlen_q=1,
                                                max_seqlen_k=0, error_flags=flags)
        assert (o == 0).all() and torch.isneginf(lse).all()
        assert int(flags.item()) == (lib.ATTN_FAULT_BAD_LENGTH if over else 0)


def _prefill_path(lib, B, Hq, Hk, D, rows, keys):
    """Which kernel a chunk takes, from its workspace: "few" rows, or the tensor-core tiles with the keys of an item in
    "whole" or dealt out in "shares"."""
    p, need = lib.PrefillParams(), ctypes.c_size_t(0)
    for name in ("q", "o", "seqlens_k", "k_cache", "v_cache", "block_table"):
        setattr(p, name, 1 << 20)  # never read
    p.batch, p.num_q_heads, p.num_kv_heads, p.head_dim, p.seqlen_q, p.seqlen_k = B, Hq, Hk, D, rows, keys
    p.scale, p.max_blocks_per_seq, p.num_blocks, p.block_size = 1.0, (keys + 15) // 16, 1 << 20, 16
    p.q_row_stride = p.o_row_stride = D
    assert lib.LIB.attn_prefill_paged_block_scaled(ctypes.byref(p), 1 << 20, 1 << 20, None, 0, ctypes.byref(need), None) == 0
    dense = 2 * (-(-B * Hk * keys * D * 2 // 256) * 256)
    return "few" if need.value < dense or not dense else "whole" if need.value == dense else "shares"


def _check_chunks(c, q, cu, lens, o, lse, causal, what):
    """Packed rows [T, Hq, D] and LSE [Hq, T] of a call over the case's pages against the definition."""
    Hq, Hk, D = c["Hq"], c["Hk"], c["D"]
    kv, vv = ref.values(c["kc"], c["ks"]), ref.values(c["vc"], c["vs"])
    for b, n in enumerate(lens):
        rows = cu[b + 1] - cu[b]
        if rows == 0:
            continue
        ids = c["table"][b, : (n + 15) // 16].long()
        k, v = (x[ids].transpose(0, 1).reshape(Hk, -1, D)[:, :n] for x in (kv, vv))
        ev = (c["vs"][ids].double() - 127).T.repeat_interleave(16, 1)[:, :n]
        limit = torch.arange(n - rows + 1, n + 1) if causal else torch.full((rows,), n)
        qs = q[cu[b]:cu[b + 1]].double().permute(1, 0, 2).reshape(Hk, Hq // Hk * rows, D)
        want, wl, tol, ltol = _attention_tol(qs, k, ev, v, c["scale"], limit.repeat(Hq // Hk), 2.0 ** -8 + 2.0 ** -11, 0)
        want, tol, wl, ltol = (x.reshape(Hq, rows, *x.shape[2:]) for x in (want, tol, wl, ltol))
        _within(o[cu[b]:cu[b + 1]].transpose(0, 1), want, tol + 2.0 ** -20 * want.abs(), f"{what} O {b}")
        # the running sum is made of exponentials within 2^-12 of the exact ones
        _within(lse[:, cu[b]:cu[b + 1]], wl, ltol + 2.0 ** -12, f"{what} LSE {b}")


def _run_chunks(lib, c, q, chunks, lens, keys, causal, packed, flags=None):
    """The call in packed or padded rows; O and LSE as packed ones, with the rows behind a padded sequence checked."""
    cu = [0] + torch.cumsum(torch.tensor(chunks), 0).tolist()
    most, Hq, D = max(chunks), c["Hq"], c["D"]
    dev = [c[n].cuda() for n in ("kc", "vc", "ks", "vs", "table")] + [_i32(lens).cuda()]
    kw = dict(scale=c["scale"], causal=causal, out_dtype=torch.float32, max_seqlen_k=keys, error_flags=flags)
    if packed:
        return lib.prefill_paged_block_scaled(q.cuda(), *dev, cu_seqlens_q=_i32(cu).cuda(), max_seqlen_q=most, **kw)
    pad = torch.zeros(len(chunks), Hq, most, D, dtype=torch.bfloat16)
    for b, n in enumerate(chunks):
        pad[b, :, :n] = q[cu[b]:cu[b + 1]].transpose(0, 1)
    out = torch.full(pad.shape, 7.0, device="cuda")
    lse = torch.full(pad.shape[:3], 7.0, device="cuda")
    lib.prefill_paged_block_scaled(pad.cuda(), *dev, seqlens_q=_i32(chunks).cuda(), out=out, lse=lse, **kw)
    for b, n in enumerate(chunks):
        assert (out[b, :, n:] == 7.0).all() and (lse[b, :, n:] == 7.0).all()
    return (torch.cat([out[b, :, :n].transpose(0, 1) for b, n in enumerate(chunks)]),
            torch.cat([lse[b, :, :n] for b, n in enumerate(chunks)], 1))


WHOLE = [(128, 5, 5), (128, 4, 2), (128, 3, 1), (128, 8, 2), (128, 16, 2), (64, 5, 5), (64, 4, 2), (64, 9, 3), (64, 8, 2), (64, 16, 2)]
# a first chunk, a sequence without rows, rows that see no key, one row, a chunk over earlier tokens, a full bound
CHUNKS, LENS = [500, 0, 300, 1, 130, 512], [500, 30, 200, 77, 333, 512]


@pytest.mark.parametrize("D,Hq,Hk", WHOLE)
def test_prefill_block_scaled_short_keys_take_whole_items(lib, D, Hq, Hk):
    assert _prefill_path(lib, len(CHUNKS), Hq, Hk, D, max(CHUNKS), 512) == "whole"


@gpu
@pytest.mark.parametrize("D,Hq,Hk", WHOLE)
@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_block_scaled_whole_items_match_definition(lib, D, Hq, Hk, packed, causal):
    """A bound of at most 512 keys and many rows, as the first chunks of a batch of prompts have them."""
    c = _decode_case(LENS, Hq, Hk, D, 61)
    q = torch.randn(sum(CHUNKS), Hq, D, generator=_gen(62)).to(torch.bfloat16)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = _run_chunks(lib, c, q, CHUNKS, LENS, 512, causal, packed, flags)
    cu = [0] + torch.cumsum(torch.tensor(CHUNKS), 0).tolist()
    _check_chunks(c, q, cu, LENS, o, lse, causal, "whole")
    if causal:  # 300 rows over 200 keys
        assert (o[cu[2]:cu[2] + 100] == 0).all() and torch.isneginf(lse[:, cu[2]:cu[2] + 100]).all()
    assert int(flags.item()) == 0


@gpu
@pytest.mark.parametrize("Hq,Hk", [(9, 3), (32, 4)])
def test_prefill_block_scaled_many_items_over_long_keys(lib, Hq, Hk):
    """More than 4096 items: each stays whole although the bound of the keys is long."""
    B, D, g = 700, 64, _gen(63)
    lens = [1 + int(x) for x in torch.randint(0, 60, (B,), generator=g)]
    chunks = [min(n, int(x)) for n, x in zip(lens, torch.randint(0, 6, (B,), generator=g))]
    lens[3], chunks[3], lens[400], chunks[400], lens[B - 1], chunks[B - 1] = 900, 256, 1300, 9, 777, 130
    most = max(chunks)
    assert _prefill_path(lib, B, Hq, Hk, D, most, 1300) == "whole"
    assert _prefill_path(lib, 40, Hq, Hk, D, most, 1300) == "shares"
    c = _decode_case(lens, Hq, Hk, D, 64)
    q = torch.randn(sum(chunks), Hq, D, generator=g).to(torch.bfloat16)
    o, lse = _run_chunks(lib, c, q, chunks, lens, 1300, True, True)
    _check_chunks(c, q, [0] + torch.cumsum(torch.tensor(chunks), 0).tolist(), lens, o, lse, True, "many")


@gpu
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_block_scaled_whole_items_nan_in_a_visible_key(lib, D):
    rows, n, Hq, Hk = 500, 510, 8, 2
    assert _prefill_path(lib, 4, Hq, Hk, D, rows, 510) == "whole"
    c = _decode_case([n] * 4, Hq, Hk, D, 65)
    q = torch.randn(4 * rows, Hq, D, generator=_gen(66)).to(torch.bfloat16)
    at = [10, 17, 300, 509]
    for b, t in enumerate(at):
        c["kc"][int(c["table"][b, t // 16]), 1, t % 16, 3 + b] = 0x7F
    o, lse = _run_chunks(lib, c, q, [rows] * 4, [n] * 4, n, True, True)
    for b, t in enumerate(at):
        x, y = o[b * rows:(b + 1) * rows].cpu(), lse[:, b * rows:(b + 1) * rows].cpu()
        sees = torch.arange(n - rows, n) >= t
        assert torch.isfinite(x[:, :4]).all() and torch.isfinite(y[:4]).all()
        for h in range(4, 8):
            assert torch.equal(torch.isnan(x[:, h]).all(-1), sees) and torch.equal(torch.isnan(y[h]), sees)
            assert torch.isfinite(x[~sees, h]).all()


# ---------------------------------------------------------------------------- value scales as far apart as their bytes allow

# A weight's exponent is a sum of numbers below 2^8, each rounding of which is off by at most 2^-17: two in a
# split, two in the merge of splits, one in the row's result: 5 * 2^-17 * ln 2 of the weight.
FAR = 5 * 2.0 ** -17 * 0.6932


def _balanced_case(lens, Hq, Hk, D, seed, order):
    """Every block's scores lie around 2^t and its values around 2^-t, t in [-100, 100]: the blocks decide the output
    alike, though their weights in the softmax are up to 2^200 apart. order: t ascends ("up"), descends, or is shuffled."""
    g = _gen(seed)
    c = _decode_case(lens, Hq, Hk, D, seed, 0.0)
    c["q"] = (c["q"].float() * 0.1).to(torch.bfloat16)
    c["q"][:, :, 0] = 1.0
    c["scale"] = 1.0
    for b, n in enumerate(lens):
        blocks = (n + 15) // 16
        t = torch.linspace(-100, 100, blocks) if blocks > 1 else torch.zeros(blocks)
        t = {"up": t, "down": t.flip(0), "shuffled": t[torch.randperm(blocks, generator=g)]}[order]
        k0 = (t * math.log(2)).to(torch.float8_e4m3fn)  # 4 significant bits: the values follow what it became
        for j in range(blocks):
            blk, live = int(c["table"][b, j]), min(16, n - 16 * j)
            c["ks"][blk] = 127
            c["kc"][blk, :, :live] = torch.randn(Hk, live, D, generator=g).to(torch.float8_e4m3fn).view(torch.uint8)
            c["kc"][blk, :, :live, 0] = k0.view(torch.uint8)[j]
            c["vs"][blk] = 120 - round(float(k0[j]) / math.log(2))
    return c


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("order", ["up", "down", "shuffled"])
def test_decode_block_scaled_scales_of_any_distance(lib, order, D):
    c = _balanced_case([3000, 200, 33], 8, 2, D, 5 + D, order)
    o, lse, tol, ltol = _decode_want(c)
    pv = _values_sum(c)
    for splits in (1, 0, 4, 16):
        go, gl, flags = _decode_run(lib, c, num_splits=splits, out_dtype=torch.float32, max_seq_len=3000)
        assert flags == 0
        _within(go, o, tol + FAR * pv + 2.0 ** -21 * o.abs(), f"O splits {splits}")
        _within(gl, lse, ltol, f"LSE splits {splits}")


def _values_sum(c):
    """sum_j p_j |v_j| of every row."""
    kv, vv = ref.values(c["kc"], c["ks"]), ref.values(c["vc"], c["vs"])
    out = []
    for b, n in enumerate(c["lens"]):
        ids = c["table"][b, : (n + 15) // 16].long()
        k, v = (x[ids].transpose(0, 1).reshape(c["Hk"], -1, c["D"])[:, :n] for x in (kv, vv))
        q = c["q"][b].double().reshape(c["Hk"], -1, c["D"])
        out.append(ref.attend_ref(q, k, v, c["scale"], torch.full((q.shape[1],), n))[2].reshape(c["Hq"], c["D"]))
    return torch.stack(out)


def _few_rows_want(c, q, table, n, limit):
    """One sequence's rows [Hq, rows, D] by the definition, with the tolerances of the few-rows kernel."""
    Hk, (Hq, rows, D) = c["Hk"], q.shape
    ids = table[: (n + 15) // 16].long()
    k, v = (ref.values(c[a], c[s])[ids].transpose(0, 1).reshape(Hk, -1, D)[:, :n] for a, s in (("kc", "ks"), ("vc", "vs")))
    ev = (c["vs"][ids].double() - 127).T.repeat_interleave(16, 1)[:, :n]
    qs, limit = q.double().reshape(Hk, Hq // Hk * rows, D), limit.repeat(Hq // Hk)
    want, wl, tol, ltol = _attention_tol(qs, k, ev, v, c["scale"], limit, 2.0 ** -11, 2.0 ** -25)
    tol = tol + FAR * ref.attend_ref(qs, k, v, c["scale"], limit)[2] + 2.0 ** -21 * want.abs()
    return [x.reshape(Hq, rows, *x.shape[2:]) for x in (want, wl, tol, ltol)]


@gpu
@pytest.mark.parametrize("context", [500, 40000])
@pytest.mark.parametrize("order", ["up", "shuffled"])
def test_prefill_block_scaled_short_chunk_scales_of_any_distance(lib, order, context):
    """Three rows go to the few-rows kernel: one cluster, and (40000 keys) several."""
    rows, D, Hq, Hk = 3, 128, 4, 2
    n = context + rows
    c = _balanced_case([n], Hq, Hk, D, 7, order)
    q = (torch.randn(1, Hq, rows, D, generator=_gen(9)) * 0.1).to(torch.bfloat16)
    q[..., 0] = 1.0
    dev = [c[k].cuda() for k in ("kc", "vc", "ks", "vs", "table")]
    o, lse = lib.prefill_paged_block_scaled(q.cuda(), *dev, _i32([n]).cuda(), scale=1.0, out_dtype=torch.float32, max_seqlen_k=n)
    want, wl, tol, ltol = _few_rows_want(c, q[0], c["table"][0], n, torch.arange(context + 1, n + 1))
    _within(o[0], want, tol, "O")
    _within(lse[0], wl, ltol, "LSE")


# ---------------------------------------------------------------------------- rotary: far positions


def _remainder(position, freq):
    """position * freq (an fp64 number, exactly) modulo 2 pi, in [-pi, pi], rounded once to 64 bits."""
    getcontext().prec = 60
    tau = Fraction(2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459"))
    a = Fraction(freq) * position
    return float(a - round(a / tau) * tau)


@gpu
@pytest.mark.parametrize("fast", [False, True])
def test_rotary_keeps_its_accuracy_at_far_positions(lib, fast):
    """fp32 rows at positions up to 2^31 - 1, both ways round, within the bound of near ones: the usual frequencies,
    and up to a turn per position, where one 64-bit product would be off by 2^-18 rad."""
    pos = [2 ** 31 - 1, 2 ** 31 - 1000, 2 ** 30 + 1, 2 ** 28 + 12345, 2 ** 27 - 7, 999999937, 5]
    freq = torch.linspace(0.1, 6.2, 64, dtype=torch.float64) if fast else ref.frequencies(128)
    x = torch.randn(len(pos), 3, 128, generator=_gen(3))
    a = torch.tensor([[_remainder(p, f) for f in freq.tolist()] for p in pos], dtype=torch.float64)[:, None]
    x1, x2 = x.double().split(64, -1)
    size = torch.cat((x1.abs() + x2.abs(),) * 2, -1)
    for sign, inverse in ((1.0, False), (-1.0, True)):
        y, _ = lib.rotary(x.cuda(), None, freq.cuda(), _i32(pos).cuda(), inverse=inverse)
        c, s = torch.cos(a), torch.sin(a) * sign
        _within(y, torch.cat((x1 * c - x2 * s, x2 * c + x1 * s), -1), size * ref.TURN_REL, "far")


# ---------------------------------------------------------------------------- faults: what is left out, what is kept


def _guarded(shape, dtype):
    """A contiguous output inside a larger buffer of 7s, and the check that its surroundings are still 7."""
    buf = torch.full((shape[0] + 8, *shape[1:]), 7.0, dtype=dtype, device="cuda")
    return buf[4:-4], lambda: bool((buf[:4] == 7.0).all() and (buf[-4:] == 7.0).all())


def _decode_guarded(lib, c, **kw):
    B = len(c["lens"])
    out, out_kept = _guarded((B, c["Hq"], c["D"]), torch.float32)
    lse, lse_kept = _guarded((B, c["Hq"]), torch.float32)
    _, _, flags = _decode_run(lib, c, out=out, lse=lse, **kw)
    assert out_kept() and lse_kept()
    return out, lse, flags


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("splits", [0, 1, 2, 16])
def test_decode_block_scaled_leaves_the_keys_of_bad_blocks_out(lib, D, splits):
    """An entry outside the pool in the middle, and at the end of a long sequence: flagged, its keys are not seen."""
    c = _decode_case([64, 64, 2500], 4, 1, D, 9)
    fine = {k: v for k, v in c.items()}
    fine["table"], fine["lens"] = c["table"].clone(), [64, 48, 2496]
    fine["table"][1, 2] = c["table"][1, 3]  # three blocks are left
    want, wl, tol, ltol = _decode_want(fine)
    for bad in (10 ** 6, -1):
        c["table"][1, 2] = c["table"][2, 156] = bad  # the second one holds the last four tokens
        o, lse, flags = _decode_guarded(lib, c, num_splits=splits)
        assert flags == lib.ATTN_FAULT_BAD_BLOCK
        _within(o, want, tol + 2.0 ** -21 * want.abs(), "O")
        _within(lse, wl, ltol, "LSE")


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("splits", [0, 1, 16])
def test_decode_block_scaled_cuts_sequences_at_the_bound(lib, D, splits):
    c = _decode_case([64, 10, 700], 4, 1, D, 10)
    for bound in (30, 16, 400):
        cut = {**c, "lens": [min(n, bound) for n in c["lens"]]}
        want, wl, tol, ltol = _decode_want(cut)
        o, lse, flags = _decode_guarded(lib, c, num_splits=splits, max_seq_len=bound)
        assert flags == lib.ATTN_FAULT_BAD_LENGTH
        _within(o, want, tol + 2.0 ** -21 * want.abs(), "O")
        _within(lse, wl, ltol, "LSE")


@gpu
@pytest.mark.parametrize("rows,keys,path", [(3, 400, "few"), (400, 500, "whole"), (400, 2000, "shares")])
def test_prefill_block_scaled_of_bad_blocks(lib, rows, keys, path):
    """An entry outside the pool is flagged. The few-rows kernel leaves its keys out, the tensor-core tiles read zeros."""
    Hq, Hk, D, B = 16, 2, 128, 2
    assert _prefill_path(lib, B, Hq, Hk, D, rows, keys) == path
    c = _decode_case([keys, keys - 7], Hq, Hk, D, 11)
    q = torch.randn(B, Hq, rows, D, generator=_gen(12)).to(torch.bfloat16).cuda()
    kw = dict(scale=c["scale"], causal=False, out_dtype=torch.float32, max_seqlen_k=keys)
    dev = [c[n].cuda() for n in ("kc", "vc", "ks", "vs")]
    table, lens = c["table"].clone(), _i32(c["lens"])
    spare = next(i for i in range(c["kc"].shape[0]) if i not in set(c["table"].flatten().tolist()))
    if path == "few":
        table[0, 5:-1] = c["table"][0, 6:].clone()  # one block less
        exact = _few_rows_want(c, q[0].cpu(), table[0], keys - 16, torch.full((rows,), keys - 16))
        table = c["table"].clone()
    else:
        table[0, 5] = spare
        for t in dev[:2]:
            t[spare] = 0
        for t in dev[2:]:
            t[spare] = 127
    want, wl = lib.prefill_paged_block_scaled(q, *dev, table.cuda(), lens.cuda(), **kw)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    table, lens = c["table"].clone(), _i32(c["lens"])
    table[0, 5] = 10 ** 7
    o, lse = lib.prefill_paged_block_scaled(q, *dev, table.cuda(), lens.cuda(), error_flags=flags, **kw)
    assert int(flags.item()) == lib.ATTN_FAULT_BAD_BLOCK and torch.equal(o[1], want[1]) and torch.equal(lse[1], wl[1])
    if path == "few":
        _within(o[0], exact[0], exact[2], "O")
        _within(lse[0], exact[1], exact[3], "LSE")
    else:
        assert torch.equal(o[0], want[0]) and torch.equal(lse[0], wl[0])


@gpu
def test_workspaces_that_repeat_memory_are_refused(lib):
    """An expanded tensor counts more elements than it has memory."""
    c = _decode_case([2500, 40], 4, 2, 64, 13)
    dev = [c[n].cuda() for n in ("kc", "vc", "ks", "vs", "table")] + [_i32(c["lens"]).cuda()]
    q, wide = c["q"].cuda(), torch.zeros(256, dtype=torch.uint8, device="cuda").expand(1 << 16, 256)
    with pytest.raises(ValueError):
        lib.decode_paged_block_scaled(q, *dev, num_splits=16, workspace=wide)
    with pytest.raises(ValueError):
        lib.prefill_paged_block_scaled(q[:, :, None].expand(2, 4, 500, 64).contiguous(), *dev, workspace=wide)


# ---------------------------------------------------------------------------- graphs and streams


@gpu
@pytest.mark.parametrize("in_place", [True, False])
def test_a_large_plan_is_replayed(lib, in_place):
    """Many CTAs, and over the old state a dependent launch that advances it: captured once, replayed."""
    B, most, width = 300, 40, 16
    g = _gen(71)
    seq, new = _i32(torch.randint(0, 100, (B,), generator=g)), _i32(torch.randint(0, most + 1, (B,), generator=g))
    pages = torch.randperm(3 * B * width, generator=g).to(torch.int32)
    table, free = pages[: B * width].reshape(B, width).clone(), pages[B * width:].contiguous()
    total, cap = int(new.sum()) + 3, width * 16
    assert total > 2048
    d = [t.cuda() for t in (seq, new, table, free, _i32([0]))]
    outs = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (B, B + 1, total, total, 1)]
    if in_place:
        outs[0], outs[4] = d[0], d[4]

    def step():
        lib.plan_paged_step(*d, total, 3 * B * width, seq_lens_out=outs[0], cu_seqlens_q=outs[1], positions=outs[2],
                            slot_map=outs[3], num_used_out=outs[4])
    start = [t.clone() for t in (d[0], d[2], d[4])]
    step()
    for t, x in zip((d[0], d[2], d[4]), start):
        t.copy_(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    state = (seq, table, 0)
    for _ in range(3):
        graph.replay()
        want = _plan_by_rows(state[0], new, state[1], free, state[2], total, cap)
        for name, a, b in zip(("lens", "cu", "positions", "slots", "used", "table"), outs + [d[2]], want):
            assert torch.equal(a.cpu(), b), name
        if in_place:
            state = (want[0], want[5], int(want[4]))
        else:
            state = (state[0], want[5], 0)


@gpu
@pytest.mark.parametrize("splits", [2, 16])
def test_decode_block_scaled_in_a_graph_and_on_two_streams(lib, splits):
    """One cluster and several: captured and replayed on two streams beside eager calls, as the lengths grow."""
    cases = []
    for seed in (81, 82):
        c = _decode_case([3000, 70, 1, 900], 8, 2, 128, seed)
        dev = [c[n].cuda() for n in ("q", "kc", "vc", "ks", "vs", "table")]
        lens = _i32(c["lens"]).cuda()
        cases.append((lens, lambda dev=dev, lens=lens: lib.decode_paged_block_scaled(*dev, lens, num_splits=splits, max_seq_len=3000)))
    for _, f in cases:
        f()
    torch.cuda.synchronize()
    graphs = []
    for _, f in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = f()
        graphs.append((graph, out))
    streams = [torch.cuda.Stream() for _ in cases]
    for lengths in ([3000, 70, 1, 900], [16, 0, 1, 17], [2999, 69, 0, 899]):
        for lens, _ in cases:
            lens.copy_(_i32(lengths))
        want = [f() for _, f in cases]
        torch.cuda.synchronize()
        both = []
        for (graph, _), (_, f), s in zip(graphs, cases, streams):
            with torch.cuda.stream(s):
                graph.replay()
                both.append(f())
        torch.cuda.synchronize()
        for w, (_, o), e in zip(want, graphs, both):
            for i in (0, 1):
                assert torch.equal(w[i], o[i]) and torch.equal(w[i], e[i])
